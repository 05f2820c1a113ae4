"""The scaled embedding lookup and its gradient (include/policy.h, embed_*) on
the GPU against their 64-bit forms, within policy_ref's bounds."""
import numpy as np
import pytest
import torch

import policy_ref as ref
from parity import gpu_available
from test_gpu_recur import TYPES, f64, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X")]


@pytest.fixture(scope="module")
def rx():
    import rl_experience_collection_amd as rx
    return rx


def check(rx, w, idx, dout, name, scale=1.5, gpu_w=None, gpu_dout=None):
    leaf = (w.cuda() if gpu_w is None else gpu_w).detach().requires_grad_()
    out = rx.embed(leaf, idx.cuda(), scale=scale)
    s = float(np.float32(scale))
    want, bound = ref.embed(f64(w), idx.numpy(), s, name)
    within(out, want, bound, "out")
    g, = torch.autograd.grad(out, leaf, dout.cuda() if gpu_dout is None else gpu_dout)
    want, bound = ref.embed_grad(f64(dout), idx.numpy(), w.shape[0], s, name)
    within(g, want, bound, "dweight")
    return out, g


def inputs(M, V, D, name, seed, spread="even", out_of_range=0.05):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(V, D, generator=g).to(TYPES[name])
    dout = torch.randn(M, D, generator=g).to(TYPES[name])
    if spread == "one":
        idx = torch.full((M,), V // 2)
    elif spread == "skew":
        idx = (V ** torch.rand(M, generator=g)).long().clamp(1, V) - 1
    else:
        idx = torch.randint(0, V, (M,), generator=g)
    bad = torch.rand(M, generator=g) < out_of_range
    idx[bad] = torch.tensor([-1, V, -2 ** 31, 2 ** 31 - 1])[torch.arange(int(bad.sum())) % 4]
    return w, idx.int(), dout


SIZES = [(1, 1, 1), (3, 2, 5), (64, 45, 128), (65, 1, 8), (255, 511, 6), (256, 512, 4),
         (257, 513, 33), (2047, 45, 3), (2049, 45, 16), (5000, 3, 40), (3, 70000, 2),
         (9000, 262145, 1), (700, 300, 1000), (511, 40, 9), (512, 31, 500), (513, 33, 511), (1030, 70, 257),
         (600, 600, 15), (1500, 20, 520)]


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,V,D", SIZES)
def test_matches_the_formula(rx, M, V, D, name):
    check(rx, *inputs(M, V, D, name, M + V + D), name)


@pytest.mark.parametrize("spread", ["one", "skew"])
@pytest.mark.parametrize("M,V,D", [(1, 9, 4), (31, 9, 4), (32, 9, 4), (33, 9, 7), (4096, 50, 8),
                                   (140001, 45, 5), (20000, 5000, 2)])
def test_hot_rows(rx, M, V, D, spread):
    check(rx, *inputs(M, V, D, "f32", M, spread), "f32")
    check(rx, *inputs(M, V, D, "bf16", M, spread, out_of_range=0.0), "bf16")


def test_nothing_named(rx):
    w, idx, dout = inputs(50, 7, 12, "f32", 1)
    idx[:] = -1
    out, g = check(rx, w, idx, dout, "f32")
    assert (out == 0).all() and (g == 0).all()
    # a NaN in the gradient of an index that names nothing goes nowhere
    dout[:] = float("nan")
    leaf = w.cuda().requires_grad_()
    g, = torch.autograd.grad(rx.embed(leaf, idx.cuda()), leaf, dout.cuda())
    assert (g == 0).all()


def test_empty_sizes(rx):
    for shape, idx_shape in [((5, 3), (0,)), ((5, 3), (4, 0)), ((5, 0), (4,)), ((0, 3), (4,))]:
        w = torch.randn(shape, device="cuda", requires_grad=True)
        idx = torch.zeros(idx_shape, dtype=torch.int64, device="cuda")
        out = rx.embed(w, idx)
        assert tuple(out.shape) == idx_shape + shape[1:] and (out == 0).all()
        g, = torch.autograd.grad(out.sum(), w)
        assert g.shape == w.shape and (g == 0).all()


@pytest.mark.parametrize("name", ["f32", "f16"])
def test_layouts(rx, name):
    """int64 indices of two dimensions, rows apart and off their alignment, a
    gradient that is one row repeated."""
    w, idx, dout = inputs(60, 20, 12, name, 3)
    wide = torch.zeros(20, 19, dtype=TYPES[name], device="cuda")
    for lo in (0, 3, 4):
        wide[:, lo:lo + 12] = w.cuda()
        check(rx, w, idx.long().view(5, 12), dout.view(5, 12, 12), name, gpu_w=wide[:, lo:lo + 12])
    rep = dout[:1].expand(60, 12)
    check(rx, w, idx, rep, name, gpu_dout=dout[:1].cuda().expand(60, 12))


def test_far_offsets(rx):
    """Rows whose offset passes 2^32 elements and bytes: the last rows of a
    weight of 4.4 G elements are read, and their gradient lands there."""
    V, D = 4_300_000, 1024
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    w[-3:] = torch.arange(3, device="cuda")[:, None] + 1
    idx = torch.tensor([V - 1, 0, V - 3, V, V - 1, V - 2], dtype=torch.int32, device="cuda")
    leaf = w.requires_grad_()
    out = rx.embed(leaf, idx, scale=2.0)
    assert out[:, 0].tolist() == [6.0, 0.0, 2.0, 0.0, 6.0, 4.0] and (out == out[:, :1]).all()
    g, = torch.autograd.grad(out, leaf, torch.ones_like(out))
    assert g[-3:, 5].tolist() == [2.0, 2.0, 4.0] and g[0, 7] == 2.0
    assert float(g[1:-3].abs().max()) == 0.0
    # and far rows of the output
    big = torch.zeros(V, dtype=torch.int32, device="cuda")
    big[-1] = V - 1
    out = rx.embed(leaf.detach(), big)
    assert (out[-1] == 3).all() and float(out[:-1].abs().max()) == 0.0


def test_rows_between_the_outputs_are_left_alone(rx):
    from rl_experience_collection_amd import policy
    w, idx, dout = inputs(40, 30, 5, "f32", 7)
    lib, s = rx.load_library(), torch.cuda.current_stream().cuda_stream
    cw, ci, cd = w.cuda(), idx.cuda(), dout.cuda()
    out = torch.full((41, 8), 7.0, device="cuda")
    dw = torch.full((31, 8), 7.0, device="cuda")
    assert lib.embed_forward(0, cw.data_ptr(), 30, 5, 5, ci.data_ptr(), 4, 40, 2.0, out.data_ptr(), 8, s) == 0
    size = lib.embed_workspace(0, 30, 5, 40)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert lib.embed_backward(0, cd.data_ptr(), 5, ci.data_ptr(), 4, 40, 30, 5, 2.0, dw.data_ptr(), 8,
                              ws.data_ptr(), size, s) == 0
    torch.cuda.synchronize()
    assert (out[40] == 7).all() and (out[:, 5:] == 7).all()
    assert (dw[30] == 7).all() and (dw[:, 5:] == 7).all()
    within(out[:40, :5], *ref.embed(f64(w), idx.numpy(), 2.0, "f32"), "out")
    within(dw[:30, :5], *ref.embed_grad(f64(dout), idx.numpy(), 30, 2.0, "f32"), "dweight")


@pytest.mark.parametrize("M,V", [(100, 45), (30000, 3000)])
def test_captured_training_pass(rx, M, V):
    """Two graphs replayed in turn on new inputs, eager calls between: the
    eager bits each time."""
    data = [inputs(M, V, 16, "bf16", s, "skew") for s in (1, 2, 3)]
    buf = [t.cuda() for t in data[0]]

    def once(w, idx, dout):
        leaf = w.detach().requires_grad_()
        out = rx.embed(leaf, idx, 3.0)
        return out.detach(), torch.autograd.grad(out, leaf, dout)[0]

    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        once(*buf)
    st.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            out = once(*buf)
        graphs.append((g, out))
    for d in data + data:
        for b, v in zip(buf, d):
            b.copy_(v)
        want = once(*[t.cuda() for t in d])
        for g, out in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_two_streams_at_once(rx):
    data = [[t.cuda() for t in inputs(20000, 600, 24, "f32", s, "skew")] for s in (1, 2)]

    def once(w, idx, dout):
        leaf = w.detach().requires_grad_()
        return torch.autograd.grad(rx.embed(leaf, idx), leaf, dout)[0]

    want = [once(*d) for d in data]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in data], []
    for _ in range(4):
        for d, st in zip(data, streams):
            with torch.cuda.stream(st):
                got.append(once(*d))
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        assert torch.equal(g, want[k % 2])


@pytest.mark.parametrize("spread", ["even", "skew", "one"])
@pytest.mark.parametrize("M,V,D", [(300, 8191, 9), (512, 8192, 40), (511, 16384, 6), (77, 40000, 24),
                                   (512, 270000, 4)])
def test_few_indices_in_a_large_vocabulary(rx, M, V, D, spread):
    check(rx, *inputs(M, V, D, "bf16", M + V, spread), "bf16")


def test_wide_indices_that_name_no_row(rx):
    """64-bit indices whose low words alone would name one."""
    w, _, dout = inputs(6, 9, 8, "f32", 2)
    idx = torch.tensor([3, 2 ** 32 + 3, -2 ** 32 + 3, 3 - 2 ** 63, 8, 2 ** 62])
    check(rx, w, idx, dout, "f32")
    big = idx.repeat(200)
    check(rx, w, big, dout.repeat(200, 1), "f32")


@pytest.mark.parametrize("spread", ["even", "skew", "one"])
@pytest.mark.parametrize("M,V,D", [(1023, 45, 128), (1024, 45, 129), (1025, 45, 128), (1000, 3, 700), (1024, 300000, 9),
                                   (640, 20000, 300), (900, 33, 1)])
def test_about_a_thousand_indices(rx, M, V, D, spread):
    check(rx, *inputs(M, V, D, "f32", M + D, spread), "f32")
    check(rx, *inputs(M, V, D, "bf16", M + D, spread, out_of_range=0.0), "bf16")


def test_indices_of_neighbouring_rows(rx):
    """All of them within the rows that one workgroup owns, in mixed order."""
    w, idx, dout = inputs(1024, 270000, 40, "f32", 4)
    idx = torch.randint(5 * 32 - 3, 6 * 32 + 3, (1024,), generator=torch.Generator().manual_seed(5)).int()
    check(rx, w, idx, dout, "f32")
