"""Penalties, bias and mask on logits (include/policy.h, logits_*) on the GPU
against their 64-bit form, within policy_ref's bounds."""
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


def bits_of(allowed):
    """[K, V] truth values -> [K, ceil(V / 32)] int32; the bits past V are set."""
    K, V = allowed.shape
    W = (V + 31) // 32
    full = np.ones((K, W * 32), np.uint64)
    full[:, :V] = allowed
    words = (full.reshape(K, W, 32) << np.arange(32, dtype=np.uint64)).sum(2)
    return torch.from_numpy(words.astype(np.uint32).view(np.int32))


def inputs(R, V, H, name, seed, mask="none", bias=True):
    """Tensors for shape_logits on the CPU, and the reference's arguments."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    a = dict(logits=(torch.randn(R, V, generator=g) * 3).to(TYPES[name]))
    a["bias"] = torch.randn(V, generator=g) if bias else None
    if H:
        h = torch.randint(-2, V + 2, (R, H), generator=g)
        h[:, ::3] = h[:, :1].clone()  # repeats
        a["history"] = h.int()
        a["history_len"] = torch.randint(-1, H + 2, (R,), generator=g).int()
    for k, lo, hi in (("repetition", 0.7, 1.6), ("presence", -0.5, 1.0), ("frequency", 0.0, 0.3)):
        a[k] = lo + (hi - lo) * torch.rand(R, generator=g)
    allowed = None
    if mask != "none":
        K = dict(bytes=R, bits=R, shared=1, table=5)[mask]
        table = rng.random((K, V)) < 0.6
        table[-1] = False  # nothing allowed there
        a["mask"] = torch.from_numpy(table) if mask in ("bytes", "shared") else bits_of(table)
        allowed = table
        if mask == "table":
            rows = rng.integers(-2, K + 2, R).astype(np.int32)
            a["mask_rows"] = torch.from_numpy(rows)
            allowed = np.concatenate([table, np.ones((1, V), bool)])[
                np.where((rows >= 0) & (rows < K), rows, K)]
    return a, allowed


def check(rx, a, allowed, name, seed=0, train=True, gpu=None):
    gpu = dict({k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in a.items()}, **(gpu or {}))
    leaves = [gpu["logits"].detach().requires_grad_()]
    gpu["logits"] = leaves[0]
    if gpu.get("bias") is not None and gpu["bias"].dim() == 1:
        gpu["bias"] = gpu["bias"].detach().requires_grad_()
        leaves.append(gpu["bias"])
    out = rx.shape_logits(**gpu)
    V = out.shape[-1]
    dout = torch.randn(out.shape, generator=torch.Generator().manual_seed(seed)).to(out.dtype)
    np_ = {k: (f64(v) if v.is_floating_point() else v.numpy().reshape(-1, v.shape[-1]) if k == "history"
               else v.numpy().reshape(-1)) if isinstance(v, torch.Tensor) else v
           for k, v in a.items() if k not in ("mask", "mask_rows")}
    z = np_.pop("logits").reshape(-1, V)
    if np_.get("bias") is not None and np_["bias"].ndim > 1:
        np_["bias"] = np_["bias"].reshape(-1, V)
    w = ref.logits(z, name, allowed=allowed, dout=f64(dout).reshape(-1, V),
                   **{k: v for k, v in np_.items() if v is not None})
    got = f64(out).reshape(-1, V)
    assert (np.isneginf(got) == np.isneginf(w["out"])).all()
    fin = ~np.isneginf(got)
    off = np.abs(np.where(fin, got, 0) - np.where(fin, w["out"], 0)) - w["eout"]
    assert (off <= 0).all(), float(off.max())
    if train:
        g = torch.autograd.grad(out, leaves, dout.cuda())
        within(g[0].reshape(-1, V), w["dlogits"], w["edl"], "dlogits")
        if len(leaves) > 1:
            within(g[1], w["dbias"], w["edb"], "dbias")
    return out


SIZES = [(1, 1, 1), (3, 2, 4), (5, 7, 0), (128, 45, 20), (1000, 45, 3), (4097, 3, 2), (17, 2047, 9),
         (9, 2048, 70), (6, 2049, 300), (3, 4096, 5), (2, 4097, 1100), (2, 20011, 64), (600, 31, 1),
         (70, 32, 33), (300, 1, 5)]


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("mask", ["none", "bytes", "bits", "shared", "table"])
@pytest.mark.parametrize("R,V,H", SIZES)
def test_matches_the_formula(rx, R, V, H, mask, name):
    check(rx, *inputs(R, V, H, name, R + V + H, mask), name)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("mask", ["none", "bytes", "bits", "shared", "table"])
@pytest.mark.parametrize("R,V,H", [(512, 45, 20), (513, 45, 20), (1200, 45, 20), (2600, 33, 300), (600, 512, 9),
                                   (601, 513, 9), (520, 1024, 70), (530, 1025, 4), (9000, 1, 3), (700, 257, 0)])
def test_many_rows(rx, R, V, H, mask, name):
    check(rx, *inputs(R, V, H, name, R + V + H, mask), name)


def test_many_rows_in_place_and_masked(rx):
    """Tiles of many rows: written over their own input; what a masked place
    holds does not matter; each argument left out."""
    a, allowed = inputs(700, 45, 20, "f32", 12, "bits")
    c = {k: v.cuda() for k, v in a.items()}
    want = rx.shape_logits(**c)
    z = torch.where(torch.from_numpy(allowed).cuda(), c["logits"], float("nan"))
    out = rx.shape_logits(**dict(c, logits=z), out=z)
    assert out is z and torch.equal(z, want)
    for drop in ("bias", "history_len", "repetition", "presence", "frequency", "mask"):
        check(rx, {k: v for k, v in a.items() if k != drop}, None if drop == "mask" else allowed, "f32")
    b = dict(a, bias=torch.randn(700, 45))
    check(rx, b, allowed, "f32")


@pytest.mark.parametrize("drop", ["bias", "history_len", "repetition", "presence", "frequency"])
def test_each_argument_alone(rx, drop):
    a, allowed = inputs(40, 45, 20, "f32", 5, "bits")
    a = {k: v for k, v in a.items() if k != drop}
    check(rx, a, allowed, "f32")
    a = {k: v for k, v in a.items() if k in ("logits", "mask")}
    check(rx, a, allowed, "f32")
    check(rx, dict(a, history=inputs(40, 45, 20, "f32", 6)[0]["history"], repetition=1.25, presence=0.5,
                   frequency=0.125), allowed, "f32")


@pytest.mark.parametrize("V", [45, 3001])
def test_more_dimensions_and_row_strides(rx, V):
    a, _ = inputs(24, V, 11, "bf16", 8, "bytes")
    allowed = a["mask"].numpy()
    b = {k: v.reshape((4, 6) + tuple(v.shape[1:])) if k != "bias" else v for k, v in a.items()}
    check(rx, b, allowed, "bf16")
    b["bias"] = torch.randn(4, 6, V)
    check(rx, b, allowed, "bf16")
    wide = torch.full((24, V + 5), float("nan"), dtype=torch.bfloat16, device="cuda")
    for lo in (0, 3):
        wide[:, lo:lo + V] = a["logits"].cuda()
        check(rx, a, allowed, "bf16", gpu=dict(logits=wide[:, lo:lo + V]))
        wide[:] = float("nan")


@pytest.mark.parametrize("V", [45, 2049])
def test_masked_places_do_not_matter(rx, V):
    """NaN, infinities and the type's lowest value at masked places, in the
    logits, the bias and the gradient."""
    a, allowed = inputs(20, V, 8, "f32", 9, "bits")
    c = {k: v.cuda() for k, v in a.items()}
    ok = torch.from_numpy(allowed).cuda()
    want = rx.shape_logits(**c)
    dout = torch.randn_like(want)
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(torch.float32).min):
        z = torch.where(ok, c["logits"], bad).requires_grad_()
        bias = c["bias"].clone().requires_grad_()
        got = rx.shape_logits(**dict(c, logits=z, bias=bias))
        assert torch.equal(got, want)
        g, gb = torch.autograd.grad(got, (z, bias), torch.where(ok, dout, bad))
        assert torch.isfinite(g).all() and (g[~ok] == 0).all() and torch.isfinite(gb).all()
    # the lowest value where it is allowed stays that value, or goes to -inf
    z = torch.full_like(want, torch.finfo(torch.float32).min)
    got = rx.shape_logits(z, mask=c["mask"])
    assert (got[ok] == torch.finfo(torch.float32).min).all() and torch.isneginf(got[~ok]).all()


def test_unmasked_infinities_and_nan_pass(rx):
    z = torch.tensor([[float("inf"), -float("inf"), float("nan"), 1.0]], device="cuda")
    h = torch.tensor([[0, 1, 2, 3, 3]], dtype=torch.int32, device="cuda")
    got = rx.shape_logits(z, history=h, repetition=2.0, presence=0.5, frequency=0.25)[0].tolist()
    assert got[0] == float("inf") and got[1] == -float("inf") and got[2] != got[2]
    assert got[3] == 0.5 - 0.5 - 0.5


@pytest.mark.parametrize("R,V", [(30, 45), (3, 5000)])
def test_in_place(rx, R, V):
    a, _ = inputs(R, V, 6, "bf16", 10, "table")
    c = {k: v.cuda() for k, v in a.items()}
    want = rx.shape_logits(**c)
    out = rx.shape_logits(**c, out=c["logits"])
    assert out is c["logits"] and torch.equal(out, want)


def test_empty_sizes(rx):
    for shape in [(0, 45), (4, 0), (0, 0), (2, 0, 45)]:
        z = torch.randn(shape, device="cuda", requires_grad=True)
        b = torch.zeros(shape[-1], device="cuda", requires_grad=True)
        out = rx.shape_logits(z, bias=b)
        assert out.shape == z.shape
        g, gb = torch.autograd.grad(out.sum(), (z, b))
        assert g.shape == z.shape and (gb == 0).all()
    one = rx.shape_logits(torch.ones(45, device="cuda"), history=torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert (one == 1).all()
    none = rx.shape_logits(torch.ones(2, 40, device="cuda"),
                           mask=torch.zeros(0, 2, dtype=torch.int32, device="cuda"),
                           mask_rows=torch.tensor([0, -1], dtype=torch.int32, device="cuda"))
    assert (none == 1).all()  # a table without rows bans nothing


def test_one_gradient_only(rx):
    a, allowed = inputs(50, 45, 5, "f32", 11, "bytes")
    c = {k: v.cuda() for k, v in a.items()}
    dout = torch.randn(50, 45, device="cuda")
    z, b = c["logits"].clone().requires_grad_(), c["bias"].clone().requires_grad_()
    both = torch.autograd.grad(rx.shape_logits(**dict(c, logits=z, bias=b)), (z, b), dout)
    gz, = torch.autograd.grad(rx.shape_logits(**dict(c, logits=z)), z, dout)
    gb, = torch.autograd.grad(rx.shape_logits(**dict(c, bias=b)), b, dout)
    assert torch.equal(gz, both[0]) and torch.equal(gb, both[1])


def test_rows_between_the_outputs_are_left_alone(rx):
    import ctypes as C
    from rl_experience_collection_amd import policy
    lib, s = rx.load_library(), torch.cuda.current_stream().cuda_stream
    for V in (5, 3000):
        z = torch.randn(7, V, device="cuda")
        out = torch.full((8, V + 3), 7.0, device="cuda")
        grad = out.clone()
        a = policy.LogitsArgs(rows=7, vocab=V, dtype=0, logits=z.data_ptr(), logits_row=V, repetition=1.0)
        assert lib.logits_forward(C.byref(a), out.data_ptr(), V + 3, s) == 0
        assert lib.logits_backward(C.byref(a), z.data_ptr(), V, grad.data_ptr(), V + 3, None, None, 0, s) == 0
        torch.cuda.synchronize()
        for t in (out, grad):
            assert torch.equal(t[:7, :V], z) and (t[7] == 7).all() and (t[:, V:] == 7).all()


@pytest.mark.parametrize("R,V", [(200, 45), (3, 9000), (2000, 45)])
def test_captured_training_pass(rx, R, V):
    data = [{k: v.cuda() for k, v in inputs(R, V, 9, "bf16", s, "table")[0].items()} for s in (1, 2, 3)]
    buf = {k: v.clone() for k, v in data[0].items()}
    dout = torch.randn(R, V, device="cuda").bfloat16()

    def once(c):
        z, b = c["logits"].detach().requires_grad_(), c["bias"].detach().requires_grad_()
        out = rx.shape_logits(**dict(c, logits=z, bias=b))
        return (out.detach(),) + torch.autograd.grad(out, (z, b), dout)

    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        once(buf)
    st.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            out = once(buf)
        graphs.append((g, out))
    for d in data + data:
        for k in buf:
            buf[k].copy_(d[k])
        want = once(d)
        for g, out in graphs:
            g.replay()
            torch.cuda.synchronize()
            for x, y in zip(out, want):
                assert torch.equal(x, y)


@pytest.mark.parametrize("V", [45, 3000])
def test_extreme_repetition(rx, V):
    """Repetitions near the ends of fp32: the quotient is the division's."""
    rho = torch.tensor([1e-45, 1e-39, 1e-30, 0.3, 7.0, 1e30, 1e38, 3e38], device="cuda")
    z = torch.randn(8, V, device="cuda") * torch.tensor([1e-44, 1e-38, 1e-9, 1, 1, 1e9, 1e38, 3e38],
                                                        device="cuda")[:, None]
    h = torch.arange(40, dtype=torch.int32, device="cuda").repeat(8, 1)
    got = rx.shape_logits(z, history=h, repetition=rho)
    want = z.clone()
    want[:, :40] = torch.where(z > 0, z / rho[:, None], z * rho[:, None])[:, :40]
    d, r = got.cpu().double().numpy(), want.cpu().double().numpy()
    assert (np.isfinite(d) == np.isfinite(r)).all()
    m = np.isfinite(r)
    # two roundings of a quotient at most, or of the smallest values
    assert (np.abs(d[m] - r[m]) <= 2 * ref.U * np.abs(r[m]) + 2.0 ** -149).all()


@pytest.mark.parametrize("R,V", [(96_000_000, 45), (135_000, 32003)])
def test_far_offsets(rx, R, V):
    """More than 2^32 logits: the first and the last rows give the bits of the
    same rows on their own, the gradient included."""
    z = torch.empty(R, V, dtype=torch.bfloat16, device="cuda")
    step = R // 8
    for lo in range(0, R, step):
        z[lo:lo + step].normal_()
    a, _ = inputs(8, V, 4, "bf16", 3, "table")
    c = {k: v.cuda() for k, v in a.items()}
    kw = dict(bias=c["bias"], history=c["history"][:1].expand(R, 4).contiguous(), repetition=1.25,
              frequency=0.25, mask=c["mask"], mask_rows=torch.arange(R, dtype=torch.int32, device="cuda") % 5)
    leaf = z.requires_grad_()
    out = rx.shape_logits(leaf, **kw)
    g, = torch.autograd.grad(out, leaf, out.detach().clamp(min=-1))
    for rows in (slice(0, 1000), slice(R - 1000, R)):
        few = dict(kw, history=kw["history"][rows].contiguous(), mask_rows=kw["mask_rows"][rows].contiguous())
        one = z.detach()[rows].clone().requires_grad_()
        want = rx.shape_logits(one, **few)
        assert torch.equal(out.detach()[rows], want.detach())
        gw, = torch.autograd.grad(want, one, want.detach().clamp(min=-1))
        assert torch.equal(g[rows], gw)
