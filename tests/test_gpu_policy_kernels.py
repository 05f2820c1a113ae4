"""The policy operators' kernels that large passes use, each reached at a
small size: many tiles of many columns in lanes of one, two and four channels;
sums over pieces, groups and joins of whole numbers, which 32 bits hold
exactly in any order, so that a lost or doubled row shows; whole rows of
logits as tiles; the sorted gradient's row strides."""

import numpy as np
import pytest
import torch

import policy_ref as ref
import test_gpu_logits as lg
from parity import gpu_available
from test_gpu_recur import TYPES, check, inputs

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X")]


@pytest.fixture(scope="module")
def rx():
    import rl_experience_collection_amd as rx
    return rx


# ---------------------------------------------------------------- recurrence
# lanes of four channels (16 bits; a width that is no multiple of four), of two
# and of one, 8 waves and 16, each over several tiles
@pytest.mark.parametrize("sig", [False, True])
@pytest.mark.parametrize("L,N,D,name", [(200, 2048, 34, "bf16"), (200, 2048, 34, "f16"), (150, 2730, 30, "bf16"),
                                        (200, 600, 66, "bf16"), (500, 128, 128, "f32"), (300, 700, 66, "f32"),
                                        (300, 257, 65, "f32"), (500, 128, 128, "bf16")])
def test_walks_over_many_tiles(rx, L, N, D, name, sig):
    check(rx, inputs(L, N, D, name, sig, 0.01, L + N), name, sig)


@pytest.mark.parametrize("L,N,D,name", [(200, 2048, 34, "bf16"), (500, 128, 128, "f32"), (300, 700, 66, "f32")])
def test_walks_over_gates_without_maps(rx, L, N, D, name):
    """Linear gates whose product overflows over a row of zeros, in some tiles."""
    i = inputs(L, N, D, name, False, 0.01, 41)
    i["gate"] = torch.ones_like(i["gate"])
    for k in ("x", "dh"):
        i[k][:, ::3] = 0
    for k in ("h0", "dl"):
        i[k][::3] = 0
    for lo in (16, L - 40):
        i["gate"][lo:lo + 24, ::3] = 2e5
    h, _ = check(rx, i, name, False)
    assert (h[:, ::3] == 0).all()


@pytest.mark.parametrize("sig", [False, True])
@pytest.mark.parametrize("L,N,D,name", [(300, 2048, 34, "bf16"), (500, 128, 128, "f32"), (300, 700, 66, "f32")])
def test_walks_past_a_finished_episode(rx, L, N, D, name, sig):
    """A NaN and an infinity behind dones, tiles away from the end: every other
    element keeps its bits."""
    i = inputs(L, N, D, name, sig, 0.0, 42)
    i["dones"] = torch.zeros(L, N, dtype=torch.uint8)
    i["dones"][150, 3] = i["dones"][97, 70] = 1
    c = {k: v.cuda() for k, v in i.items()}
    form = "sigmoid" if sig else "linear"

    def run(x, dh):
        leaves = [x.clone().requires_grad_(), c["gate"].clone().requires_grad_(), c["h0"].clone().requires_grad_()]
        out = rx.recurrence(*leaves, c["dones"], form=form)
        return list(out) + list(torch.autograd.grad(out, leaves, (dh, c["dl"])))

    clean = run(c["x"], c["dh"])
    x, dh = c["x"].clone(), c["dh"].clone()
    x[70, 3, 5], x[20, 70, 1] = float("nan"), float("inf")
    dh[160, 3, 5] = float("nan")
    got = run(x, dh)
    assert torch.isnan(got[0][70:151, 3, 5]).all() and not torch.isfinite(got[0][20:98, 70, 1]).any()
    assert torch.isnan(got[2][151:161, 3, 5]).all()
    for t in (got, clean):
        t[0][70:151, 3, 5] = 0  # h
        t[0][20:98, 70, 1] = 0
        t[2][151:161, 3, 5] = 0  # dx
        t[3][70:161, 3, 5] = 0  # dgate
        t[3][20:98, 70, 1] = 0
    for a, b in zip(got, clean):
        assert torch.equal(a, b)


# ----------------------------------------------------------------- embedding
def whole(shape, seed, most=7):
    return torch.randint(-most, most + 1, shape, generator=torch.Generator().manual_seed(seed))


def exact_rows(dout, idx, V, scale):
    want = torch.zeros(V, dout.shape[1], dtype=torch.int64)
    known = (idx >= 0) & (idx < V)
    want.index_add_(0, idx[known].long(), dout[known].long())
    assert int(want.abs().max()) < 2 ** 24
    return (want * scale).float()  # (a scale of a power of two)


@pytest.mark.parametrize("spread", ["one", "skew", "even"])
@pytest.mark.parametrize("M,V,D", [(140001, 45, 5), (20000, 5000, 2), (64000, 45, 130), (5000, 1, 33), (70001, 9000, 40),
                                   (1024, 45, 128), (1000, 3, 700), (33, 7, 9)])
def test_every_row_counts_once(rx, M, V, D, spread):
    g = torch.Generator().manual_seed(M)
    idx = {"one": torch.full((M,), V // 2), "even": torch.randint(-1, V + 1, (M,), generator=g),
           "skew": (V ** torch.rand(M, generator=g)).long().clamp(1, V) - 1}[spread].int()
    dout = whole((M, D), M + 1)
    want = exact_rows(dout, idx, V, 2)
    for name in ("f32", "bf16"):
        w = torch.zeros(V, D, dtype=TYPES[name], device="cuda", requires_grad=True)
        g, = torch.autograd.grad(rx.embed(w, idx.cuda(), 2.0), w, dout.to(TYPES[name]).cuda())
        assert torch.equal(g.cpu(), want.to(TYPES[name]))


@pytest.mark.parametrize("index_bytes", [4, 8])
@pytest.mark.parametrize("dout_row", [0, 6, 11])
@pytest.mark.parametrize("M", [40, 3000, 20000])
def test_row_strides_of_the_gradient(rx, M, dout_row, index_bytes):
    V, D, R = 30, 6, 8
    lib, s = rx.load_library(), torch.cuda.current_stream().cuda_stream
    idx = torch.randint(-1, V + 1, (M,), generator=torch.Generator().manual_seed(M))
    idx = idx.int() if index_bytes == 4 else idx
    rows = whole((1 if dout_row == 0 else M, D), 5)
    src = torch.full((rows.shape[0], max(dout_row, D)), 7.0)
    src[:, :D] = rows
    want = exact_rows(rows.expand(M, D), idx, V, 2)
    dw = torch.full((V + 1, R), 7.0, device="cuda")
    cd, ci = src.cuda(), idx.cuda()
    size = lib.embed_workspace(0, V, D, M)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    assert lib.embed_backward(0, cd.data_ptr(), dout_row, ci.data_ptr(), index_bytes, M, V, D, 2.0, dw.data_ptr(), R,
                              ws.data_ptr(), size, s) == 0
    torch.cuda.synchronize()
    assert torch.equal(dw[:V, :D].cpu(), want) and (dw[V] == 7).all() and (dw[:, D:] == 7).all()


# -------------------------------------------------------------------- logits
@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("mask", ["none", "bytes", "bits"])
@pytest.mark.parametrize("R,V", [(9000, 1), (4097, 3), (20000, 45), (1200, 500), (300, 45), (700, 2049), (2600, 4097)])
def test_every_row_of_the_bias_gradient_counts_once(rx, R, V, mask, name):
    a, allowed = lg.inputs(R, V, 0, name, R + V, mask)
    dout = whole((R, V), R)
    ok = torch.ones(R, V, dtype=torch.bool) if allowed is None else torch.from_numpy(np.broadcast_to(allowed, (R, V)).copy())
    z, b = a["logits"].cuda().requires_grad_(), a["bias"].cuda().requires_grad_()
    out = rx.shape_logits(z, bias=b, mask=None if allowed is None else a["mask"].cuda())
    g, gb = torch.autograd.grad(out, (z, b), dout.to(TYPES[name]).cuda())
    want = torch.where(ok, dout, 0)
    assert torch.equal(g.cpu().long(), want)
    assert torch.equal(gb.cpu().long(), want.sum(0))


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("R", [20, 700])
@pytest.mark.parametrize("V", [45, 500, 2049])
def test_a_table_of_byte_masks(rx, R, V, name):
    a, _ = lg.inputs(R, V, 9, name, R + V)
    rng = np.random.default_rng(V)
    table = rng.random((6, V)) < 0.6
    table[5] = False
    rows = rng.integers(-2, 8, R).astype(np.int32)
    allowed = np.concatenate([table, np.ones((1, V), bool)])[np.where((rows >= 0) & (rows < 6), rows, 6)]
    lg.check(rx, dict(a, mask=torch.from_numpy(table), mask_rows=torch.from_numpy(rows)), allowed, name)


@pytest.mark.parametrize("kind", ["bits", "bytes", "table"])
@pytest.mark.parametrize("V", [45, 500])
def test_masked_places_of_whole_rows_do_not_matter(rx, V, kind):
    a, allowed = lg.inputs(700, V, 8, "f32", 9, kind)
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


@pytest.mark.parametrize("V", [45, 500])
def test_one_gradient_of_whole_rows_only(rx, V):
    a, _ = lg.inputs(700, V, 5, "f32", 11, "bytes")
    c = {k: v.cuda() for k, v in a.items()}
    dout = torch.randn(700, V, device="cuda")
    z, b = c["logits"].clone().requires_grad_(), c["bias"].clone().requires_grad_()
    both = torch.autograd.grad(rx.shape_logits(**dict(c, logits=z, bias=b)), (z, b), dout)
    gz, = torch.autograd.grad(rx.shape_logits(**dict(c, logits=z)), z, dout)
    gb, = torch.autograd.grad(rx.shape_logits(**dict(c, bias=b)), b, dout)
    assert torch.equal(gz, both[0]) and torch.equal(gb, both[1])


def test_extreme_repetition_of_whole_rows(rx):
    V, H = 45, 40
    rho = torch.tensor([1e-45, 1e-39, 1e-30, 0.3, 7.0, 1e30, 1e38, 3e38], device="cuda").repeat(100)
    size = torch.tensor([1e-44, 1e-38, 1e-9, 1, 1, 1e9, 1e38, 3e38], device="cuda").repeat(100)
    z = torch.randn(800, V, device="cuda") * size[:, None]
    h = torch.arange(H, dtype=torch.int32, device="cuda").repeat(800, 1)
    leaf = z.clone().requires_grad_()
    got = rx.shape_logits(leaf, history=h, repetition=rho)
    want = z.clone()
    want[:, :H] = torch.where(z > 0, z / rho[:, None], z * rho[:, None])[:, :H]
    g, = torch.autograd.grad(got, leaf, z)
    for d, r in ((got.detach(), want), (g, want)):  # dout = z: the gradient is scaled like the logits
        d, r = d.cpu().double().numpy(), r.cpu().double().numpy()
        assert (np.isfinite(d) == np.isfinite(r)).all()
        m = np.isfinite(r)
        # two roundings of a quotient at most, or of the smallest values
        assert (np.abs(d[m] - r[m]) <= 2 * ref.U * np.abs(r[m]) + 2.0 ** -149).all()


def test_unmasked_infinities_and_nan_pass_whole_rows(rx):
    z = torch.tensor([[float("inf"), -float("inf"), float("nan"), 1.0]], device="cuda").repeat(700, 1)
    h = torch.tensor([[0, 1, 2, 3, 3]], dtype=torch.int32, device="cuda").repeat(700, 1)
    got = rx.shape_logits(z, history=h, repetition=2.0, presence=0.5, frequency=0.25)
    assert (got[:, 0] == float("inf")).all() and (got[:, 1] == -float("inf")).all()
    assert torch.isnan(got[:, 2]).all() and (got[:, 3] == 0.5 - 0.5 - 0.5).all()
