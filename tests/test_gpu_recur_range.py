"""The recurrence where products of gates leave fp32's range and the states
do not: the answer is that of the steps one by one, whatever runs of steps
the kernels fold into one map, and however many columns there are."""
import numpy as np
import pytest
import torch

import policy_ref as ref
from parity import gpu_available
from test_gpu_recur import f64, inputs

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X")]

# few columns (chained where long) and enough to fill the chip
COLUMNS = [(5, 33), (5, 3300)]


@pytest.fixture(scope="module")
def rx():
    import rl_experience_collection_amd as rx
    return rx


def check(rx, i, name, sig):
    """The 64-bit form within policy_ref's bounds, wherever a 32-bit answer
    exists: a state or gradient of 2^127 and more, in the 64-bit form itself, is
    near or past the largest fp32 number, 2^128 - 2^104; it rounds to infinity
    there, and inf * a + b stays infinite (or becomes a NaN) until a done.
    These places, and those after them, are left out."""
    n = {k: f64(v) for k, v in i.items()}
    with np.errstate(over="ignore", invalid="ignore"):
        w = ref.recurrence_grad(n["x"], n["gate"], n["h0"], n["dones"], n["dh"], n["dl"], sig, name)
        d = w["dx"] / w["keep"] if sig else w["dx"]
    L, m, top = len(d), w["m"], 2.0 ** 127
    out_f, out_b = np.zeros_like(d, bool), np.zeros_like(d, bool)
    f = b = np.zeros(d.shape[1:], bool)
    for t in range(L):
        out_f[t] = f = (f & m[t]) | ~(np.abs(w["h"][t]) < top)
        s = L - 1 - t
        out_b[s] = ~(np.abs(d[s]) < top) | (b & m[s + 1])
        with np.errstate(invalid="ignore"):
            b = out_b[s] | ~(np.abs(w["a"][s] * d[s]) < top)
    before = np.concatenate([np.zeros_like(out_f[:1]), out_f[:-1]]) & m[:L]
    c = {k: None if v is None else v.cuda() for k, v in i.items()}
    leaves = [c[k].requires_grad_() for k in ("x", "gate", "h0")]
    h, last = rx.recurrence(*leaves, c["dones"], form="sigmoid" if sig else "linear")
    g = torch.autograd.grad((h, last), leaves, (c["dh"], c["dl"]))
    for got, k, e, out in ((h, "h", "eh", out_f), (last, "h_last", "elast", f & m[L]), (g[0], "dx", "edx", out_b),
                           (g[1], "dgate", "edg", out_b | before | ~(np.abs(w["dgate"]) < top)),
                           (g[2], "dh0", "edh0", b)):
        with np.errstate(invalid="ignore"):
            off = np.where(out, 0.0, np.abs(f64(got) - w[k]) - w[e])
        assert (off <= 0).all(), (k, float(np.nanmax(off)), np.argwhere(~(off <= 0))[0], out.mean())
        assert out.mean() <= 0.4  # (of plain's five rows only two have inputs or a gradient that can grow)
    return h.detach(), last.detach()


def plain(L, N, D, name, seed):
    """Gates of 1, no input but in row 2, no done but in row 3 (by the caller)."""
    i = inputs(L, N, D, name, False, 0.0, seed)
    i["gate"] = torch.ones_like(i["gate"])
    i["dones"] = torch.zeros(L, N, dtype=torch.uint8)
    for k in ("x", "dh"):
        i[k][:, [0, 1, 3, 4]] = 0
    i["h0"][1] = i["dl"][1] = 0
    return i


@pytest.mark.parametrize("N,D", COLUMNS)
@pytest.mark.parametrize("L,lo,n,gate", [(40, 0, 8, 1e-6), (40, 3, 8, 1e-6), (70, 20, 16, 1e-3), (600, 256, 128, 0.4),
                                         (1300, 300, 100, 0.3), (1300, 256, 256, 0.7)])
@pytest.mark.parametrize("growth_first", [False, True])
@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_a_product_that_underflows_and_grows_again(rx, L, lo, n, gate, growth_first, name, N, D):
    """n gates far below 1, then n of their inverse (or the inverse first, so
    that it is the gradient's product that underflows).  The states stay in
    fp32's range: 1e20 down and back up, or 1e-20 up and back down."""
    i = plain(L, N, D, name, 31)
    down, up = slice(lo, lo + n), slice(lo + n, lo + 2 * n)
    if growth_first:
        down, up = up, down
    i["gate"][down], i["gate"][up] = gate, 1 / gate
    i["dones"][lo + n, 3] = 1
    far = 1e-20 if growth_first else 1e20
    i["h0"][[0, 3, 4]] = torch.sign(i["h0"][[0, 3, 4]]) * far
    i["dl"][[0, 3, 4]] = torch.sign(i["dl"][[0, 3, 4]]) / far
    # an input that a tiny state meets in the middle
    i["x"][lo + n, 4] = far * 1e-30
    h, last = check(rx, i, name, False)
    assert (last[0].abs() > abs(far) * 1e-4).all() and (last[1] == 0).all()


def wandering(L, N, D, seed):
    """Scales that wander over 2^-100 .. 2^100, so that products of gates often
    leave fp32 either way and states do not, but behind the few gates that are
    past its range themselves."""
    rng = np.random.default_rng(seed)
    i = inputs(L, N, D, "f32", False, 0.01, 32)
    w = np.clip(np.cumsum(rng.uniform(-45, 45, (L + 1, N, D)), 0), -100, 100)
    kept = rng.random((L + 1, N, D)) < 0.4
    for t in range(1, L + 1):
        w[t] = np.where(kept[t], w[t - 1], w[t])
    w[L] = 0
    u = torch.from_numpy(rng.uniform(0.5, 1.0, (L, N, D)) * rng.choice([-1, 1], (L, N, D)))
    i["gate"] = (u * torch.from_numpy(2.0 ** (w[1:] - w[:-1]))).float()
    some = torch.from_numpy((rng.random((L, N, D)) < 0.3))
    i["x"] = (i["x"].double() * torch.from_numpy(2.0 ** w[1:]) * some).float()
    i["dh"] = (i["dh"].double() * torch.from_numpy(2.0 ** -w[1:]) * ~some).float()
    i["h0"] = (i["h0"].double() * torch.from_numpy(2.0 ** w[0])).float()
    return i


@pytest.mark.parametrize("N,D", COLUMNS)
@pytest.mark.parametrize("L", [60, 900])
def test_states_of_any_size(rx, L, N, D):
    check(rx, wandering(L, N, D, L + D), "f32", False)


def same(a, b):
    """Equal, a NaN like a NaN: some of wandering's gates are past fp32's range."""
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


def test_timing_does_not_matter(rx):
    """Chained tiles that hand on maps, faint maps or states as they come:
    repeats, two streams at once and replays of captured graphs between eager
    calls give the same bits."""
    data = [{k: v.cuda() for k, v in wandering(6000, 2, 70, s).items()} for s in (1, 2)]
    decay = {k: v.cuda() for k, v in inputs(6000, 2, 70, "f32", False, 0.001, 38).items()}
    decay["gate"] = torch.rand(6000, 2, 70, generator=torch.Generator().manual_seed(39)).cuda() * 0.6
    decay["x"][:, 1] = 0
    data.append(decay)

    def once(c):
        leaves = [c[k].detach().requires_grad_() for k in ("x", "gate", "h0")]
        out = rx.recurrence(*leaves, c["dones"], form="linear")
        return [t.detach() for t in out] + list(torch.autograd.grad(out, leaves, (c["dh"], c["dl"])))

    want = [once(c) for c in data]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in data], []
    for _ in range(6):
        for c, st in zip(data, streams):
            with torch.cuda.stream(st):
                got.append(once(c))
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        for a, b in zip(g, want[k % 3]):
            assert same(a, b)
    graphs = []
    for c, st in zip(data, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            out = once(c)
        graphs.append((g, out))
    for _ in range(4):
        eager = once(data[0])
        for (g, out), w in zip(graphs, want):
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, w):
                assert same(a, b)
        assert same(eager[0], want[0][0])


@pytest.mark.parametrize("name", ["f32", "f16"])
@pytest.mark.parametrize("with_input", [False, True])
def test_long_decays(rx, name, with_input):
    """Products of a chained tile's gates are below fp32's range throughout."""
    i = inputs(3000, 2, 70, name, False, 0.0, 33)
    i["gate"] = (torch.rand(3000, 2, 70, generator=torch.Generator().manual_seed(34)) * 0.2 + 0.3).to(i["x"].dtype)
    if not with_input:
        i["x"], i["dh"] = torch.zeros_like(i["x"]), torch.zeros_like(i["dh"])
    check(rx, i, name, False)


@pytest.mark.parametrize("N,D", COLUMNS)
@pytest.mark.parametrize("L", [40, 1300])
def test_gates_of_zero(rx, L, N, D):
    """A zero gate forgets, whatever the gates around it would underflow or
    overflow to; -0 is a zero like any other."""
    i = inputs(L, N, D, "f32", False, 0.0, 35)
    i["gate"][:, 0] = 1e-9
    i["gate"][:, 1] = 1e-9
    i["x"][:, [1, 2]] = 0
    i["gate"][4::16] = 0.0
    i["gate"][11::16] = -0.0
    i["gate"][L // 2 + 1:L // 2 + 3, 3] = 1e25
    i["gate"][L // 2 + 3, 3] = 0.0
    check(rx, i, "f32", False)


@pytest.mark.parametrize("N,D", COLUMNS)
@pytest.mark.parametrize("L,lo", [(40, 0), (40, 16), (1300, 256), (1300, 600)])
def test_a_state_that_cancels_before_a_growth(rx, L, lo, N, D):
    """The input at `lo` cancels the state, then gates grow: a map of these
    steps would hold an infinite sum, the states are zero."""
    i = plain(L, N, D, "f32", 36)
    i["x"][:] = 0
    i["dh"][:] = 0
    i["h0"][:] = -2.0 ** 110
    i["dl"][:] = 2.0 ** -60
    i["gate"][lo] = 2.0 ** -10
    i["x"][lo] = 2.0 ** 100
    i["gate"][lo + 1:lo + 3] = 2.0 ** 20
    h, last = check(rx, i, "f32", False)
    assert (h[lo:] == 0).all() and (last == 0).all()


@pytest.mark.parametrize("N,D", COLUMNS)
@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_an_infinite_state_stays_infinite(rx, N, D, name, bad):
    """Sigmoid gates shrink it and never make it a NaN, however many steps go
    by; a done ends it."""
    L = 1300
    i = inputs(L, N, D, name, True, 0.0, 37)
    i["gate"] = torch.full_like(i["gate"], -2.0)
    i["gate"][:, 1] = -30.0
    i["dones"] = torch.zeros(L, N, dtype=torch.uint8)
    i["dones"][900] = 1
    i["h0"][:2] = bad
    c = {k: v.cuda() for k, v in i.items()}
    h, last = rx.recurrence(c["x"], c["gate"], c["h0"], c["dones"])
    assert (h[:901, :2] == bad).all()
    assert torch.isfinite(h[901:]).all() and torch.isfinite(h[:, 2:]).all() and torch.isfinite(last).all()
    leaves = [c[k].clone().requires_grad_() for k in ("x", "gate", "h0")]
    c["dl"][:2] = bad
    c["dh"][:] = 0
    out = rx.recurrence(leaves[0], leaves[1], leaves[2])
    dx, _, dh0 = torch.autograd.grad(out, leaves, (c["dh"], c["dl"]))
    assert (dx[:, :2] == bad).all() and (dh0[:2] == bad).all()
    assert torch.isfinite(dx[:, 2:]).all()
