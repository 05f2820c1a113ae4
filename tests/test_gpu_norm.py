"""The norms around a block and dropout (include/block.h, norm_*, drop_*) on
the GPU against their 64-bit forms."""
import numpy as np
import pytest
import torch

import block_ref as ref
from parity import gpu_available
from test_gpu_scan import TYPES, f64, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X")]

LEAVES = ("residual", "branch", "weight", "branch_weight", "gate")


@pytest.fixture(scope="module")
def rx():
    import rl_experience_collection_amd as rx
    return rx


def inputs(R, D, name, gate, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    t = TYPES[name]
    i = dict(residual=2 * n(R, D), branch=n(R, D), gate={"none": None, "full": n(R, D), "channel": n(D)}[gate])
    i = {k: v if v is None or v.dim() == 1 else v.to(t) for k, v in i.items()}
    return dict(i, weight=1 + 0.2 * n(D), branch_weight=1 + 0.2 * n(D)), \
        dict(dstream=n(R, D).to(t), dnormed=n(R, D).to(t))


def check(rx, i, g, name, act="none", rs=1.0, bs=0.5, branch_norm=True, eps=1e-6, p=0.0, seed=3, offset=0, gpu=None):
    n = {k: f64(v) for k, v in dict(i, **g).items()}
    R, D = i["residual"].shape
    kept, scale = (None, 1.0)
    if p:
        kept, scale = ref.kept(R * D, p, seed, offset)
        kept = kept.reshape(R, D)
    f32 = lambda v: float(np.float32(v))
    r = ref.norm(*[n[k] for k in LEAVES], name, act=act, rs=f32(rs), bs=f32(bs), branch_norm=branch_norm, eps=f32(eps),
                 kept=kept, scale=scale, dstream=n["dstream"], dnormed=n["dnormed"])
    dev = dict({k: None if v is None else v.cuda() for k, v in dict(i, **g).items()}, **(gpu or {}))
    leaves = {k: dev[k].detach().requires_grad_() for k in LEAVES if dev[k] is not None}
    out = rx.residual_norm(**{k: leaves.get(k) for k in LEAVES}, activation=act, residual_scale=rs, branch_scale=bs,
                           branch_norm=branch_norm, eps=eps, dropout=p, seed=seed, offset=offset)
    within(out[0], r["stream"], r["estream"], "stream")
    within(out[1], r["normed"], r["enormed"], "normed")
    outs = [(o, dev[k]) for o, k in zip(out, ("dstream", "dnormed")) if dev[k] is not None]
    grads = torch.autograd.grad([o for o, _ in outs], list(leaves.values()), [d for _, d in outs])
    for k, got in zip(leaves, grads):
        within(got, r["d" + k], r["ed" + k], "d" + k)


SIZES = [(1, 1), (3, 3), (5, 8), (2, 9), (100, 45), (70, 64), (33, 128), (17, 129), (9, 512), (40, 513), (3, 2048), (5, 2049),
         (2, 4096), (3, 5001), (2, 8191), (1, 8192)]


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gate", ["none", "full", "channel"])
@pytest.mark.parametrize("R,D", SIZES)
def test_matches_the_formula(rx, R, D, gate, name):
    check(rx, *inputs(R, D, name, gate, R * 31 + D), name, act="sigmoid" if gate == "full" else "none")


@pytest.mark.parametrize("act", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("gate", ["full", "channel"])
def test_activations(rx, gate, act):
    check(rx, *inputs(20, 70, "f32", gate, 4), "f32", act=act, rs=0.7, bs=-1.3, eps=1e-5)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["none", "full", "channel"])
@pytest.mark.parametrize("R,D,p", [(7, 5, 0.5), (30, 64, 0.1), (9, 129, 0.3), (3, 2051, 0.25), (4, 300, 1.0)])
def test_dropout_inside(rx, R, D, p, gate, name):
    check(rx, *inputs(R, D, name, gate, 6), name, act="silu" if gate == "full" else "none", p=p, seed=-77, offset=9)


@pytest.mark.parametrize("D", [20, 600])
def test_options(rx, D):
    i, g = inputs(25, D, "bf16", "full", 7)
    check(rx, dict(i, branch_weight=None), g, "bf16", branch_norm=False)
    check(rx, dict(i, weight=None, branch_weight=None, gate=None), g, "bf16")
    check(rx, i, dict(g, dstream=None), "bf16")
    check(rx, i, dict(g, dnormed=None), "bf16")
    check(rx, dict(i, branch=None, branch_weight=None, gate=None), g, "bf16", rs=1.5)


def test_many_rows(rx):
    check(rx, *inputs(40000, 24, "f32", "channel", 8), "f32")


def test_shapes_and_strides(rx):
    i, g = inputs(24, 20, "bf16", "full", 9)
    wide = {k: torch.full((24, 31), 7.0, dtype=torch.bfloat16, device="cuda") for k in ("residual", "branch", "gate")}
    for lo, k in enumerate(wide):
        wide[k][:, lo + 1:lo + 21] = i[k].cuda()
        wide[k] = wide[k][:, lo + 1:lo + 21]
    check(rx, i, g, "bf16", act="sigmoid", gpu=wide)
    check(rx, i, dict(g, dnormed=g["dnormed"][:1].expand(24, 20)), "bf16", act="sigmoid",
          gpu=dict(dnormed=g["dnormed"][:1].cuda().expand(24, 20)))
    dev = {k: v.cuda() for k, v in i.items()}
    flat = rx.residual_norm(**dev)
    three = rx.residual_norm(**{k: v.view(4, 6, 20) if v.dim() == 2 else v for k, v in dev.items()})
    assert three[0].shape == (4, 6, 20)
    assert all(torch.equal(a, b.view(24, 20)) for a, b in zip(flat, three))
    # one row of fp32 values is a gate for all rows, whichever way it is read
    one = torch.randn(20, device="cuda")
    a = rx.residual_norm(dev["residual"][0].float(), dev["branch"][0].float(), gate=one)
    b = rx.residual_norm(dev["residual"][:1].float(), dev["branch"][:1].float(), gate=one[None])
    assert all(torch.equal(u, v[0]) for u, v in zip(a, b))


def test_dropped_places_hold_anything(rx):
    R, D = 6, 40
    i, g = inputs(R, D, "f32", "full", 10)
    kept, _ = ref.kept(R * D, 0.4, 5)
    off = torch.from_numpy(~kept.reshape(R, D))
    bad = dict(i, gate=torch.where(off, torch.tensor(float("nan")), i["gate"]))
    run = lambda v: rx.residual_norm(**{k: t.cuda() for k, t in v.items()}, dropout=0.4, seed=5)
    for a, b in zip(run(i), run(bad)):
        assert torch.equal(a, b)


def test_a_row_of_zeros(rx):
    z = torch.zeros(3, 30, device="cuda", requires_grad=True)
    out = rx.residual_norm(z, z)
    assert not out[0].any() and not out[1].any()
    g, = torch.autograd.grad(out, z, [torch.ones_like(z)] * 2)
    assert torch.isfinite(g).all()


@pytest.mark.parametrize("gate", ["none", "channel"])
def test_no_rows(rx, gate):
    z = lambda *s: torch.zeros(*s, device="cuda", requires_grad=True)
    leaves = [z(0, 6), z(0, 6), z(6), z(6)] + ([z(6)] if gate == "channel" else [])
    out = rx.residual_norm(leaves[0], leaves[1], leaves[2], branch_weight=leaves[3], gate=leaves[4] if len(leaves) > 4 else None)
    grads = torch.autograd.grad(out, leaves, [torch.ones_like(t) for t in out])
    assert all(a.shape == b.shape and not a.any() for a, b in zip(grads, leaves))


def test_norm_captured_and_replayed(rx):
    i, g = inputs(200, 128, "bf16", "full", 11)
    dev = {k: v.cuda() for k, v in dict(i, **g).items()}
    leaves = {k: dev[k].requires_grad_() for k in LEAVES}
    seed = torch.tensor([5], device="cuda")

    def run():
        out = rx.residual_norm(**leaves, activation="silu", dropout=0.3, seed=seed)
        return list(out) + list(torch.autograd.grad(out, list(leaves.values()), (dev["dstream"], dev["dnormed"])))

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for turn in range(3):
        seed += 1
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), turn


# ------------------------------------------------------------------- dropout
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("count,p", [(1, 0.5), (7, 0.3), (8, 0.1), (1000, 0.25), (4099, 0.9), (64, 0.0), (64, 1.0), (64, 5e-6)])
def test_dropout(rx, count, p, name):
    x = torch.randn(count, generator=torch.Generator().manual_seed(count)).to(TYPES[name])
    kept, scale = ref.kept(count, p, 1234567890123, 6)
    d = x.cuda().requires_grad_()
    y = rx.dropout(d, p, 1234567890123, offset=6)
    want = np.where(kept, f64(x) * scale, 0.0)
    # the scale rounded to fp32, its product: two roundings
    within(y, want, ref.fin(name, want, 2 * ref.U * np.abs(want)), "y")
    dy = torch.randn(count, generator=torch.Generator().manual_seed(1)).to(TYPES[name])
    got, = torch.autograd.grad(y, d, dy.cuda())
    want = np.where(kept, f64(dy) * scale, 0.0)
    within(got, want, ref.fin(name, want, 2 * ref.U * np.abs(want)), "dx")


def test_dropped_elements_are_zero_whatever_they_hold(rx):
    kept, _ = ref.kept(64, 0.5, 9)
    x = torch.full((64,), float("nan"), device="cuda")
    y = f64(rx.dropout(x, 0.5, 9))
    assert np.array_equal(np.isnan(y), kept) and not y[~kept].any()
    assert not rx.dropout(x, 1.0, 9).any()


def test_a_seed_on_the_device(rx):
    x = torch.randn(5, 77, device="cuda")
    seed = torch.tensor(-123, device="cuda")
    assert torch.equal(rx.dropout(x, 0.3, seed), rx.dropout(x, 0.3, -123))
    assert not torch.equal(rx.dropout(x, 0.3, -123), rx.dropout(x, 0.3, -123, offset=1))


def test_dropout_is_what_the_norm_drops(rx):
    r, b = torch.randn(2, 30, 33, device="cuda")
    a, _ = rx.residual_norm(torch.zeros_like(r), b, branch_norm=False, dropout=0.4, seed=8, offset=2)
    assert torch.equal(a, rx.dropout(b, 0.4, 8, offset=2))


def test_dropout_captured_and_replayed(rx):
    x = torch.randn(1001, device="cuda", requires_grad=True)
    seed = torch.tensor([1], device="cuda")
    dy = torch.randn(1001, device="cuda")

    def run():
        y = rx.dropout(x, 0.5, seed)
        return y, torch.autograd.grad(y, x, dy)[0]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    before = None
    for turn in range(3):
        seed += 1
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        assert before is None or not torch.equal(before, out[0])
        before = out[0].clone()


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("R,D", [(6, 40), (5, 3), (4, 600)])
def test_gradients_of_dropped_places_hold_anything(rx, R, D, act, name):
    """NaN and infinities of the gate, the branch (not normed) and the stream's
    gradient at dropped places: the gradients are those without them."""
    i, g = inputs(R, D, name, "full", 10)
    kept, _ = ref.kept(R * D, 0.4, 5)
    off = torch.from_numpy(~kept.reshape(R, D))
    nan, inf = torch.tensor(float("nan"), dtype=TYPES[name]), torch.tensor(-float("inf"), dtype=TYPES[name])
    i["branch_weight"] = None

    def run(i, g, branch_norm):
        dev = {k: v.cuda() for k, v in dict(i, **g).items() if v is not None}
        leaves = {k: dev[k].requires_grad_() for k in LEAVES if k in dev}
        out = rx.residual_norm(**leaves, activation=act, dropout=0.4, seed=5, branch_norm=branch_norm)
        return dict(zip(leaves, torch.autograd.grad(out, list(leaves.values()), (dev["dstream"], dev["dnormed"]))))

    for branch_norm in (True, False):
        clean = run(i, g, branch_norm)
        for bad in (nan, inf):
            got = run(dict(i, gate=torch.where(off, bad, i["gate"])), g, branch_norm)
            assert all(torch.equal(got[k], clean[k]) for k in clean)
            got = run(i, dict(g, dstream=torch.where(off, bad, g["dstream"])), branch_norm)
            assert all(torch.equal(got[k], clean[k]) for k in clean if k != "residual")
            if not branch_norm:
                got = run(dict(i, branch=torch.where(off, bad, i["branch"])), g, branch_norm)
                assert all(torch.equal(got[k], clean[k]) for k in clean)


@pytest.mark.parametrize("act", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("D", [40, 600])
def test_gradients_where_all_is_dropped(rx, D, act):
    """Weights and a channel gate that are no numbers meet no element."""
    i, g = inputs(5, D, "f32", "channel", 12)
    i["gate"][::3], i["gate"][1::3] = float("nan"), float("inf")
    i["branch_weight"][::2] = float("nan")
    dev = {k: v.cuda() for k, v in dict(i, **g).items()}
    leaves = {k: dev[k].requires_grad_() for k in LEAVES}
    out = rx.residual_norm(**leaves, activation=act, dropout=1.0, seed=5)
    got = dict(zip(LEAVES, torch.autograd.grad(out, list(leaves.values()), (dev["dstream"], dev["dnormed"]))))
    assert not got["branch"].any() and not got["branch_weight"].any() and not got["gate"].any()
    assert torch.isfinite(got["residual"]).all() and torch.isfinite(got["weight"]).all()


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_an_activation_without_a_gate_has_no_effect(rx, act):
    i, g = inputs(5, 40, "f32", "none", 13)
    dev = {k: v.cuda() for k, v in i.items() if v is not None}
    for a, b in zip(rx.residual_norm(**dev), rx.residual_norm(**dev, activation=act)):
        assert torch.equal(a, b)
