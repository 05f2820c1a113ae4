"""The short causal convolution (include/block.h, conv_*) on the GPU against
its 64-bit form, element by element within the bound that block_ref derives."""
import numpy as np
import pytest
import torch

import block_ref as ref
from parity import gpu_available
from test_gpu_scan import TYPES, f64, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X")]

LEAVES = ("x", "weight", "bias", "state")


@pytest.fixture(scope="module")
def rx():
    import rl_experience_collection_amd as rx
    return rx


def inputs(L, N, D, W, name, p_done, seed, bare=False):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    t = TYPES[name]
    return dict(x=n(L, N, D).to(t), weight=n(D, W), bias=None if bare else n(D),
                state=None if bare else n(N, W - 1, D).to(t),
                dones=(torch.rand(L, N, generator=g) < p_done).to(torch.uint8) if p_done else None), \
        dict(dy=n(L, N, D).to(t), dnew=n(N, W - 1, D).to(t))


def wanted(i, g, silu, name):
    n = {k: f64(v) for k, v in dict(i, **g).items()}
    return ref.conv(n["x"], n["weight"], n["bias"], n["state"], n["dones"], silu, name, n["dy"], n["dnew"])


def check(rx, i, g, name, silu=True, gpu=None):
    r = wanted(i, g, silu, name)
    dev = dict({k: None if v is None else v.cuda() for k, v in dict(i, **g).items()}, **(gpu or {}))
    leaves = {k: dev[k].detach().requires_grad_() for k in LEAVES if dev[k] is not None}
    y, new = rx.causal_conv(**{k: leaves.get(k) for k in LEAVES}, dones=dev["dones"],
                            activation="silu" if silu else "none")
    within(y, r["y"], r["ey"], "y")
    assert np.array_equal(f64(new), r["new_state"])
    grads = torch.autograd.grad((y, new), list(leaves.values()), (dev["dy"], dev["dnew"]))
    for k, got in zip(leaves, grads):
        within(got, r["d" + k], r["ed" + k], "d" + k)


SIZES = [(1, 1, 1, 4), (2, 3, 5, 4), (3, 2, 8, 4), (7, 1, 64, 3), (33, 2, 65, 2), (20, 4, 6, 1), (40, 3, 17, 8),
         (5, 2, 33, 7), (130, 5, 7, 5), (513, 1, 130, 4), (300, 2, 40, 6), (16, 2, 2100, 4), (64, 300, 9, 3)]


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("L,N,D,W", SIZES)
def test_matches_the_formula(rx, L, N, D, W, name):
    check(rx, *inputs(L, N, D, W, name, 0.1, L * 31 + D), name)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("p_done", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("L,W", [(1, 4), (2, 8), (3, 4), (70, 4), (70, 8)])
def test_dones(rx, L, W, p_done, name):
    i, g = inputs(L, 3, 12, W, name, p_done, 5)
    check(rx, i, g, name)
    check(rx, i, g, name, silu=False)


@pytest.mark.parametrize("silu", [False, True])
def test_without_bias_and_state(rx, silu):
    check(rx, *inputs(50, 3, 20, 4, "bf16", 0.05, 6, bare=True), "bf16", silu=silu)


def test_what_a_finished_episode_holds_stays_there(rx):
    i, g = inputs(60, 2, 10, 4, "f32", 0.0, 7)
    i["dones"] = torch.zeros(60, 2, dtype=torch.uint8)
    i["dones"][29] = 1
    r = wanted(i, g, True, "f32")
    bad = dict(i, x=i["x"].clone())
    bad["x"][28, 0, 3], bad["x"][29, 1, 4] = float("nan"), float("inf")
    bg = dict(g, dy=g["dy"].clone())
    bg["dy"][31, 1, 5] = float("nan")
    dev = {k: v.cuda() for k, v in dict(bad, **bg).items()}
    leaves = {k: dev[k].requires_grad_() for k in LEAVES}
    y, new = rx.causal_conv(**leaves, dones=dev["dones"])
    within(y[30:], r["y"][30:], r["ey"][30:], "y")
    dx = torch.autograd.grad((y, new), leaves["x"], (dev["dy"], dev["dnew"]))[0]
    # (x of step 28 is in p of the steps 28 and 29, whose gradients reach back to step 25)
    within(dx[:25], r["dx"][:25], r["edx"][:25], "dx before")
    clean = np.ones((30, 2, 10), bool)
    clean[25:, 0, 3] = clean[25:, 1, 4] = False
    got = np.where(clean, f64(dx)[:30], r["dx"][:30])
    assert (np.abs(got - r["dx"][:30]) <= r["edx"][:30]).all()


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_strides(rx, name):
    L, N, D = 45, 3, 12
    i, g = inputs(L, N, D, 4, name, 0.05, 9)
    bf = lambda t: t.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    check(rx, i, g, name, gpu=dict(x=bf(i["x"])))

    def sliced(t, lo):
        wide = torch.full((L, N, 19), 7.0, dtype=t.dtype, device="cuda")
        wide[:, :, lo:lo + D] = t.cuda()
        return wide[:, :, lo:lo + D]

    check(rx, i, g, name, gpu=dict(x=sliced(i["x"], 3), dy=sliced(g["dy"], 1)))
    check(rx, dict(i, x=i["x"][:, :1].expand(L, N, D)), g, name, gpu=dict(x=i["x"][:, :1].cuda().expand(L, N, D)))
    check(rx, i, dict(g, dy=g["dy"][:1, :1].expand(L, N, D)), name, gpu=dict(dy=g["dy"][:1, :1].cuda().expand(L, N, D)))


def test_a_rollout_cut_in_two(rx):
    i, g = inputs(50, 3, 9, 4, "bf16", 0.1, 13)
    dev = {k: v.cuda() for k, v in i.items()}
    whole, last = rx.causal_conv(**{k: dev[k] for k in LEAVES}, dones=dev["dones"])
    state, ys = dev["state"], []
    for a, b in ((0, 2), (2, 2), (2, 31), (31, 50)):
        y, state = rx.causal_conv(dev["x"][a:b], dev["weight"], dev["bias"], state, dones=dev["dones"][a:b])
        ys.append(y)
    # the taps are added in one order wherever a chunk begins
    assert torch.equal(torch.cat(ys), whole) and torch.equal(state, last)


@pytest.mark.parametrize("L,N,D", [(0, 3, 4), (5, 0, 4), (5, 3, 0)])
def test_empty(rx, L, N, D):
    z = lambda *s: torch.zeros(*s, device="cuda", requires_grad=True)
    leaves = [z(L, N, D), z(D, 4), z(D), torch.ones(N, 3, D, device="cuda", requires_grad=True)]
    y, new = rx.causal_conv(*leaves)
    assert y.shape == (L, N, D)
    dx, dw, db, ds = torch.autograd.grad((y, new), leaves, (y.detach(), torch.ones_like(new)))
    assert not dw.any() and not db.any()
    if L == 0:
        assert torch.equal(new, leaves[3].detach()) and torch.equal(ds, torch.ones_like(new))


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,D,W", [(1, 1, 4), (3, 5, 4), (128, 64, 4), (7, 12, 1), (5, 33, 8), (2, 9, 2), (9, 6, 3)])
def test_step(rx, N, D, W, name):
    i, g = inputs(1, N, D, W, name, 0.0, N + D)
    resets = (torch.rand(N, generator=torch.Generator().manual_seed(N)) < 0.3).to(torch.uint8)
    i["state"][resets != 0] = float("nan")
    zero = torch.zeros((), dtype=i["state"].dtype)
    r = wanted(dict(i, state=torch.where(resets[:, None, None] != 0, zero, i["state"])), g, True, name)
    dev = {k: None if v is None else v.cuda() for k, v in i.items()}
    args = dict(x=dev["x"][0], weight=dev["weight"], bias=dev["bias"], state=dev["state"], resets=resets.cuda())
    y, new = rx.causal_conv_step(**args)
    within(y, r["y"][0], r["ey"][0], "y")
    assert np.array_equal(f64(new), r["new_state"])
    y2, same = rx.causal_conv_step(**args, out_state=args["state"])
    assert same.data_ptr() == args["state"].data_ptr()
    assert torch.equal(y2, y) and torch.equal(same, new)


def test_captured_and_replayed(rx):
    i, g = inputs(80, 4, 24, 4, "bf16", 0.05, 22)
    dev = {k: v.cuda() for k, v in dict(i, **g).items()}
    leaves = {k: dev[k].requires_grad_() for k in LEAVES}

    def run():
        y, new = rx.causal_conv(**leaves, dones=dev["dones"])
        return [y, new] + list(torch.autograd.grad((y, new), list(leaves.values()), (dev["dy"], dev["dnew"])))

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for turn in range(3):
        with torch.no_grad():
            dev["x"].copy_(torch.randn(80, 4, 24, generator=torch.Generator().manual_seed(turn)))
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), turn
