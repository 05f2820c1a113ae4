"""The selective state space scan (include/block.h, scan_*) on the GPU against
its 64-bit form, element by element within the bound that block_ref derives."""
import numpy as np
import pytest
import torch

import block_ref as ref
from parity import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X")]

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
STEPWISE = ("x", "delta", "b", "c", "gate")
LEAVES = ("x", "delta", "rate", "b", "c", "skip", "gate", "delta_bias", "state")


@pytest.fixture(scope="module")
def rx():
    import rl_experience_collection_amd as rx
    return rx


def inputs(L, N, D, S, G, name, p_done, seed, gate=True, bare=False, decay=1.0):
    """bare: without skip, bias, state and gate."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    bc = (L, N, S) if G == 0 else (L, N, G, S)
    i = dict(x=n(L, N, D), delta=n(L, N, D) - 1, b=n(*bc), c=n(*bc), gate=n(L, N, D) if gate and not bare else None)
    i = {k: None if v is None else v.to(TYPES[name]) for k, v in i.items()}
    i.update(rate=-torch.exp(n(D, S)) * decay, skip=None if bare else n(D), delta_bias=None if bare else 0.3 * n(D),
             state=None if bare else n(N, D, S),
             dones=(torch.rand(L, N, generator=g) < p_done).to(torch.uint8) if p_done else None)
    return i, dict(dy=n(L, N, D).to(TYPES[name]), dnew=n(N, D, S))


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def within(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = np.abs(got - want) - bound
    assert (off <= 0).all(), (what, float(np.nanmax(off)), np.unravel_index(np.nanargmax(off), off.shape),
                              int((~(off <= 0)).sum()), off.size)


def wanted(i, g, name, soft=True):
    n = {k: f64(v) for k, v in dict(i, **g).items()}
    if n["b"].ndim == 3:
        n["b"], n["c"] = n["b"][:, :, None], n["c"][:, :, None]
    r = ref.scan(n["x"], n["delta"], n["rate"], n["b"], n["c"], n["skip"], n["gate"], n["delta_bias"], n["state"],
                 n["dones"], soft, name, n["dy"], n["dnew"])
    if i["b"].dim() == 3:
        for k in ("db", "edb", "dc", "edc"):
            r[k] = r[k][:, :, 0]
    return r


def check(rx, i, g, name, soft=True, gpu=None, train=True, only=None):
    """gpu: device tensors to pass instead of copies (other strides)."""
    r = wanted(i, g, name, soft)
    dev = dict({k: None if v is None else v.cuda() for k, v in dict(i, **g).items()}, **(gpu or {}))
    leaves = {k: dev[k].detach().requires_grad_(train) for k in LEAVES if dev[k] is not None}
    y, new = rx.selective_scan(**{k: leaves.get(k) for k in LEAVES}, dones=dev["dones"], softplus=soft)
    within(y, r["y"], r["ey"], "y")
    within(new, r["new_state"], r["enew_state"], "new_state")
    if train:
        grads = torch.autograd.grad((y, new), list(leaves.values()), (dev["dy"], dev["dnew"]))
        for k, got in zip(leaves, grads):
            within(got, r["d" + k], r["ed" + k], "d" + k)
    return y, new


# (L, N, D, S, G); G 0: b and c without a groups' dimension
SIZES = [(1, 1, 1, 1, 0), (2, 3, 5, 16, 0), (7, 1, 64, 16, 0), (8, 2, 65, 16, 1), (9, 4, 6, 3, 2), (17, 2, 130, 7, 2),
         (16, 3, 33, 17, 3), (25, 1, 96, 32, 0), (11, 2, 40, 33, 0), (30, 2, 20, 64, 1), (23, 1, 70, 48, 0)]


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("L,N,D,S,G", SIZES)
def test_matches_the_formula(rx, L, N, D, S, G, name):
    check(rx, *inputs(L, N, D, S, G, name, 0.1, L * 31 + D), name)


# long enough to be cut into chunks
CHUNKED = [(33, 1, 64, 16, 0), (100, 2, 65, 16, 0), (257, 3, 20, 16, 2), (500, 2, 130, 5, 0), (131, 1, 9, 40, 0),
           (1025, 1, 3, 16, 0)]


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("p_done", [0.0, 0.02])
@pytest.mark.parametrize("L,N,D,S,G", CHUNKED)
def test_chunks(rx, L, N, D, S, G, p_done, name):
    check(rx, *inputs(L, N, D, S, G, name, p_done, L + D, decay=0.1), name)


# so many chunks that their summaries are joined by a kernel of their own
@pytest.mark.parametrize("p_done", [0.0, 0.004])
@pytest.mark.parametrize("L,N,D,S,G", [(545, 1, 64, 16, 0), (2049, 1, 70, 16, 2), (1500, 2, 7, 37, 0)])
def test_more_chunks(rx, L, N, D, S, G, p_done):
    check(rx, *inputs(L, N, D, S, G, "f32", p_done, L + D, decay=0.02), "f32")


@pytest.mark.parametrize("name", ["f32", "f16"])
def test_many_columns_are_not_cut(rx, name):
    check(rx, *inputs(40, 600, 6, 16, 0, name, 0.05, 3), name)


@pytest.mark.parametrize("L", [12, 300])
@pytest.mark.parametrize("soft", [True, False])
def test_without_the_options(rx, L, soft):
    i, g = inputs(L, 2, 10, 16, 0, "f32", 0.0, L, bare=True)
    if not soft:
        i["delta"] = i["delta"].abs() * 0.2
    check(rx, i, g, "f32", soft=soft)


@pytest.mark.parametrize("L", [20, 150])
def test_every_step_done_and_no_step_done(rx, L):
    for p in (1.0, 0.0):
        i, g = inputs(L, 3, 7, 16, 0, "f32", p, 5)
        check(rx, i, g, "f32")


@pytest.mark.parametrize("L", [21, 150])
def test_what_a_finished_episode_holds_stays_there(rx, L):
    """NaN and infinities before a done: the next episode's values and
    gradients are those without them."""
    i, g = inputs(L, 2, 6, 16, 0, "f32", 0.0, 6)
    cut = L // 2 + 1
    i["dones"] = torch.zeros(L, 2, dtype=torch.uint8)
    i["dones"][cut - 1] = 1
    clean = {k: v.clone() if v is not None else None for k, v in i.items()}
    i["x"][cut - 3, 0, 2], i["state"][1, 3, 4], i["b"][1, 1, 5] = float("nan"), float("inf"), float("inf")
    dev = {k: v.cuda() for k, v in dict(i, **g).items()}
    leaves = {k: dev[k].requires_grad_() for k in LEAVES}
    y, new = rx.selective_scan(**leaves, dones=dev["dones"])
    grads = dict(zip(LEAVES, torch.autograd.grad((y, new), list(leaves.values()), (dev["dy"], dev["dnew"]))))
    r = wanted(clean, g, "f32")
    within(y[cut:], r["y"][cut:], r["ey"][cut:], "y")
    within(new, r["new_state"], r["enew_state"], "new_state")
    for k in STEPWISE:
        within(grads[k][cut:], r["d" + k][cut:], r["ed" + k][cut:], "d" + k)


def test_a_gradient_that_is_no_number_stays_in_its_episode(rx):
    L = 150
    i, g = inputs(L, 2, 6, 16, 0, "f32", 0.0, 8)
    i["dones"] = torch.zeros(L, 2, dtype=torch.uint8)
    i["dones"][70] = 1
    r = wanted(i, g, "f32")
    g = {k: v.clone() for k, v in g.items()}
    g["dy"][100, 0, 1] = float("nan")
    dev = {k: v.cuda() for k, v in dict(i, **g).items()}
    leaves = {k: dev[k].requires_grad_() for k in LEAVES}
    y, new = rx.selective_scan(**leaves, dones=dev["dones"])
    grads = dict(zip(LEAVES, torch.autograd.grad((y, new), list(leaves.values()), (dev["dy"], dev["dnew"]))))
    for k in STEPWISE:
        within(grads[k][:71], r["d" + k][:71], r["ed" + k][:71], "d" + k)
    within(grads["state"], r["dstate"], r["edstate"], "dstate")


@pytest.mark.parametrize("L", [19, 130])
@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_strides(rx, L, name):
    """Batch-first, slices of wider rows at odd offsets, one row for all:
    the same results."""
    N, D, S = 3, 12, 16
    i, g = inputs(L, N, D, S, 2, name, 0.05, 9)
    bf = lambda t: t.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    check(rx, i, g, name, gpu={k: bf(i[k]) for k in STEPWISE})

    def sliced(t, lo):
        wide = torch.full(t.shape[:-1] + (t.shape[-1] + 9,), 7.0, dtype=t.dtype, device="cuda")
        wide[..., lo:lo + t.shape[-1]] = t.cuda()
        return wide[..., lo:lo + t.shape[-1]]

    check(rx, i, g, name, gpu={k: sliced(i[k], o) for k, o in zip(STEPWISE, (4, 3, 1, 5, 2))} | dict(dy=sliced(g["dy"], 1)))
    # one projection's output holds delta's row and b and c's groups
    one = torch.cat([i["b"].flatten(2), i["c"].flatten(2)], -1).cuda()
    check(rx, i, g, name, gpu=dict(b=one[..., :2 * S].unflatten(2, (2, S)), c=one[..., 2 * S:].unflatten(2, (2, S))))
    rep = dict(i, x=i["x"][:, :1].expand(L, N, D))
    check(rx, rep, g, name, gpu=dict(x=i["x"][:, :1].cuda().expand(L, N, D)))


def test_gradients_of_broadcast_inputs_are_sums(rx):
    i, g = inputs(30, 4, 8, 16, 0, "f32", 0.05, 11)
    r = wanted(dict(i, b=i["b"][:, :1].expand(30, 4, 16)), g, "f32")
    one = i["b"][:, :1].cuda().requires_grad_()
    dev = {k: v.cuda() for k, v in dict(i, **g).items()}
    y, new = rx.selective_scan(**{k: one.expand(30, 4, 16) if k == "b" else dev[k] for k in LEAVES}, dones=dev["dones"])
    got, = torch.autograd.grad((y, new), one, (dev["dy"], dev["dnew"]))
    # torch adds four values: three more roundings of their magnitudes
    within(got, r["db"].sum(1, keepdims=True), r["edb"].sum(1, keepdims=True) +
           3 * 2.0 ** -24 * np.abs(r["db"]).sum(1, keepdims=True), "db")


def test_gradient_of_one_output_alone(rx):
    i, g = inputs(90, 2, 5, 16, 0, "f32", 0.05, 12)
    dev = {k: v.cuda() for k, v in dict(i, **g).items()}
    leaves = {k: dev[k].requires_grad_() for k in LEAVES}
    for which in ("dy", "dnew"):
        r = wanted(i, {k: v if k == which else torch.zeros_like(v) for k, v in g.items()}, "f32")
        out = rx.selective_scan(**leaves, dones=dev["dones"])["dy dnew".split().index(which)]
        for k, got in zip(LEAVES, torch.autograd.grad(out, list(leaves.values()), dev[which])):
            within(got, r["d" + k], r["ed" + k], "d" + k)


def test_a_rollout_cut_in_two(rx):
    i, g = inputs(77, 3, 9, 16, 0, "f32", 0.1, 13)
    r = wanted(i, g, "f32")
    dev = {k: v.cuda() for k, v in i.items()}
    state, ys = dev["state"], []
    for a, b in ((0, 30), (30, 30), (30, 77)):
        part = {k: dev[k][a:b] if k in STEPWISE else dev[k] for k in LEAVES}
        y, state = rx.selective_scan(**dict(part, state=state), dones=dev["dones"][a:b])
        ys.append(y)
    within(torch.cat(ys), r["y"], 2 * r["ey"], "y")
    within(state, r["new_state"], 2 * r["enew_state"], "new_state")


@pytest.mark.parametrize("L,N,D", [(0, 3, 4), (5, 0, 4), (5, 3, 0)])
def test_empty(rx, L, N, D):
    z = lambda *s: torch.zeros(*s, device="cuda", requires_grad=True)
    leaves = dict(x=z(L, N, D), delta=z(L, N, D), rate=z(D, 16), b=z(L, N, 16), c=z(L, N, 16), skip=z(D), delta_bias=z(D),
                  state=torch.ones(N, D, 16, device="cuda", requires_grad=True))
    y, new = rx.selective_scan(**leaves)
    assert y.shape == (L, N, D) and torch.equal(new, torch.ones(N, D, 16, device="cuda") if L == 0 else new)
    grads = dict(zip(leaves, torch.autograd.grad((y, new), list(leaves.values()), (y.detach(), torch.ones_like(new)))))
    for k in ("rate", "skip", "delta_bias"):
        assert not grads[k].any()
    if L == 0:
        assert torch.equal(grads["state"], torch.ones_like(new))


# -------------------------------------------------------------- single steps
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,D,S,G", [(1, 1, 1, 0), (3, 5, 16, 0), (128, 64, 16, 0), (7, 12, 3, 2), (5, 33, 64, 1), (2, 9, 33, 3)])
def test_step(rx, N, D, S, G, name):
    i, g = inputs(1, N, D, S, G, name, 0.0, N + D)
    resets = (torch.rand(N, generator=torch.Generator().manual_seed(N)) < 0.3).to(torch.uint8)
    i["state"][resets != 0] = float("nan")  # what a reset row holds does not matter
    clean = dict(i, state=torch.where(resets[:, None, None] != 0, torch.zeros(()), i["state"]))
    r = wanted(clean, g, name)
    dev = {k: None if v is None else v.cuda() for k, v in i.items()}
    args = {k: dev[k][0] if k in STEPWISE else dev[k] for k in LEAVES}
    y, new = rx.selective_scan_step(**args, resets=resets.cuda())
    within(y, r["y"][0], r["ey"][0], "y")
    within(new, r["new_state"], r["enew_state"], "new_state")
    y2, same = rx.selective_scan_step(**args, resets=resets.cuda() != 0, out_state=args["state"])
    assert same.data_ptr() == args["state"].data_ptr()
    assert torch.equal(y2, y) and torch.equal(same, new)


def test_steps_follow_the_scan(rx):
    i, g = inputs(40, 5, 7, 16, 0, "f32", 0.1, 20)
    r = wanted(i, g, "f32")
    dev = {k: v.cuda() for k, v in i.items()}
    state = dev["state"].clone()
    for t in range(40):
        args = {k: dev[k][t] if k in STEPWISE else dev[k] for k in LEAVES}
        y, _ = rx.selective_scan_step(**dict(args, state=state), resets=dev["dones"][t - 1] if t else None, out_state=state)
        within(y, r["y"][t], r["ey"][t], t)


# ------------------------------------------------- streams, graphs, the rest
def test_another_stream_and_repeatable(rx):
    i, g = inputs(200, 4, 70, 16, 0, "bf16", 0.02, 21)
    dev = {k: v.cuda() for k, v in dict(i, **g).items()}
    leaves = {k: dev[k].requires_grad_() for k in LEAVES}

    def run():
        y, new = rx.selective_scan(**leaves, dones=dev["dones"])
        return [y.detach(), new.detach()] + list(torch.autograd.grad((y, new), list(leaves.values()), (dev["dy"], dev["dnew"])))

    first = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = run()
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(first, other):
        assert torch.equal(a, b)


@pytest.mark.parametrize("L", [40, 400])
def test_captured_and_replayed(rx, L):
    i, g = inputs(L, 2, 12, 16, 0, "f32", 0.05, 22)
    dev = {k: v.cuda() for k, v in dict(i, **g).items()}
    leaves = {k: dev[k].requires_grad_() for k in LEAVES}

    def run():
        y, new = rx.selective_scan(**leaves, dones=dev["dones"])
        return [y, new] + list(torch.autograd.grad((y, new), list(leaves.values()), (dev["dy"], dev["dnew"])))

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for turn in range(3):
        with torch.no_grad():
            dev["x"].copy_(torch.randn(L, 2, 12, generator=torch.Generator().manual_seed(turn)))
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), turn


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("L,N,D,S,G", [(30, 2, 5, 16, 0), (30, 2, 65, 16, 1), (30, 2, 10, 20, 2), (300, 2, 5, 16, 0),
                                       (300, 1, 65, 16, 1), (300, 2, 15, 40, 3), (1100, 1, 6, 16, 0)])
def test_channels_past_a_group_add_nothing(rx, L, N, D, S, G, name):
    """Step sizes are positive, the bias alone is not: a lane without a channel
    that took the bias for its step size would grow by exp(4) to exp(8) a step
    from the state that it was given."""
    i, g = inputs(L, N, D, S, G, name, 0.0, L + D)
    u = torch.Generator().manual_seed(D)
    i["delta"] = (0.59 + 0.02 * torch.rand(L, N, D, generator=u)).to(TYPES[name])
    i["delta_bias"] = torch.full((D,), -0.5)
    i["rate"] = -8 - 8 * torch.rand(D, S, generator=u)
    check(rx, i, g, name, soft=False)


@pytest.mark.parametrize("L,N,D,S", [(1, 4097, 3, 2), (2, 300001, 1, 1), (1, 1 << 20, 1, 1)])
def test_sums_over_many_rows_have_short_chains(rx, L, N, D, S):
    """Equal summands, whose roundings go one way: the parameters' gradients
    stay within the bound, which has no term that grows with the rows."""
    i, g = inputs(L, N, D, S, 0, "f32", 0.0, N)
    for k, v in dict(x=1.1, delta=-0.7, b=0.9, c=0.7, gate=0.3, skip=1.3, delta_bias=0.1, state=1.1, rate=-0.7).items():
        i[k].fill_(v)
    g["dy"].fill_(1.1), g["dnew"].fill_(0.3)
    check(rx, i, g, "f32")
