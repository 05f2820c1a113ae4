"""The policy operators in a row, as a policy with memory uses them on a
collection's buffers: the previous action's embedding, the recurrence over
the rollout with its dones, and masked logits; forward and every gradient
against 64 bits, and acting step by step against the scan."""
import numpy as np
import pytest
import torch

import synthdata
from parity import gpu_available
from test_gpu_logits import bits_of

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X")]

N, L, D, A = 16, 60, 32, 45


@pytest.fixture(scope="module")
def rollout():
    """A collection: its actions and dones are the policy's inputs."""
    import rl_experience_collection_amd as rx
    inp = synthdata.ppo_inputs(dict(N=N, L=L, n_bars=2000, seed=3), bias_scale=0.1)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    col = rx.Collector(N, L, {k: [dev(w) for w in inp["weights"][k]] for k in ("actor", "critic", "curiosity")},
                       dev(inp["features"]), dev(inp["prices"]))
    out = col.collect(dev(inp["starts"]), seed=11)
    torch.cuda.synchronize()
    assert int(out["dones"].sum()) > 0
    return out


def parameters():
    g = torch.Generator().manual_seed(5)
    shape = dict(table=(A, D), wx=(D, D), wg=(D, D), wo=(A, D), bias=(A,))
    return {k: (torch.randn(s, generator=g) * s[-1] ** -0.5).cuda() for k, s in shape.items()}


def inputs(rollout):
    actions, dones = rollout["actions"], rollout["dones"]
    # the first step of the rollout and of every episode has no previous action
    prev = torch.full_like(actions, -1)
    prev[1:] = torch.where(dones[:-1] != 0, -1, actions[:-1])
    g = torch.Generator().manual_seed(6)
    table = torch.rand(7, A, generator=g).numpy() < 0.7
    table[:, 0] = True
    mask = bits_of(table).cuda()
    rows = torch.randint(0, 7, (L, N), generator=g, dtype=torch.int32).cuda()
    # the last 20 actions of each step's own episode
    window = torch.full((L, N, 20), -1, dtype=torch.int32, device="cuda")
    for t in range(L):
        if t:
            window[t, :, 1:] = window[t - 1, :, :-1]
            window[t, :, 0] = actions[t - 1]
            window[t][dones[t - 1] != 0] = -1
    h0 = torch.randn(N, D, generator=g).cuda()
    return prev.contiguous(), dones, window, torch.from_numpy(table).cuda(), mask, rows, h0


def run(rx, p, prev, dones, window, mask, rows, h0):
    e = rx.embed(p["table"], prev, scale=2.0)
    h, last = rx.recurrence(e @ p["wx"], e @ p["wg"] + 1.0, h0, dones)
    z = rx.shape_logits(h @ p["wo"].t(), bias=p["bias"], history=window, repetition=1.2, presence=0.3,
                        frequency=0.1, mask=mask, mask_rows=rows)
    return z, last


def plain(p, prev, dones, window, table, rows, h0):
    """The same in 64 bits on the CPU, from the definitions."""
    e = torch.where((prev >= 0)[..., None], p["table"][prev.clamp(min=0).long()] * 2.0, 0.0)
    x, gate = e @ p["wx"], e @ p["wg"] + 1.0
    state, hs = h0, []
    for t in range(L):
        if t:
            state = torch.where((dones[t - 1] != 0)[:, None], 0.0, state)
        a = torch.sigmoid(gate[t])
        state = a * state + (1 - a) * x[t]
        hs.append(state)
    z = torch.stack(hs) @ p["wo"].t()
    count = torch.stack([(window == v).sum(-1) for v in range(A)], -1)
    z = torch.where(count > 0, torch.where(z > 0, z / np.float32(1.2), z * np.float32(1.2)), z)
    z = z - (count > 0) * float(np.float32(0.3)) - count * float(np.float32(0.1)) + p["bias"]
    z = torch.where(table[rows.long()], z, -float("inf"))
    return z, torch.where((dones[L - 1] != 0)[:, None], 0.0, state)


def test_forward_and_every_gradient(rollout):
    import rl_experience_collection_amd as rx
    prev, dones, window, table, mask, rows, h0 = inputs(rollout)
    actions = rollout["actions"].long()
    p = {k: v.requires_grad_() for k, v in parameters().items()}
    h0 = h0.requires_grad_()
    # a policy-gradient loss on the actions that the mask allows
    ok = table[rows.long()].gather(2, actions[..., None])[..., 0]
    w = torch.where(ok, rollout["advantages"], 0.0)

    def loss(z, last, actions, w):
        lp = torch.log_softmax(z, -1).gather(2, actions[..., None])[..., 0]
        return (torch.where(w != 0, lp, 0.0) * w).sum() + (last * last).sum()

    z, last = run(rx, p, prev, dones, window, mask, rows, h0)
    leaves = list(p.values()) + [h0]
    got = torch.autograd.grad(loss(z, last, actions, w), leaves)

    q = {k: v.detach().cpu().double().requires_grad_() for k, v in p.items()}
    r0 = h0.detach().cpu().double().requires_grad_()
    c = lambda t: t.detach().cpu()
    rz, rlast = plain(q, c(prev), c(dones), c(window), c(table), c(rows), r0)
    want = torch.autograd.grad(loss(rz, rlast, c(actions), c(w).double()), list(q.values()) + [r0])
    zc = c(z).double()
    assert torch.equal(torch.isneginf(zc), torch.isneginf(rz))
    # Forward: three products of 32 terms (33 roundings each), the scan's 12
    # roundings over a memory of at most 60 steps, the logits' 5: below 2000
    # half steps of the largest magnitude in play, which |z| and the 32-term
    # sums keep under 20.
    fin = ~torch.isneginf(zc)
    assert (zc[fin] - rz[fin]).abs().max() < 2000 * 2.0 ** -24 * 20
    assert (c(last).double() - rlast).abs().max() < 2000 * 2.0 ** -24 * 20
    # Gradients are sums of at most L N = 960 such terms; relative to the
    # largest, the same count of roundings once forward and once back.
    for name, a, b in zip(list(p) + ["h0"], got, want):
        err = float((c(a).double() - b).abs().max() / b.abs().max())
        assert err < 2 * (2000 + 960) * 2.0 ** -24, (name, err)


def test_acting_step_by_step_follows_the_scan(rollout):
    import rl_experience_collection_amd as rx
    prev, dones, window, table, mask, rows, h0 = inputs(rollout)
    p = parameters()
    with torch.no_grad():
        z, last = run(rx, p, prev, dones, window, mask, rows, h0)
        state = h0.clone()
        for t in range(L):
            e = rx.embed(p["table"], prev[t], scale=2.0)
            h, _ = rx.recurrence_step(e @ p["wx"], e @ p["wg"] + 1.0, state,
                                      resets=dones[t - 1] if t else None, out_state=state)
            zt = rx.shape_logits(h @ p["wo"].t(), bias=p["bias"], history=window[t], repetition=1.2,
                                 presence=0.3, frequency=0.1, mask=mask, mask_rows=rows[t])
            assert torch.equal(torch.isneginf(zt), torch.isneginf(z[t]))
            fin = ~torch.isneginf(zt)
            # both are within the bound of the test above of the same values
            assert (zt[fin] - z[t][fin]).abs().max() < 2 * 2000 * 2.0 ** -24 * 20
        state[dones[L - 1] != 0] = 0
        assert (state - last).abs().max() < 2 * 2000 * 2.0 ** -24 * 20
