"""The operators of a residual block in a row, as a policy's trunk with a
selective memory uses them on a collection's buffers: embedding of the previous
action, norm, convolution, scan, gate, dropout and residual, logits; forward and
every gradient against 64 bits, and acting step by step against the rollout."""
import numpy as np
import pytest
import torch

import block_ref as ref
from parity import gpu_available
from test_gpu_policy_path import rollout  # noqa: F401  (a collection)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X")]

N, L, D, S, W, A = 16, 60, 32, 16, 4, 45
BLOCKS = 2
DROP, SEED = 0.2, 77


def parameters():
    g = torch.Generator().manual_seed(15)
    n = lambda *s: torch.randn(*s, generator=g)
    p = dict(table=n(A, D), norm=1 + 0.1 * n(D), out=n(A, D) * D ** -0.5)
    for i in range(BLOCKS):
        p.update({f"inp{i}": n(D, D) * D ** -0.5, f"gatew{i}": n(D, D) * D ** -0.5, f"conv{i}": n(D, W) * W ** -0.5,
                  f"convb{i}": 0.1 * n(D), f"proj{i}": n(D, D + 2 * S) * D ** -0.5, f"rate{i}": -torch.exp(0.5 * n(D, S)),
                  f"skip{i}": 1 + 0.1 * n(D), f"bias{i}": 0.3 * n(D) - 1, f"post{i}": 1 + 0.1 * n(D),
                  f"scale{i}": 0.5 + 0.1 * n(D), f"pre{i}": 1 + 0.1 * n(D)})
    state = [(n(N, W - 1, D), n(N, D, S)) for _ in range(BLOCKS)]
    return {k: v.cuda() for k, v in p.items()}, [tuple(t.cuda() for t in s) for s in state]


def previous(rollout):
    actions, dones = rollout["actions"], rollout["dones"]
    prev = torch.full_like(actions, -1)
    prev[1:] = torch.where(dones[:-1] != 0, -1, actions[:-1])
    return prev.contiguous(), dones


def trunk(rx, p, prev, states, conv, scan, drop):
    """conv and scan: the rollout's operators or the steps'; drop(i): options."""
    stream = rx.embed(p["table"], prev)
    stream, x = rx.residual_norm(stream, weight=p["norm"])
    after = []
    for i in range(BLOCKS):
        h, cs = conv(x @ p[f"inp{i}"], p[f"conv{i}"], states[i][0], p[f"convb{i}"])
        d, b, c = (h @ p[f"proj{i}"]).split([D, S, S], -1)
        y, ss = scan(h, d, p[f"rate{i}"], b, c, states[i][1], skip=p[f"skip{i}"], gate=x @ p[f"gatew{i}"],
                     delta_bias=p[f"bias{i}"])
        stream, x = rx.residual_norm(stream, y, p[f"pre{i}"], branch_weight=p[f"post{i}"], gate=p[f"scale{i}"], **drop(i))
        after.append((cs, ss))
    return rx.shape_logits(x @ p["out"].t()), after


def plain(p, prev, dones, states):
    """The same in 64 bits on the CPU, step by step, from the definitions."""
    kept = []
    for i in range(BLOCKS):
        k, scale = ref.kept(L * N * D, DROP, SEED, i)
        kept.append(torch.from_numpy(k.reshape(L, N, D)) * scale)
    rms = lambda v: v / torch.sqrt((v * v).mean(-1, keepdim=True) + float(np.float32(1e-6)))
    states = [list(s) for s in states]
    zs = []
    for t in range(L):
        if t:
            m = (dones[t - 1] == 0)[:, None, None]
            states = [[torch.where(m, v, 0.0) for v in s] for s in states]
        stream = torch.where((prev[t] >= 0)[:, None], p["table"][prev[t].clamp(min=0).long()], 0.0)
        x = rms(stream) * p["norm"]
        for i in range(BLOCKS):
            window = torch.cat([states[i][0], (x @ p[f"inp{i}"])[:, None]], 1)
            h = torch.nn.functional.silu((window * p[f"conv{i}"].t()).sum(1) + p[f"convb{i}"])
            d, b, c = (h @ p[f"proj{i}"]).split([D, S, S], -1)
            dt = torch.nn.functional.softplus(d + p[f"bias{i}"])
            s = torch.exp(dt[..., None] * p[f"rate{i}"]) * states[i][1] + (dt * h)[..., None] * b[:, None]
            y = ((s * c[:, None]).sum(-1) + p[f"skip{i}"] * h) * torch.nn.functional.silu(x @ p[f"gatew{i}"])
            stream = stream + p[f"scale{i}"] * rms(y) * p[f"post{i}"] * kept[i][t]
            x = rms(stream) * p[f"pre{i}"]
            states[i] = [window[:, 1:], s]
        zs.append(x @ p["out"].t())
    return torch.stack(zs), states


def test_forward_and_every_gradient(rollout):  # noqa: F811
    import rl_experience_collection_amd as rx
    prev, dones = previous(rollout)
    p, states = parameters()
    for v in list(p.values()) + [t for s in states for t in s]:
        v.requires_grad_()
    z, after = trunk(rx, p, prev, states, lambda x, w, s, b: rx.causal_conv(x, w, b, s, dones=dones),
                     lambda x, d, r, b, c, s, **kw: rx.selective_scan(x, d.contiguous(), r, b, c, state=s, dones=dones, **kw),
                     lambda i: dict(dropout=DROP, seed=SEED, offset=i))
    actions = rollout["actions"].long()
    weight = rollout["advantages"]

    def loss(z, actions, weight):
        return (torch.log_softmax(z, -1).gather(2, actions[..., None])[..., 0] * weight).sum()

    leaves = list(p.values()) + [t for s in states for t in s]
    got = torch.autograd.grad(loss(z, actions, weight), leaves)
    c = lambda t: t.detach().cpu()
    q = {k: c(v).double().requires_grad_() for k, v in p.items()}
    r0 = [tuple(c(t).double().requires_grad_() for t in s) for s in states]
    rz, rafter = plain(q, c(prev), c(dones), r0)
    want = torch.autograd.grad(loss(rz, c(actions), c(weight).double()), list(q.values()) + [t for s in r0 for t in s])
    # Each of the two blocks is five products of 32 terms, a scan of at most 60
    # steps with 30 roundings a step, two norms of 40 and some 100 others:
    # about 2200 roundings, each of at most u of values that the norms bring
    # back to order 1; a norm and a gate may multiply what comes in by 4 at
    # most here. Relative to the largest output 2 * 2200 * 4 u stays below:
    tol = 2 * 2200 * 4 * 2.0 ** -24
    assert (c(z).double() - rz).abs().max() < tol * rz.abs().max()
    for i in range(BLOCKS):
        ended = (c(dones)[L - 1] == 0)[:, None, None]
        for a, b in zip(after[i], rafter[i]):
            b = torch.where(ended, b, 0.0)
            assert (c(a).double() - b).abs().max() < tol * b.abs().max()
    # the gradients pass the same way back, over forward values with that error
    for name, a, b in zip(list(p) + ["state"] * 4, got, want):
        err = float((c(a).double() - b).abs().max() / b.abs().max())
        assert err < 2 * tol, (name, err)


def test_acting_step_by_step_follows_the_rollout(rollout):  # noqa: F811
    import rl_experience_collection_amd as rx
    prev, dones = previous(rollout)
    p, states = parameters()
    with torch.no_grad():
        z, after = trunk(rx, p, prev, states, lambda x, w, s, b: rx.causal_conv(x, w, b, s, dones=dones),
                         lambda x, d, r, b, c, s, **kw: rx.selective_scan(x, d, r, b, c, state=s, dones=dones, **kw),
                         lambda i: {})
        states = [tuple(t.clone() for t in s) for s in states]
        for t in range(L):
            cut = dones[t - 1] if t else None
            zt, _ = trunk(rx, p, prev[t], states,
                          lambda x, w, s, b: rx.causal_conv_step(x, w, s, bias=b, resets=cut, out_state=s),
                          lambda x, d, r, b, c, s, **kw: rx.selective_scan_step(x, d, r, b, c, s, resets=cut, out_state=s, **kw),
                          lambda i: {})
            # both are within the tolerance of the test above of the same values
            # (the first step has no previous action: all is 0)
            assert (zt - z[t]).abs().max() <= 2 * 2 * 2200 * 4 * 2.0 ** -24 * z[t].abs().max(), t
        for s, a in zip(states, after):
            for u, v in zip(s, a):
                u = u.clone()
                u[dones[L - 1] != 0] = 0
                assert (u - v).abs().max() < 2 * 2 * 2200 * 4 * 2.0 ** -24 * v.abs().max()
