"""The operators of a residual block (include/block.h) on arrays whose offsets
pass 32 bits, against the same values close together."""
import numpy as np
import pytest
import torch

import block_ref as ref
from parity import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X")]

FAR = 2 ** 31 + 64  # elements between steps or rows: more than 4 GiB of bf16


@pytest.fixture(scope="module")
def rx():
    import rl_experience_collection_amd as rx
    yield rx
    torch.cuda.empty_cache()


def spread(t):
    """The same values, the first axis FAR elements apart."""
    out = torch.empty((t.shape[0] - 1) * FAR + t[0].numel(), dtype=t.dtype, device="cuda")
    out = out.as_strided(t.shape, (FAR,) + t.stride()[1:])
    return out.copy_(t)


def grads(outs, leaves, douts):
    return list(outs) + list(torch.autograd.grad(outs, leaves, douts))


def test_steps_far_apart(rx):
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g).cuda()
    L, N, D, S = 3, 2, 40, 16
    bf = lambda t: t.bfloat16()
    x, delta, gate, b, c, dy = bf(n(L, N, D)), bf(n(L, N, D)), bf(n(L, N, D)), bf(n(L, N, S)), bf(n(L, N, S)), bf(n(L, N, D))
    rate, state, w = -torch.exp(n(D, S)), n(N, D, S), n(D, 4)

    def scan(f):
        leaves = [f(t).requires_grad_() for t in (x, delta, gate, b, c)]
        y, new = rx.selective_scan(leaves[0], leaves[1], rate, leaves[3], leaves[4], gate=leaves[2], state=state)
        return [t.contiguous() for t in grads((y, new), leaves, (f(dy), new.detach()))]

    def conv(f):
        leaf = f(x).requires_grad_()
        y, new = rx.causal_conv(leaf, w)
        return [t.contiguous() for t in grads((y, new), [leaf], (f(dy), new.detach()))]

    for run in (scan, conv):
        for a, b2 in zip(run(lambda t: t.clone()), run(spread)):
            assert torch.equal(a, b2)


def test_rows_far_apart(rx):
    g = torch.Generator().manual_seed(2)
    n = lambda *s: torch.randn(*s, generator=g).cuda().bfloat16()
    res, br, gate = n(2, 130), n(2, 130), n(2, 130)

    def run(f):
        leaves = [f(t).requires_grad_() for t in (res, br, gate)]
        out = rx.residual_norm(leaves[0], leaves[1], gate=leaves[2], activation="sigmoid", dropout=0.3, seed=4)
        return grads(out, leaves, [torch.ones_like(t) for t in out])

    for a, b in zip(run(lambda t: t.clone()), run(spread)):
        assert torch.equal(a, b)


def test_more_than_2_to_32_elements(rx):
    D = 8192
    R = 2 ** 32 // D + 3
    x = torch.empty(R, D, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(3, D, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    x[:-3] = 1.0
    x[-3:] = tail
    stream, normed = rx.residual_norm(x, residual_scale=0.5)
    want = rx.residual_norm(tail, residual_scale=0.5)
    assert torch.equal(stream[-3:], want[0]) and torch.equal(normed[-3:], want[1])
    assert torch.equal(stream[0], torch.full((D,), 0.5, dtype=torch.bfloat16, device="cuda"))
    del stream, normed
    y = rx.dropout(x, 0.25, 11)
    for start in (0, 2 ** 32 - 500, R * D - 1000):
        kept, scale = ref.kept(1000, 0.25, 11, start=start)
        got = y.view(-1)[start:start + 1000].cpu().double().numpy()
        want = np.where(kept, x.view(-1)[start:start + 1000].cpu().double().numpy() * scale, 0.0)
        assert (np.abs(got - want) <= ref.fin("bf16", want, 2 * ref.U * np.abs(want))).all()


@pytest.mark.parametrize("name", [torch.bfloat16, torch.float32])
def test_as_many_channels_as_are_allowed(rx, name):
    """2^28 - 1 channels of 3 taps: more workgroups across a row than a grid's
    second dimension holds, 2^30 - 4 columns of parameters' gradients."""
    D = 2 ** 28 - 1
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(1, 1, D, generator=g, device="cuda").to(name).requires_grad_()
    w = torch.randn(D, 3, generator=g, device="cuda").requires_grad_()
    bias = torch.randn(D, generator=g, device="cuda").requires_grad_()
    y, _ = rx.causal_conv(x, w, bias, activation="none")
    dy = torch.randn(1, 1, D, generator=g, device="cuda").to(name)
    dx, dw, db = torch.autograd.grad(y, (x, w, bias), dy)
    # one product each, exact in 64 bits, and its roundings to fp32 and to the type
    u = ref.U if name == torch.float32 else ref.U + 2.0 ** -8
    with torch.no_grad():
        xf, dyf = x[0, 0].double(), dy[0, 0].double()
        for got, want, near in ((dx[0, 0], dyf * w[:, 2], u), (dw[:, 2], dyf * xf, ref.U)):
            off = (got.double() - want).abs_() - 1.01 * near * want.abs()
            assert (off <= ref.TINY).all()
            del off, want
        p = xf * w[:, 2]
        off = (y[0, 0].double() - (p + bias)).abs_() - 1.01 * u * (p + bias).abs()
        off -= 1.01 * ref.U * p.abs_()
        assert (off <= ref.TINY).all()
        assert torch.equal(db, dy[0, 0].float()) and not dw[:, :2].any()
