"""The gradient of the sigmoid form in 16-bit types: the state that enters a
step counts in fp32, not as the output rounded it, because dgate takes the
difference of that state and the input."""
import ctypes as C

import numpy as np
import pytest
import torch

import policy_ref as ref
from parity import gpu_available
from test_gpu_recur import f64, inputs, within

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X")]


@pytest.fixture(scope="module")
def rx():
    import rl_experience_collection_amd as rx
    return rx


def following(L, N, D, name, noise, p_done, seed, h0=True):
    """Inputs that the state comes close to: a constant per channel and a little noise."""
    i = inputs(L, N, D, name, True, p_done, seed, h0)
    g = torch.Generator().manual_seed(seed + 1000)
    x = torch.randn(1, N, D, generator=g) + noise * torch.randn(L, N, D, generator=g)
    return dict(i, x=x.to(i["x"].dtype))


def bounds(i, name):
    """The 64-bit form with the bounds of states in fp32; each output is then
    rounded once to its type."""
    n = {k: f64(v) for k, v in i.items()}
    w = ref.recurrence_grad(n["x"], n["gate"], n["h0"], n["dones"], n["dh"], n["dl"], True, "f32")
    for k, e in (("h", "eh"), ("dx", "edx"), ("dgate", "edg")):
        w[e] = w[e] + ref.half(name, np.abs(w[k]) + w[e])
    return w


def grads(rx, c):
    leaves = [c[k].detach().clone().requires_grad_() for k in ("x", "gate", "h0") if c[k] is not None]
    out = rx.recurrence(leaves[0], leaves[1], leaves[2] if len(leaves) > 2 else None, c["dones"])
    return list(out) + list(torch.autograd.grad(out, leaves, (c["dh"], c["dl"])))


def compare(got, w):
    for t, k, e in zip(got, ("h", "h_last", "dx", "dgate", "dh0"), ("eh", "elast", "edx", "edg", "edh0")):
        within(t, w[k], w[e], k)


# one lane a channel and two and four, one tile and many, tiles in a chain,
# widths that are no multiple of a lane's channels
SIZES = [(1, 1, 1), (7, 2, 5), (8, 3, 2), (9, 3, 33), (64, 2, 65), (100, 4, 130), (129, 3, 1), (300, 5, 63),
         (700, 2, 70), (2050, 1, 9), (200, 550, 66), (200, 2048, 34), (150, 2730, 30)]


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("L,N,D", SIZES)
def test_states_that_follow_their_input(rx, L, N, D, name):
    i = following(L, N, D, name, 0.01, 0.02, L * 7 + D)
    compare(grads(rx, {k: v.cuda() for k, v in i.items()}), bounds(i, name))


@pytest.mark.parametrize("p_done", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("L,N,D", [(70, 3, 10), (1100, 2, 6), (70, 2048, 34)])
def test_dones_and_no_start(rx, L, N, D, p_done):
    i = following(L, N, D, "bf16", 0.01, p_done, 5, h0=False)
    c = {k: None if v is None else v.cuda() for k, v in i.items()}
    compare(grads(rx, c), bounds(i, "bf16"))


def test_strides(rx):
    L, N, D = 700, 3, 13
    i = following(L, N, D, "bf16", 0.01, 0.02, 9)
    c = {k: v.cuda() for k, v in i.items()}
    wide = torch.full((N, L, 2 * D + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :, :D], wide[:, :, D + 3:] = c["x"].transpose(0, 1), c["gate"].transpose(0, 1)
    leaf = wide.requires_grad_()
    out = rx.recurrence(leaf[:, :, :D].transpose(0, 1), leaf[:, :, D + 3:].transpose(0, 1), c["h0"], c["dones"])
    g, = torch.autograd.grad(out, leaf, (c["dh"], c["dl"]))
    w = bounds(i, "bf16")
    within(g[:, :, :D].transpose(0, 1), w["dx"], w["edx"], "dx")
    within(g[:, :, D + 3:].transpose(0, 1), w["dgate"], w["edg"], "dgate")


@pytest.mark.parametrize("L", [40, 300, 1300])
def test_a_finished_episode_stays_behind_its_done(rx, L):
    i = following(L, 2, 5, "bf16", 0.01, 0.0, 11)
    i["dones"] = torch.zeros(L, 2, dtype=torch.uint8)
    i["dones"][9, 0] = 1
    c = {k: v.cuda() for k, v in i.items()}
    clean = grads(rx, c)
    x = c["x"].clone()
    x[5, 0, 1] = float("nan")
    got = grads(rx, dict(c, x=x))
    assert torch.isnan(got[3][6:10, 0, 1]).all()
    for k in (0, 2, 3):
        assert torch.equal(got[k][10:], clean[k][10:]) and torch.equal(got[k][:, 1], clean[k][:, 1])
    assert torch.equal(got[3][:5], clean[3][:5])


def test_the_output_may_change_before_the_gradient(rx):
    """The gradient does not read h: a residual sum in place is allowed."""
    i = following(300, 3, 20, "bf16", 0.1, 0.02, 12)
    c = {k: v.cuda() for k, v in i.items()}
    want = grads(rx, c)
    leaves = [c[k].detach().clone().requires_grad_() for k in ("x", "gate", "h0")]
    h, last = rx.recurrence(*leaves, c["dones"])
    h += 1
    for a, b in zip(torch.autograd.grad((h, last), leaves, (c["dh"], c["dl"])), want[2:]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("L,N,D", [(1, 1, 1), (64, 3, 5), (700, 2, 70), (150, 2048, 34)])
def test_gradient_without_kept_states(rx, L, N, D, name):
    """recur_backward of the C interface forms the states again: the same bits
    as with the states that the forward pass kept."""
    from rl_experience_collection_amd import policy
    i = following(L, N, D, name, 0.01, 0.02, 13)
    c = {k: v.cuda() for k, v in i.items()}
    want = grads(rx, c)
    lib, dt = rx.load_library(), policy._DTYPES[c["x"].dtype]
    size = lib.recur_workspace(L, N, D, dt)
    assert size >= lib.recur_kept_workspace(L, N, D, dt) + 4 * ((L + 7) // 8) * N * D
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    dx, dg, dh0 = torch.empty_like(c["x"]), torch.empty_like(c["x"]), torch.empty_like(c["h0"])
    row = dict(x_step=N * D, x_row=D, gate_step=N * D, gate_row=D, dh_step=N * D, dh_row=D,
               dx_step=N * D, dx_row=D, dgate_step=N * D, dgate_row=D)
    a = policy.RecurGradArgs(steps=L, rows=N, width=D, dtype=dt, form=1, x=c["x"].data_ptr(),
                             gate=c["gate"].data_ptr(), h0=c["h0"].data_ptr(), dones=c["dones"].data_ptr(),
                             dh=c["dh"].data_ptr(), dh_last=c["dl"].data_ptr(), dx=dx.data_ptr(),
                             dgate=dg.data_ptr(), dh0=dh0.data_ptr(), workspace=ws.data_ptr(),
                             workspace_bytes=size, **row)
    assert lib.recur_backward(C.byref(a), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    for got, w in zip((dx, dg, dh0), want[2:]):
        assert torch.equal(got, w)


def test_kept_states_are_the_forward_passs(rx):
    from rl_experience_collection_amd import policy
    L, N, D = 45, 3, 6
    i = following(L, N, D, "bf16", 0.1, 0.1, 14)
    c = {k: v.cuda() for k, v in i.items()}
    lib = rx.load_library()
    kept = torch.full((7, N, D), 7.0, device="cuda")
    h = torch.empty_like(c["x"])
    a = policy.RecurArgs(steps=L, rows=N, width=D, dtype=1, form=1, x_step=N * D, x_row=D, gate_step=N * D,
                         gate_row=D, h_step=N * D, h_row=D, x=c["x"].data_ptr(), gate=c["gate"].data_ptr(),
                         h0=c["h0"].data_ptr(), dones=c["dones"].data_ptr(), h=h.data_ptr())
    assert lib.recur_kept_workspace(L, N, D, 1) == 0
    s = torch.cuda.current_stream().cuda_stream
    assert lib.recur_forward_kept(C.byref(a), kept.data_ptr(), s) == 0
    torch.cuda.synchronize()
    assert torch.equal(kept[0], c["h0"]) and (kept[6] == 7).all()
    # (state 8 k - 1, rounded, is the output of that step)
    assert torch.equal(kept[1:6].bfloat16(), h[7:40:8])
