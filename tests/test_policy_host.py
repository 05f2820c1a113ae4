"""The policy operators (include/policy.h) without a GPU: exported symbols,
struct layouts, the refusals of the C entry points and of the binding, and
the 64-bit reference's gradients against differences."""
import ctypes as C
import os
import re

import numpy as np
import pytest
import torch

import policy_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, OK = -1, 0


@pytest.fixture(scope="module")
def rx():
    import rl_experience_collection_amd as rx
    rx.load_library()
    return rx


@pytest.fixture(scope="module")
def policy(rx):
    from rl_experience_collection_amd import policy
    return policy


def test_library_exports_the_header(rx, policy):
    txt = open(os.path.join(ROOT, "include", "policy.h")).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    names = set(re.findall(r"^\s*(?:int|int64_t)\s+(\w+)\s*\(", txt, flags=re.M))
    assert names == set(policy.EXPORTED)
    for n in names:
        assert hasattr(rx.load_library(), n)


def test_recur_struct_sizes(policy):
    # 5 ints (padded to 24 bytes), strides, pointers, workspace size
    assert C.sizeof(policy.RecurArgs) == 24 + 8 * (6 + 7 + 1)
    assert C.sizeof(policy.RecurGradArgs) == 24 + 8 * (12 + 11 + 1)


def _recur_args(policy, **kw):
    a = policy.RecurArgs(steps=4, rows=2, width=3, dtype=0, form=0, x_step=6, x_row=3, gate_step=6,
                         gate_row=3, h_step=6, h_row=3, x=64, gate=64, h=64)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,text", [
    (dict(steps=-1), "negative size"), (dict(rows=-2), "negative size"),
    (dict(rows=1 << 20, width=1 << 11), "2\\^31"), (dict(dtype=3), "dtype"), (dict(form=2), "form"),
    (dict(x=None), "x is NULL"), (dict(gate=None), "gate is NULL"), (dict(h=None), "h is NULL"),
    (dict(x=66), "aligned"), (dict(dtype=1, gate=65), "aligned"), (dict(h0=2), "h0 is not aligned"),
    (dict(x_step=-6), "stride"), (dict(h_row=-1), "stride"),
    (dict(steps=100000), "workspace")])
def test_recur_forward_refuses(rx, policy, change, text):
    lib = rx.load_library()
    assert lib.recur_forward(C.byref(_recur_args(policy, **change)), None) == EINVAL
    assert re.search(text, rx.rollout_last_error()), rx.rollout_last_error()


def test_recur_other_refusals(rx, policy):
    lib = rx.load_library()
    assert lib.recur_forward(None, None) == EINVAL
    assert lib.recur_backward(None, None) == EINVAL
    assert lib.recur_workspace(5, -1, 3, 0) == EINVAL
    assert lib.recur_workspace(5, 1, 3, 9) == EINVAL
    assert lib.recur_workspace(5, 1, 3, 0) == 0
    assert [lib.recur_workspace(*z, 0) for z in ((0, 3, 4), (100000, 0, 4), (5, 3, 0))] == [0, 0, 0]
    assert lib.recur_workspace(100000, 1, 3, 0) > 0
    g = policy.RecurGradArgs(steps=4, rows=2, width=3, dtype=0, form=1, gate=64, h=64, dh=64, dx=64,
                             dgate=64)
    assert lib.recur_backward(C.byref(g), None) == EINVAL
    assert "x is NULL" in rx.rollout_last_error()
    g.form, g.dx = 0, None
    assert lib.recur_backward(C.byref(g), None) == EINVAL
    assert "dx is NULL" in rx.rollout_last_error()
    assert lib.recur_step(2, 3, 0, 0, 64, 3, 64, 3, None, None, 64, 3, 64, None) == EINVAL
    assert "state is NULL" in rx.rollout_last_error()
    assert lib.recur_step(2, 3, 0, 5, 64, 3, 64, 3, 64, None, 64, 3, 64, None) == EINVAL
    # nothing to do: accepted without a device
    assert lib.recur_forward(C.byref(_recur_args(policy, rows=0)), None) == OK
    assert lib.recur_forward(C.byref(_recur_args(policy, width=0)), None) == OK
    assert lib.recur_step(0, 3, 0, 0, None, 3, None, 3, None, None, None, 3, None, None) == OK


def test_recurrence_binding_refusals(rx):
    x = torch.zeros(4, 2, 3)
    for kw, text in [(dict(form="tanh"), "form"), (dict(gate=torch.zeros(4, 2, 2)), "shape"),
                     (dict(gate=x.bfloat16()), "dtype"), (dict(x=x.double()), "float32"),
                     (dict(x=x[0]), r"\[L, N, D\]"), (dict(h0=torch.zeros(2, 4)), "h0"),
                     (dict(h0=torch.zeros(2, 3).half()), "h0"),
                     (dict(dones=torch.zeros(4, 2)), "dones"),
                     (dict(dones=torch.zeros(2, 4, dtype=torch.uint8)), "dones"),
                     (dict(x=x.permute(1, 2, 0), gate=x.permute(1, 2, 0)), "last dimension"),
                     (dict(), "device")]:
        args = dict(dict(x=x, gate=x), **kw)
        if not torch.cuda.is_available() and text == "device":
            continue  # the device itself cannot be asked for
        with pytest.raises(ValueError, match=text):
            rx.recurrence(**args)
    s = torch.zeros(2, 3)
    for kw, text in [(dict(state=s.half()), "state"), (dict(resets=torch.zeros(3, dtype=torch.bool)), "resets"),
                     (dict(out_state=torch.zeros(3, 3)), "out_state"),
                     (dict(x=x[0].clone().requires_grad_()), "no_grad")]:
        with pytest.raises(ValueError, match=text):
            rx.recurrence_step(**dict(dict(x=x[0], gate=x[0], state=s), **kw))


@pytest.mark.parametrize("sig", [False, True])
def test_reference_recurrence_gradient_against_differences(sig):
    rng = np.random.default_rng(3)
    L, N, D = 7, 2, 3
    x, dh = rng.standard_normal((2, L, N, D))
    gate = rng.standard_normal((L, N, D)) if sig else rng.uniform(0.3, 1, (L, N, D))
    h0, dl = rng.standard_normal((2, N, D))
    dones = (rng.random((L, N)) < 0.3).astype(np.uint8)
    g = ref.recurrence_grad(x, gate, h0, dones, dh, dl, sig, "f32")

    def loss(x, gate, h0):
        f = ref.recurrence(x, gate, h0, dones, sig, "f32")
        return (f["h"] * dh).sum() + (f["h_last"] * dl).sum()

    for k, got in enumerate((g["dx"], g["dgate"], g["dh0"])):
        args = [x, gate, h0]
        num = np.zeros_like(args[k])
        for i in np.ndindex(num.shape):
            e = np.zeros_like(num)
            e[i] = 1e-6
            up, dn = list(args), list(args)
            up[k], dn[k] = args[k] + e, args[k] - e
            num[i] = (loss(*up) - loss(*dn)) / 2e-6
        # a central difference of step 1e-6: truncation ~1e-12, rounding ~1e-9
        assert np.abs(num - got).max() < 1e-7
