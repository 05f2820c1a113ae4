"""recur_forward_kept and recur_backward_kept (include/policy.h) without a
GPU: their refusals, and what their workspaces hold."""
import ctypes as C

import pytest

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


def forward_args(policy, **kw):
    return policy.RecurArgs(**dict(dict(steps=4, rows=2, width=3, dtype=1, form=1, x_step=6, x_row=3,
                                        gate_step=6, gate_row=3, h_step=6, h_row=3, x=64, gate=64, h=64),
                                   **kw))


def backward_args(policy, **kw):
    return policy.RecurGradArgs(**dict(dict(steps=4, rows=2, width=3, dtype=1, form=1, x=64, gate=64, h=None,
                                            dh=64, dx=64, dgate=64), **kw))


def test_kept_refusals(rx, policy):
    lib = rx.load_library()
    assert lib.recur_forward_kept(None, 64, None) == EINVAL
    assert lib.recur_backward_kept(None, 64, None) == EINVAL
    for kept, text in ((None, "kept is NULL"), (66, "kept is not aligned")):
        assert lib.recur_forward_kept(C.byref(forward_args(policy)), kept, None) == EINVAL
        assert text in rx.rollout_last_error()
        assert lib.recur_backward_kept(C.byref(backward_args(policy)), kept, None) == EINVAL
        assert text in rx.rollout_last_error()
    # the 16-bit sigmoid gradient takes the states, not h; the others take h
    for kw in (dict(dtype=0), dict(form=0)):
        assert lib.recur_backward_kept(C.byref(backward_args(policy, **kw)), 64, None) == EINVAL
        assert "h is NULL" in rx.rollout_last_error()
    assert lib.recur_kept_workspace(5, -1, 3, 0) == EINVAL
    assert lib.recur_forward_kept(C.byref(forward_args(policy, rows=0)), None, None) == OK
    assert lib.recur_backward_kept(C.byref(backward_args(policy, width=0)), None, None) == OK


def test_workspaces(rx, policy):
    lib = rx.load_library()
    for L, N, D in ((1, 1, 1), (9, 2, 3), (500, 8192, 64), (100000, 1, 3)):
        kept = 4 * ((L + 7) // 8) * N * D
        assert lib.recur_workspace(L, N, D, 0) == lib.recur_kept_workspace(L, N, D, 0)
        for dt in (1, 2):
            assert lib.recur_workspace(L, N, D, dt) >= lib.recur_kept_workspace(L, N, D, dt) + kept
    for z in ((0, 3, 4), (100000, 0, 4), (5, 3, 0)):
        assert lib.recur_workspace(*z, 1) == 0 and lib.recur_kept_workspace(*z, 1) == 0


def test_the_gradient_without_kept_states_needs_its_workspace(rx, policy):
    lib = rx.load_library()
    a = backward_args(policy, workspace=64, workspace_bytes=lib.recur_workspace(4, 2, 3, 1) - 1)
    assert lib.recur_backward(C.byref(a), None) == EINVAL
    assert "workspace" in rx.rollout_last_error()
