"""What the policy binding tells torch's autograd, without a GPU: a stand-in
takes the library's place and writes nothing."""
import pytest
import torch
import torch.autograd.forward_ad as fwd


@pytest.fixture
def rx(monkeypatch):
    import rl_experience_collection_amd as rx
    from rl_experience_collection_amd import policy
    policy._lib()
    monkeypatch.setattr(policy, "_here", lambda name, *tensors: 0)
    monkeypatch.setattr(policy, "_there", lambda t: 0)
    monkeypatch.setattr(policy, "_call", lambda fn, *args: None)
    return rx


def calls(rx):
    """Each operator as a function of one tensor, by input."""
    x, s, w = torch.ones(4, 2, 3), torch.ones(2, 3), torch.ones(5, 3)
    i, z = torch.zeros(4, dtype=torch.int32), torch.ones(2, 5)
    history = torch.zeros(2, 3, dtype=torch.int32)
    return {
        "embed weight": (w, lambda t: rx.embed(t, i)),
        "recurrence x": (x, lambda t: rx.recurrence(t, x)),
        "recurrence gate": (x, lambda t: rx.recurrence(x, t, form="linear")),
        "recurrence h0": (s, lambda t: rx.recurrence(x, x, t)),
        "recurrence_step x": (s, lambda t: rx.recurrence_step(t, s, s)),
        "recurrence_step gate": (s, lambda t: rx.recurrence_step(s, t, s)),
        "recurrence_step state": (s, lambda t: rx.recurrence_step(s, s, t)),
        "recurrence_step out_state": (s, lambda t: rx.recurrence_step(s, s, s, out_state=t)),
        "shape_logits logits": (z, lambda t: rx.shape_logits(t)),
        "shape_logits bias": (z[0], lambda t: rx.shape_logits(z, bias=t)),
        "shape_logits repetition": (z[:, 0].clone(), lambda t: rx.shape_logits(z, history=history, repetition=t)),
        "shape_logits presence": (z[:, 0].clone(), lambda t: rx.shape_logits(z, history=history, presence=t)),
        "shape_logits frequency": (z[:, 0].clone(), lambda t: rx.shape_logits(z, history=history, frequency=t)),
        "shape_logits with out": (z, lambda t: rx.shape_logits(t, out=torch.empty(2, 5))),
        "shape_logits out": (z, lambda t: rx.shape_logits(z, out=t)),
    }


NAMES = ["embed weight", "recurrence x", "recurrence gate", "recurrence h0", "recurrence_step x",
         "recurrence_step gate", "recurrence_step state", "recurrence_step out_state", "shape_logits logits",
         "shape_logits bias", "shape_logits repetition", "shape_logits presence", "shape_logits frequency",
         "shape_logits with out", "shape_logits out"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("grad_mode", [True, False])
def test_forward_mode_derivatives_are_refused(rx, name, grad_mode):
    """A dual tensor asks for no gradient; its tangent must not be lost in silence."""
    t, call = calls(rx)[name]
    call(t)
    with fwd.dual_level():
        call(t)  # no tangent: the call is like any other
        with torch.set_grad_enabled(grad_mode), pytest.raises(NotImplementedError, match="forward-mode"):
            call(fwd.make_dual(t.clone(), torch.ones_like(t)))


@pytest.mark.parametrize("name", NAMES)
def test_function_transforms_are_refused(rx, name):
    t, call = calls(rx)[name]
    with pytest.raises(RuntimeError):
        torch.func.jvp(call, (t,), (torch.ones_like(t),))
    with pytest.raises((RuntimeError, ValueError)):
        torch.func.vmap(call)(torch.stack([t, t]))


@pytest.mark.parametrize("name", [n for n in NAMES if "step" not in n and "out" not in n and
                                  n.split()[1] not in ("repetition", "presence", "frequency")])
def test_a_tangent_in_the_gradient_is_refused(rx, name):
    """Forward over reverse: the gradient that a backward pass is given is dual."""
    t, call = calls(rx)[name]
    leaf = t.clone().requires_grad_()
    out = call(leaf)
    out = out[0] if isinstance(out, tuple) else out
    with fwd.dual_level(), pytest.raises(NotImplementedError, match="forward-mode"):
        torch.autograd.grad(out, leaf, fwd.make_dual(torch.ones_like(out), torch.ones_like(out)))
