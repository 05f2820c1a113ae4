"""Inputs that take no gradient, without a GPU: refused where they would be
asked for one, and fine under torch.no_grad()."""
import pytest
import torch

from test_policy_autograd_host import rx  # noqa: F401  (the stand-in)


@pytest.mark.parametrize("name,shape", [("bias", (2, 5)), ("repetition", (2,)), ("presence", (2,)),
                                        ("frequency", (2,))])
def test_leaves_without_a_gradient_of_their_own(rx, name, shape):
    z, history = torch.ones(2, 5), torch.zeros(2, 3, dtype=torch.int32)
    leaf = torch.ones(shape, requires_grad=True)
    with pytest.raises(ValueError, match="gradient"):
        rx.shape_logits(z, history=history, **{name: leaf})
    with torch.no_grad():
        out = rx.shape_logits(z, history=history, **{name: leaf})
    assert out.shape == z.shape and not out.requires_grad
