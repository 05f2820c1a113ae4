"""Outputs that the caller hands to the policy operators, without a GPU: what
autograd learns of the write, and what is refused.  A stand-in takes the
library's place and writes nothing."""
import pytest
import torch

from test_policy_autograd_host import rx  # noqa: F401  (the stand-in)


def into(rx, t):
    """The calls that write into t [2, 5]."""
    s = torch.ones(2, 5)
    return [lambda: rx.shape_logits(s, out=t), lambda: rx.recurrence_step(s, s, s.clone(), out_state=t)]


@pytest.mark.parametrize("k", [0, 1])
def test_a_graph_that_holds_the_old_values_notices(rx, k):
    """y's gradient by w needs what t held: overwritten, it is gone."""
    t, w = torch.ones(2, 5), torch.ones(2, 5, requires_grad=True)
    y = (w * t).sum()
    with torch.no_grad():
        into(rx, t)[k]()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@pytest.mark.parametrize("k", [0, 1])
def test_a_view_shares_its_base(rx, k):
    base, w = torch.ones(4, 5), torch.ones(4, 5, requires_grad=True)
    y = (w * base).sum()
    into(rx, base[1:3])[k]()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@pytest.mark.parametrize("k", [0, 1])
def test_inference_mode(rx, k):
    with torch.inference_mode():
        into(rx, torch.ones(2, 5))[k]()


@pytest.mark.parametrize("k", [0, 1])
def test_an_output_that_asks_for_a_gradient_is_refused(rx, k):
    leaf = torch.ones(2, 5, requires_grad=True)
    with pytest.raises(ValueError, match="no_grad"):
        into(rx, leaf)[k]()
    with pytest.raises(ValueError, match="no_grad"):
        into(rx, leaf * 2)[k]()
    with torch.no_grad():
        into(rx, leaf)[k]()
