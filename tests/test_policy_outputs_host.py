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


def test_a_shifted_output_is_refused(rx):
    """The output may be the input itself or lie apart from it; where they share
    some elements only, it would be written while others still read it."""
    flat = torch.ones(64)
    z = flat[:40].view(8, 5)
    for lo in (1, 5, 24):
        with pytest.raises(ValueError, match="overlap"):
            rx.shape_logits(z, out=flat[lo:lo + 40].view(8, 5))
        with pytest.raises(ValueError, match="overlap"):
            rx.recurrence_step(torch.ones(8, 5), torch.ones(8, 5), z, out_state=flat[lo:lo + 40].view(8, 5))
    for same in (z, z.view(8, 5)):
        rx.shape_logits(z, out=same)
        rx.recurrence_step(torch.ones(8, 5), torch.ones(8, 5), z, out_state=same)
    rx.shape_logits(flat[:20].view(4, 5), out=flat[20:40].view(4, 5))
    rx.shape_logits(z[:1], out=z[:1])
    rx.shape_logits(z[:0], out=z[:0])


def test_rows_side_by_side_are_not_an_overlap(rx):
    wide = torch.ones(8, 12)
    rx.shape_logits(wide[:, :5], out=wide[:, 5:10])
    rx.shape_logits(wide[:, 7:], out=wide[:, :5])
    rx.shape_logits(wide[:, 2:7], out=wide[:, 2:7])
    rx.shape_logits(wide[1:, 7:], out=wide[:-1, :5])
    for a, b in ((wide[:, :5], wide[:, 4:9]), (wide[:, 7:], wide[:, 4:9]), (wide[1:, :5], wide[:-1, :5]),
                 (wide[1:, 7:], wide[:-1, 5:10])):
        with pytest.raises(ValueError, match="overlap"):
            rx.shape_logits(a, out=b)
    # 16-bit rows between each other, one set the row's other half
    half = torch.ones(8, 10, dtype=torch.bfloat16)
    rx.shape_logits(half[:, 5:], out=half[:, :5])


def test_rows_of_different_strides(rx):
    """Against the elements themselves, over layouts of one small buffer."""
    buffer = torch.ones(60)
    verdicts = set()
    for rows, width in ((1, 3), (2, 3), (3, 2)):
        for s0 in range(width, 9):
            for s1 in range(width, 9):
                for lo in range(0, 24):
                    z = buffer.as_strided((rows, width), (s0, 1), 10)
                    out = buffer.as_strided((rows, width), (s1, 1), lo)
                    cells = [{o + r * s + c for r in range(rows) for c in range(width)}
                             for o, s in ((10, s0), (lo, s1))]
                    same = lo == 10 and (rows == 1 or s0 == s1)
                    fine = same or not cells[0] & cells[1]
                    verdicts.add((fine, s0 == s1))
                    if fine:
                        rx.shape_logits(z, out=out)
                    else:
                        with pytest.raises(ValueError, match="overlap"):
                            rx.shape_logits(z, out=out)
    assert len(verdicts) == 4
