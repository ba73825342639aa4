"""The router's choice where group scores are hard to tell apart, against the
formulas in 64 bits, with the bounds of test_gpu_routing.py."""
import pytest
import torch

from test_gpu_routing import _check, _rand, _scores

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.mark.parametrize("most", [1e3, 1e5, 1e6])
@pytest.mark.parametrize("size", [2, 4])
@pytest.mark.parametrize("where", ["all", "half", "off"])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_group_sums_that_cancel(most, size, where, scores):
    """Biases of +most and -most in every group, in every other one, or in all but
    two whose experts all have -most: the sum of a group's two best choices is some
    2^-24 of them or less, which fp32 choices do not hold.  Rows with two sums or two
    choices nearer than both sides' arithmetic are left out: it is exact to 2^-44 of
    the terms in the kernel and 2^-53 in 64 bits, 2^-42 in all."""
    T, groups, kept = 20000, 8, 3
    E = groups * size
    bias = torch.full((groups, size), -most)
    bias[:, 1] = most
    if where == "half":
        bias[::2] = 0.0
    if where == "off":
        bias[:2] = -most
    bias = bias.flatten()
    logits = _rand((T, E), F32, E, 2.0)
    c = _scores(logits, scores) + bias.double()
    sums = c.view(T, groups, size).topk(2, 2).values.sum(2)
    best = sums.sort(dim=1, descending=True)
    keep = torch.zeros((T, groups), dtype=torch.bool).scatter_(1, best.indices[:, :kept], True)
    left = c.masked_fill(~keep.repeat_interleave(size, 1), -float("inf"))
    left = left.sort(dim=1, descending=True).values
    near = 2.0 ** -42 * most
    ok = (best.values[:, kept - 1] - best.values[:, kept] > near) & (
        (left[:, :kept] - left[:, 1:kept + 1]).amin(1) > near)
    assert int(ok.sum()) > 0.9 * T
    _check(logits[ok], kept, scores, bias, groups, kept, "top2", True, 2.5)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,topk_groups", [(1023, 3, 2), (771, 3, 1), (768, 3, 2),
                                                  (640, 5, 3), (645, 5, 3), (576, 9, 4),
                                                  (585, 9, 4), (544, 17, 5), (1020, 17, 5)])
@pytest.mark.parametrize("biased", [False, True])
def test_groups_on_both_sides_of_their_lanes(scores, E, groups, topk_groups, biased):
    """Three groups of 256 experts have their own lanes of a warp, of 257 to 341 not; five
    of 128, nine of 64 and seventeen of 32, but not of more."""
    bias = _rand((E,), F32, 9, 0.1) if biased else None
    for by in ("top2", "max"):
        _check(_rand((37, E), F32, E, 2.0), 8, scores, bias, groups, topk_groups, by)
