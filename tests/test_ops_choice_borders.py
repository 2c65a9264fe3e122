"""The router where 32 bits cannot tell its scores apart, or hold them: groups whose
two best nearly cancel, sums beyond float32.  The choice is that of the plain 64-bit
form, bit for bit."""
import pytest
import torch

from test_ops_choice import check, ops  # noqa: F401

pytestmark = pytest.mark.gpu


def logits_of(score, scoring):
    return torch.log(score / (1.0 - score)) if scoring == "sigmoid" else torch.log(score)


# A group of two whose biases are +b and -b: each of c = s + b and c = s - b is
# rounded by up to 2^-24 b, of which their sum, some 1, shows nothing.  Sums lie
# within a few roundings of one another.
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("big", [4.0, 64.0, 1000.0])
@pytest.mark.parametrize("groups,top", [(32, 16), (8, 3), (2, 1)])
def test_groups_whose_best_two_cancel(ops, scoring, big, groups, top):
    g = torch.Generator().manual_seed(int(big) + groups)
    T, whole = 300, 1.0 if scoring == "sigmoid" else 1.0 / groups
    part = 0.2 + 0.6 * torch.rand((T, groups), generator=g, dtype=torch.float64)
    noise = big * 2.0 ** -23 * torch.randn((T, groups), generator=g, dtype=torch.float64)
    score = torch.stack((part, 1.0 - part), 2) * whole
    score[..., 1] += noise
    logits = logits_of(score, scoring).reshape(T, -1).float().cuda()
    bias = torch.tensor([big, -big]).repeat(groups).cuda()
    for k in (1, top):
        check(ops, logits, k, scoring, bias, groups, top, 2)
    # a group of great terms beside groups of small ones, which are told apart as
    # finely as without it
    bias = torch.where(torch.arange(2 * groups) < 2, bias.cpu(), 0.25).cuda()
    check(ops, logits, top, scoring, bias, groups, top, 2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_sums_of_groups_beyond_float32(ops, scoring, sign):
    g = torch.Generator().manual_seed(12)
    logits = torch.randn((50, 32), generator=g).cuda()
    # two a group, 2e38 to 3.2e38 each, the best groups not the first ones
    size = 2.0e38 + 1.2e38 * ((torch.arange(16) * 7 % 16) / 16)
    bias = (sign * size).repeat_interleave(2).float().cuda()
    r = check(ops, logits, 4, scoring, bias, 16, 3, 2)
    want = torch.argsort(sign * size, descending=True)[:3]
    assert set(torch.unique(r.ids // 2).tolist()) <= set(want.tolist())
