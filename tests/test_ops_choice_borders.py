"""The router where 32 bits cannot tell its scores apart, or hold them: groups whose
two best nearly cancel, sums beyond float32, a softmax over an infinite logit.  The
choice is that of the plain 64-bit form, bit for bit."""
import numpy as np
import pytest
import torch

import ops_reference as ref
import ops_reference8 as ref8
from test_ops_choice import check, ops  # noqa: F401
from test_ops_routes import DT

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


# A softmax over +infinity has no scores.  The token's weights say so, all NaN, and
# its experts are those of the logits' own order: as without a bias, groups by their
# best.  Closed experts stay closed.
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("biased,groups,top,best", [(True, 1, 1, 1), (False, 8, 3, 2), (True, 8, 3, 1), (True, 8, 3, 2), (False, 8, 3, 1), (False, 1, 1, 1)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_an_infinite_logit_keeps_its_experts(ops, dtype, biased, groups, top, best, renormalize):
    g = torch.Generator().manual_seed(3)
    T, E, k = 12, 64, 6
    logits = torch.randn((T, E), generator=g).to(DT[dtype])
    bias = torch.randn(E, generator=g).cuda() if biased else None
    if biased:
        bias[50] = -float("inf")
    how = dict(bias=bias, groups=groups, top_groups=top, group_best=best, renormalize=renormalize)
    clean = ops.expert_route(logits.cuda(), k, **how)
    logits[2, 37] = logits[5, 11] = logits[5, 60] = logits[7, 0] = logits[9, 50] = float("inf")
    logits[7, 1:] = -float("inf")
    logits[9, ::3] = -float("inf")
    hit = [2, 5, 7, 9]
    r = ops.expert_route(logits.cuda(), k, **how)
    l = ref.f64(logits)
    if biased:
        l[:, 50] = -np.inf
    else:
        assert r.ids[9, 0] == 50
    with np.errstate(invalid="ignore"):
        want, _ = ref8.route(l[hit], k, "softmax", None, groups, top, 1, True, 1.0)
    np.testing.assert_array_equal(r.ids[hit].cpu().numpy(), want)
    assert r.ids[2, 0] == 37 and r.ids[5, :2].tolist() == [11, 60] and r.ids[7].tolist() == [0] + [-1] * (k - 1)
    assert torch.isnan(r.weights[2]).all() and torch.isnan(r.weights[5]).all() and torch.isnan(r.weights[9]).all() and torch.isnan(r.weights[7, 0])
    others = [t for t in range(T) if t not in hit]
    assert torch.equal(r.ids[others], clean.ids[others]) and torch.equal(r.weights[others], clean.weights[others])
    # and so its rows go where the logits say, and show that they have no weights
    plan = ops.expert_sort(r.ids, E)
    y = ops.combine(torch.ones((T * k, 8), device="cuda"), r.weights, plan)
    assert torch.isnan(y[hit]).all() and torch.isfinite(y[others]).all()
