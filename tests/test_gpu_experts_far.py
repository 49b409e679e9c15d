"""The choice of experts at its ends.  Where scores leave the normal range of 64 bits: far
below zero (sigmoid) or far below the largest logit (softmax) they differ by
powers of two down to 2^-1074, and the order is that of the numbers there too."""

import math

import pytest
import torch

import expert_ref as R
from nf4_bit_weight_amd import nf4_route

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


def check_choice(logits, k, **how):
    r = nf4_route(logits.to(DEV), k, **{n: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for n, v in how.items()})
    w, e = R.route(logits, k, **how)
    assert torch.equal(r.experts.cpu(), e), how
    return r, w


# Logits around the ends: e^-708.4 is the last normal number, e^-745.1 the last above zero.
FAR = [(-709.0, -701.0, -705.0), (-700.0, -699.0, -699.5), (-730.0, -709.0, -720.0), (-744.0, -742.0, -743.0), (-1000.0, -744.0, -745.0)]


@pytest.mark.parametrize("E", [8, 64, 300, 1000])
@pytest.mark.parametrize("others,best,second", FAR)
def test_far_scores_keep_their_order_under_a_bias(E, others, best, second):
    l = torch.full((3, E), others)
    l[:, 5], l[:, 6] = best, second
    l[1] = l[1].flip(0)
    zero = torch.zeros(E)
    check_choice(l, 2, score="sigmoid", bias=zero)
    check_choice(l, 2, score="sigmoid", bias=zero, renormalize=True)
    l[:, 7] = 0.0                                               # the largest, from which softmax counts
    check_choice(l, 3, bias=zero)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(64, 8), (60, 4), (256, 8)])
def test_far_groups_keep_their_order(score, E, groups):
    """Ranked by their best two, without a bias: 1 + 2 against 0 + 2 units of e^-720."""
    size = E // groups
    l = torch.full((4, E), -800.0)
    for g in range(groups):
        l[0, g * size: g * size + 2] = -738.0 + 3.0 * g         # the last group is the best
        l[1, g * size] = -705.0 - 2.0 * abs(g - 2)
    l[2] = l[0].flip(0)
    l[3, ::size] = torch.linspace(-740.0, -702.0, groups)
    if score == "softmax":
        l[:, 1] = 0.0
    check_choice(l, 4, score=score, groups=groups, top_groups=2, group_score="top2")
    check_choice(l, 4, score=score, groups=groups, top_groups=2, group_score="top2", bias=torch.zeros(E))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [16, 64, 512])
def test_far_scores_at_random(score, E):
    l = -690.0 - 70.0 * torch.rand((40, E), generator=torch.Generator().manual_seed(E))
    if score == "softmax":
        l[:, E // 3] = 0.0
    check_choice(l, 8, score=score, bias=torch.zeros(E))
    check_choice(l, 8, score=score, groups=4, top_groups=2, group_score="top2")


def test_far_above_zero_scores_are_one():
    """Saturated scores are equal in 64 bits: the lower index is taken, as of other equal ones."""
    l = torch.tensor([[40.0, 800.0, 60.0, 3e38, 37.0, -1.0, 700.0, 710.0]])
    r, _ = check_choice(l, 4, score="sigmoid", bias=torch.zeros(8))
    assert r.experts.tolist() == [[0, 1, 2, 3]] and r.weights.tolist() == [[1.0] * 4]


def test_scores_around_zero_keep_their_order_under_a_bias():
    """Neighbouring fp32 logits on either side of zero, where the two forms of the sigmoid meet."""
    E = 64
    l = torch.zeros(2, E)
    step = torch.arange(E // 2, dtype=torch.float32) * 2.0 ** -24
    l[0, ::2], l[0, 1::2] = -step, step
    l[1] = torch.linspace(-1e-3, 1e-3, E)
    check_choice(l, 40, score="sigmoid", bias=torch.zeros(E))
    check_choice(l, 40, score="sigmoid", bias=torch.full((E,), 0.125))
    assert math.exp(-745.0) > 0.0                                # what the plain form counts on


def test_plan_of_more_runs_than_workgroups():
    """Groups of odd size take runs of four tokens; above 2^21 of those a workgroup places several."""
    T, E = (1 << 23) + 5, 260
    l = torch.randn((T, E), device=DEV, dtype=torch.bfloat16, generator=torch.Generator(DEV).manual_seed(5))
    l[::1000] = -math.inf
    r = nf4_route(l, 1, groups=13, top_groups=2)
    best = torch.where(torch.isinf(l[:, 0]), -1, l.argmax(-1)).int()
    assert torch.equal(torch.where(r.experts[:, 0] >= 0, l.gather(1, r.experts.clamp(min=0).long())[:, 0], 0), torch.where(best >= 0, l.amax(-1), 0))
    assert torch.equal(r.experts[:, 0] < 0, best < 0)
    key = torch.where(r.experts[:, 0] < 0, E, r.experts[:, 0]).long()
    order, count = key.sort(stable=True).indices, torch.bincount(key, minlength=E + 1)
    assert torch.equal(r.offsets[1:].long(), count[:E].cumsum(0)) and int(r.offsets[0]) == 0
    used = int(r.offsets[-1])
    assert torch.equal(r.tokens[:used].long(), order[:used]) and bool((r.tokens[used:] == -1).all())
    slots = torch.full((T,), -1, device=DEV, dtype=torch.long)
    slots[order[:used]] = torch.arange(used, device=DEV)
    assert torch.equal(r.slots[:, 0].long(), slots)
