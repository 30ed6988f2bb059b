"""fp8_expert_route with a bias that is not finite: -Inf and NaN switch an expert off for the choice (its score still
counts in a softmax's sum), +Inf puts it before all finite keys.  Choices and plan exactly, weights within the bound of
expert_ref.route."""
import math

import pytest
import torch

import expert_ref as ref
from test_gpu_expert_route import check, logits_of, run

pytestmark = pytest.mark.gpu

OFF = (-math.inf, math.nan)


@pytest.fixture(scope="module")
def rt():
    import dynamic_scaling_scaled_amd as rt

    rt.lib()
    return rt


@pytest.mark.parametrize("off", OFF)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_four_experts_two_off(rt, off, score):
    """As many choices as experts: the two that are on, in order, and two empty places."""
    x = torch.tensor([[1.0, 0.5, 0.2, -0.3]]).cuda()
    o = run(rt, x, 4, score=score, bias=torch.tensor([0.0, 0.0, off, off]).cuda())
    assert o["ids"].tolist() == [[0, 1, -1, -1]] and o["slots"].tolist() == [[0, 1, -1, -1]]
    assert o["offsets"].tolist() == [0, 1, 2, 2, 2] and o["order"].tolist() == [0, 1, -7, -7]
    assert o["weights"][0, 2:].tolist() == [0.0, 0.0]


@pytest.mark.parametrize("off", OFF)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("experts,k", [(8, 8), (24, 6), (64, 6), (128, 8), (256, 16), (500, 8), (1024, 32)])
def test_switched_off(rt, off, score, renorm, experts, k):
    """None, one, most and all experts off, beside absent logits; fewer than k, k and k + 1 that are left."""
    for tokens, left in ((1, experts - 1), (17, k + 1), (70, k), (33, max(1, k - 2)), (5, 1), (3, 0)):
        g = torch.Generator().manual_seed(experts + left)
        bias = 0.1 * torch.randn(experts, generator=g)
        bias[torch.randperm(experts, generator=g)[left:]] = off
        x = logits_of(tokens, experts, seed=left)
        check(rt, x, k, bias=bias.cuda(), score=score, renorm=renorm)
        x[tokens // 2, ::3] = -math.inf
        x[0, 1::4] = math.nan
        check(rt, x, k, bias=bias.cuda(), score=score, renorm=renorm)


@pytest.mark.parametrize("off", OFF)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top", [(4, 1), (4, 3), (5, 2), (16, 7)])
@pytest.mark.parametrize("best", [1, 2])
def test_switched_off_in_groups(rt, off, score, groups, top, best):
    """Experts that are off count in no group's score: groups with all, all but one and none of theirs off."""
    experts, n = 80, 80 // groups
    bias = 0.1 * torch.randn(experts, generator=torch.Generator().manual_seed(groups))
    bias[:n] = off
    bias[n + 1:2 * n] = off
    bias[2 * n::3] = off
    for tokens in (3, 70, 300):
        check(rt, logits_of(tokens, experts, seed=top), min(6, n * top), bias=bias.cuda(), score=score, groups=groups,
              top=top, best=best)
    bias[:] = off
    check(rt, logits_of(9, experts), min(6, n * top), bias=bias.cuda(), score=score, groups=groups, top=top, best=best)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,best", [(1, 1), (4, 1), (4, 2)])
def test_always_chosen(rt, score, groups, best):
    """+Inf, alone and several (ties to the lower expert), beside experts that are off."""
    for first in ((5,), (5, 6, 17, 40, 41, 42)):
        bias = 0.1 * torch.randn(64, generator=torch.Generator().manual_seed(3))
        bias[list(first)] = math.inf
        bias[::4] = -math.inf
        bias[1::16] = math.nan
        check(rt, logits_of(70, 64), 5, bias=bias.cuda(), score=score, groups=groups, top=max(1, groups // 2), best=best)


def test_ties_beside_experts_that_are_off(rt):
    """Equal keys go to the lower expert, empty places stay behind them."""
    x = torch.zeros(66, 16).cuda()
    x[1::2, 3:9] = 1.0
    bias = torch.zeros(16)
    bias[2:15:2] = -math.inf
    bias[1] = math.nan
    for k in (3, 8, 12, 16):
        for score in ("softmax", "sigmoid"):
            check(rt, x, k, bias=bias.cuda(), score=score)


def test_many_tokens(rt):
    """The plan of several blocks of tokens, each expert at most once a token."""
    for off in OFF:
        bias = torch.zeros(64)
        bias[5:] = off
        o = run(rt, logits_of(9000, 64), 6, score="sigmoid", bias=bias.cuda())
        ids = o["ids"].cpu()
        assert bool((ids[:, 5] == -1).all()) and torch.equal(ids[:, :5].sort(1).values, torch.arange(5, dtype=torch.int32).expand(9000, 5))
        slots, order, offsets = ref.plan(ids, 64)
        assert torch.equal(o["slots"].cpu(), slots) and torch.equal(o["offsets"].cpu(), offsets)
        assert torch.equal(o["order"].cpu()[:len(order)], order) and bool((o["order"][len(order):] == -7).all())
