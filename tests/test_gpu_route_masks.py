"""Masked experts among groups, and chosen ones whose probability is zero."""
import numpy as np
import pytest
import torch

from tests.test_gpu_operators import built, check_route, gen, randn  # noqa: F401

pytestmark = pytest.mark.gpu
LOW = torch.finfo(torch.float32).min


@pytest.mark.parametrize("E,groups,tg,k", [(8, 4, 3, 3), (40, 8, 7, 22), (256, 8, 4, 8), (480, 6, 5, 26),
                                           (512, 32, 9, 10), (32, 32, 7, 5), (96, 4, 2, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("mask", [float("-inf"), float("nan"), LOW])
@pytest.mark.parametrize("biased", [False, True])
def test_groups_with_few_open_experts(E, groups, tg, k, score, mask, biased):
    """Groups keep no, one or more unmasked experts, with logits so far apart that
    the groups' order is beyond 32 bits."""
    g = gen(E + k)
    T = 200
    logits = 20.0 * randn(g, T, E)
    keep = torch.rand(T, 1, generator=g, device="cuda") * 0.5
    logits[torch.rand(T, E, generator=g, device="cuda") > keep] = mask
    # exactly one open expert in every group
    first = torch.randint(0, E // groups, (40, groups, 1), generator=g, device="cuda")
    one = torch.full((40, groups, E // groups), mask, device="cuda")
    one.scatter_(2, first, 20.0 * torch.randn(40, groups, 1, generator=g, device="cuda"))
    logits[:40] = one.view(40, E)
    bias = 1e-9 * randn(g, E) if biased else None
    check_route(logits, E, k, bias=bias, score=score, groups=groups, topk_groups=tg)


@pytest.mark.parametrize("E,k,groups,tg", [(464, 1, 1, 1), (344, 29, 1, 1), (440, 13, 11, 5), (56, 6, 2, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("mask", [LOW, -1e30, -2000.0, float("-inf")])
@pytest.mark.parametrize("renorm", [False, True])
def test_chosen_experts_of_no_probability(E, k, groups, tg, score, mask, renorm):
    """The bias makes a row choose masked experts, whose p is 0: so are the
    weights, also where all of a row's choice is masked."""
    g = gen(E)
    T = 60
    logits, bias = randn(g, T, E), 0.1 * randn(g, E)
    shut = torch.arange(E, device="cuda") % 2 == 0
    bias[shut] += 5.0
    logits[:, shut] = mask
    logits[20:40, shut & (torch.arange(E, device="cuda") % 8 == 0)] = 1.0    # some of the favoured are open
    logits[50:] = mask                                                     # nothing else is open
    got = check_route(logits, E, k, bias=bias, score=score, groups=groups, topk_groups=tg, renorm=renorm)
    assert (got["topk_w"][:20] == 0).all()


@pytest.mark.parametrize("E,k", [(8, 1), (24, 5), (64, 3), (256, 8), (512, 10)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("level", [0.0, 0.25, 1.75])
def test_equal_scores_before_a_slightly_larger_one(E, k, score, level):
    """Many masked experts share one score (the bias alone), and one or two others,
    often behind them in index order, lie above it by less than the second look
    can tell: those are chosen first."""
    g = gen(E + k)
    T = 200
    logits = torch.full((T, E), float("-inf"), device="cuda")
    # clear winners for some of the k places, then those barely above
    top = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k + 1] for _ in range(T)])
    clear = torch.randint(0, k, (T, 1), generator=g, device="cuda")
    place = torch.arange(k + 1, device="cuda")
    faint = -28.0 - 6.0 * torch.rand(T, k + 1, generator=g, device="cuda")
    vals = torch.where(place < clear, 2.0 + 0.1 * place, torch.where(place <= clear + 1, faint, float("-inf")))
    logits.scatter_(1, top, vals)
    if score == "softmax":      # a row's sum of about one, from an expert that the bias keeps out
        logits[:, 0] = 4.0
    bias = torch.full((E,), level, device="cuda")
    bias[0] = -3.0
    check_route(logits, E, k, bias=bias, score=score)


@pytest.mark.parametrize("best", [5.0, 0.0, -15.0, -19.9, -20.0, -25.0, -39.0, -41.0, -300.0])
@pytest.mark.parametrize("down", [3.0, 30.0, 49.5, 60.0])
def test_renormalised_weights_far_below_the_largest(best, down):
    """A chosen sigmoid e^-60 of the largest still has its weight, to FP32's
    roundings (its argument's too), wherever the largest lies."""
    T, E, k = 40, 64, 6
    g = gen(3)
    logits = best - down * torch.rand(T, E, generator=g, device="cuda")
    logits[:, 5], logits[:, 9] = best, best - down
    logits[:, 10:] = best - down - 1.0 - torch.rand(T, E - 10, generator=g, device="cuda")
    bias = torch.zeros(E, device="cuda")
    bias[[5, 9, 20, 30, 40, 50]] = 2.0
    got = check_route(logits, E, k, bias=bias, score="sigmoid", renorm=True)
    assert (got["topk_w"] > 0).all()
