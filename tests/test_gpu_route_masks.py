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
