"""Scores that lie 3e-10 to 1e-8 apart: too close for 32 bits, for the pairs of
floats of the second look not. Few experts (or groups) of a row are in doubt, so
that this look decides."""
import numpy as np
import pytest
import torch

from tests.test_gpu_operators import built, check_route  # noqa: F401

pytestmark = pytest.mark.gpu
E = 512


def steps(rng, n):
    """n numbers in a random order, neighbours 3e-10 to 1e-8 apart."""
    s = np.cumsum(np.exp(rng.uniform(np.log(3e-10), np.log(1e-8), n)))
    return rng.permutation(s - s[n // 2])


def logit(p):
    return np.log(p / (1 - p))


def run(logits, bias, k, **kw):
    check_route(torch.from_numpy(logits).cuda(), logits.shape[1], k,
                bias=torch.from_numpy(bias).cuda(), **kw)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("k", [1, 8])
def test_close_sigmoid_scores(seed, k):
    rng = np.random.default_rng(seed)
    sets, at = [], 0
    while at < E:
        n = min(int(rng.integers(2, 21)), E - at)
        sets.append(np.arange(at, at + n))
        at += n
    bias = np.zeros(E, np.float32)
    logits = (-20.0 + rng.standard_normal((len(sets), E))).astype(np.float32)
    for t, s in enumerate(sets):
        base = 1 / (1 + np.exp(-rng.uniform(-5, 6)))
        want = base + steps(rng, len(s))
        # the score from a logit that is off by up to 2^-9 of it, the rest by the bias
        off = 0.03 * base * (1 - base) * rng.uniform(-1, 1, len(s))
        l = logit(want + off).astype(np.float32)
        logits[t, s] = l
        bias[s] = want - 1 / (1 + np.exp(-l.astype(np.float64)))
    run(logits, bias, k, score="sigmoid")


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("k", [1, 8])
@pytest.mark.parametrize("renorm", [False, True])
def test_close_softmax_scores(seed, k, renorm):
    rng = np.random.default_rng(seed)
    sets, at = [], 1                     # (expert 0 is the row's largest, never chosen)
    while at < E:
        n = min(int(rng.integers(2, 21)), E - at)
        sets.append(np.arange(at, at + n))
        at += n
    bias = np.zeros(E, np.float32)
    bias[0] = -2.0
    logits = (-14.0 + rng.standard_normal((len(sets), E))).astype(np.float32)
    for t, s in enumerate(sets):
        logits[t, 0] = rng.uniform(0, 5)
        logits[t, s] = 0.02 * rng.standard_normal(len(s))
        l = logits[t].astype(np.float64)
        p = np.exp(l - l.max()) / np.exp(l - l.max()).sum()
        bias[s] = p[s].mean() + steps(rng, len(s)) - p[s]
    run(logits, bias, k, score="softmax", renorm=renorm)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("topk_groups,k", [(8, 8), (3, 4)])
def test_close_sums_of_groups(seed, topk_groups, k):
    """32 groups of 16 experts; a row's scores come from one pair per group, and
    2 to 14 groups around the last one kept have close sums."""
    rng = np.random.default_rng(seed)
    groups, size = 32, 16
    bias = np.zeros(E, np.float32)
    logits = (-20.0 + rng.standard_normal((size // 2, E))).astype(np.float32)
    for t in range(size // 2):
        doubt = int(rng.integers(2, 15))
        above = topk_groups - int(rng.integers(1, min(doubt, topk_groups + 1)))
        total = np.empty(groups)
        order = rng.permutation(groups)
        total[order[:above]] = 1.3 + 0.01 * np.arange(above)
        total[order[above:above + doubt]] = 1.2 + steps(rng, doubt)
        total[order[above + doubt:]] = 1.1 - 0.01 * np.arange(groups - above - doubt)
        for g in range(groups):
            a = rng.uniform(0.3, 0.5) * total[g]
            for e, want in ((g * size + 2 * t, a), (g * size + 2 * t + 1, total[g] - a)):
                l = np.float32(logit(want + 2e-3 * rng.uniform(-1, 1)))
                logits[t, e] = l
                bias[e] = want - 1 / (1 + np.exp(-np.float64(l)))
    run(logits, bias, k, score="sigmoid", groups=groups, topk_groups=topk_groups)
