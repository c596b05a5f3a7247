"""Projections of many input features with adapters, from one token to prompts."""
import pytest

from tests.test_gpu_operators import Linear, built  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [13056, 13120, 14336, 16384])
@pytest.mark.parametrize("rank", [8, 128])
@pytest.mark.parametrize("T", [5, 40, 300])
def test_linear_of_many_features(T, rank, K):
    Linear(T, K, 264, rank=rank, n=5).check()
    Linear(T, K, 200, x="e4m3", rank=rank, n=5, ids="runs", x_pad=16, y_pad=3).check()


@pytest.mark.parametrize("K,rank", [(13952, 16), (14016, 16), (13824, 32), (13568, 64), (16320, 24)])
def test_linear_around_the_token_tiles_limit(K, rank):
    Linear(700, K, 136, rank=rank, n=40).check()


def test_linear_of_many_features_orders_mixed_tokens():
    Linear(2300, 14336, 72, x="e4m3", rank=16, n=300).check()
