"""What the adapters add: entries that are no numbers."""
import pytest
import torch

from tests.test_gpu_operators import Linear, built  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [6, 40, 300, 2500])
@pytest.mark.parametrize("ids", ["mixed", "runs"])
def test_broken_entries_show_in_their_own_outputs(T, ids):
    """An infinity or a NaN in B shows in the outputs that it feeds, whatever the
    batch: no ordinary number stands there. All other outputs keep their bits."""
    clean = Linear(T, 256, 200, rank=16, n=4, ids=ids)
    assert clean.run() == 0
    c = Linear(T, 256, 200, rank=16, n=4, ids=ids)
    c.b[1, 5, 3], c.b[1, 77, 0], c.b[1, 150] = float("nan"), float("inf"), float("-inf")
    c.b[2, 9, 15] = float("-inf")
    c.run()
    fed = torch.zeros_like(c.y, dtype=torch.bool)
    for n, cols in ((1, (5, 77, 150)), (2, (9,))):
        for col in cols:
            fed[c.ids == n, col] = True
    assert fed.any() and torch.equal(c.y[~fed], clean.y[~fed])
    y = c.y[fed].float()
    assert (~y.isfinite() | (y.abs() > 1e30)).all()
