"""What the adapters add: the bits of x A^T, and entries that are no numbers."""
import pytest
import torch

from tests.test_gpu_operators import Linear, built, gen  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,N,rank", [
    (1, 2048, 264, 16), (20, 1024, 200, 24), (128, 2048, 2048, 16), (200, 4096, 1000, 16), (257, 2048, 1032, 8),
    (512, 2048, 2048, 24), (1500, 320, 201, 40), (2500, 512, 520, 128), (4096, 2048, 2048, 8)])
@pytest.mark.parametrize("ids", ["mixed", "runs"])
def test_16_bits_of_x_a(T, K, N, rank, ids):
    """Rows and A of small integers, W of zeros: x A^T are integers below 2^16,
    which 16 significant bits hold, and y their small differences, so every step
    is exact. Kept to the 8 bits of one bf16, x A^T would be off by up to 64."""
    c = Linear(T, K, N, rank=rank, n=5, ids=ids, lscale=False)
    g = gen(1)
    ints = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g, device="cuda")
    for t in c.w[1:]:
        t.zero_()
    c.x.copy_(ints(0, 3, T, K))
    a = ints(0, 7, 5, rank, K)
    # rows 2j and 2j + 1 of A differ in three places
    a[:, 1::2] = a[:, ::2]
    for _ in range(3):
        a[:, 1::2].scatter_(2, ints(0, K, 5, rank // 2, 1), ints(0, 7, 5, rank // 2, 1))
    # every output takes the differences of one pair or two
    b = torch.zeros(5, N, rank // 2, dtype=torch.int64, device="cuda")
    for _ in range(2):
        b.scatter_(2, ints(0, rank // 2, 5, N, 1), 1)
    c.a.copy_(a)
    c.b[:, :, ::2], c.b[:, :, 1::2] = b, -b
    assert c.run() == 0
    h = c.x.double() @ c.a.double().reshape(-1, K).T
    assert 256 < float(h.max()) < 2 ** 16
    want = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for i in range(5):
        rows = c.ids == i
        want[rows] = h[rows, i * rank:(i + 1) * rank] @ c.b[i].double().T
    assert float(want.abs().max()) <= 256
    assert (want != 0).any() or not ((c.ids >= 0) & (c.ids < 5)).any()
    assert torch.equal(c.y.double(), want)


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
