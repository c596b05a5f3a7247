"""Batches in which few tokens have an adapter: tiles of the product without any
adapter stage lie between tiles with some, and short K makes each tile brief."""
import pytest
import torch

import bit_grouped_gemm_gb300 as bg
from tests.test_gpu_operators import Linear, built, gen  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,N,rank,n", [
    (4093, 64, 2530, 8, 3), (3551, 64, 2976, 8, 3), (4096, 64, 4096, 16, 2), (9000, 64, 4100, 8, 5),
    (4096, 128, 2048, 24, 1), (12000, 192, 1024, 16, 3), (2500, 64, 16400, 40, 3)])
@pytest.mark.parametrize("ids", ["mixed", "none", "one", "few", "runs", "blocks"])
def test_tiles_with_and_without_adapters(T, K, N, rank, n, ids):
    """Every call ends without a wait that ran out, with the first call's bits."""
    c = Linear(T, K, N, rank=rank, n=n, ids="runs" if ids == "runs" else "mixed")
    g, at = gen(7), torch.arange(T, device="cuda")
    if ids in ("none", "one", "few"):
        c.ids.fill_(-1)
    if ids == "one":
        c.ids[T // 2] = 0
    if ids == "few":
        some = torch.randperm(T, generator=g, device="cuda")[:9]
        c.ids[some] = torch.randint(0, n, (9,), generator=g, device="cuda").int()
    if ids == "blocks":
        c.ids.copy_(torch.where((at // 300) % 3 == 0, (at // 900) % n, -1))
    h = bg.moe_linear_create(bg.linear_desc(K, N, T, rank), 0)
    assert c.run(handle=h) == 0
    c.compare()
    first, w = c.y.clone(), bg.w4(*c.w)
    for _ in range(40):
        bg.moe_linear_forward(h, c.x, T, w, c.y, lora=c.lora, adapter=c.ids)
    torch.cuda.synchronize()
    assert bg.moe_linear_get_error(h) == 0
    assert torch.equal(c.y, first)
    bg.moe_linear_destroy(h)
