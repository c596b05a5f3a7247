"""Inputs of the projection that the launch just before the call writes."""
import pytest
import torch

import bit_grouped_gemm_gb300 as bg
from tests.test_gpu_operators import Linear, built  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,N", [(4, 512, 264), (40, 2048, 1000), (300, 1024, 520), (4096, 256, 264)])
def test_ids_and_rows_made_by_the_launch_before(T, K, N):
    """Request ids and their rows change from call to call and are written by the
    last launches before each; every call's output is that of its own inputs."""
    c = Linear(T, K, N, x="e4m3", rank=16, n=9)
    h = bg.moe_linear_create(bg.linear_desc(K, N, T, 16), 0)
    w = bg.w4(*c.w)
    steps = 12
    ids = [(c.ids + 1 + 3 * i) % 10 - 1 for i in range(steps)]        # -1 .. 8, moved on each call
    scales = [c.xs * (1.0 + 0.25 * i) for i in range(steps)]
    want = []
    for i in range(steps):
        c.ids, c.xs = ids[i].to(torch.int32), scales[i]
        assert c.run(handle=h) == 0
        c.compare()
        want.append(c.y.clone())
    live, xs, out = torch.full_like(c.ids, -1), torch.zeros_like(c.xs), [torch.zeros_like(c.y) for _ in want]
    for order in (0, 1):
        for i in range(steps):
            # the ids last, then the scales last
            if order:
                live.copy_(ids[i])
            torch.mul(c.xs, 0.0, out=xs)
            torch.add(xs, scales[i], out=xs)
            if not order:
                live.copy_(ids[i])
            bg.moe_linear_forward(h, c.x, T, w, out[i], x_scale=xs, lora=c.lora, adapter=live)
        torch.cuda.synchronize()
        assert bg.moe_linear_get_error(h) == 0
        for i in range(steps):
            assert torch.equal(out[i], want[i]), (order, i)
            out[i].zero_()
    bg.moe_linear_destroy(h)
