"""Row counts at the end of the norm's range."""
import pytest
import torch

import bit_grouped_gemm_gb300 as bg
from tests.test_gpu_operators import built, check_norm, gen, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [(1 << 31) - 1, (1 << 31) - 5000])
def test_norm_of_as_many_rows_as_an_int_counts(T):
    """The walk over the rows steps past 2^31 here. 60 GB; the first and the
    last rows are checked, and that nothing past them is written."""
    H, n, past = 8, 64, 4096
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    g = gen(3)
    for s in (slice(0, n), slice(T - n, T)):
        x[s] = randn(g, n, H)
    q = torch.full((T + past, H), 77, dtype=torch.uint8, device="cuda")
    qs = torch.full((T + past, 1), -1.0, device="cuda")
    bg.moe_norm_quant(bg.norm_desc(H), x, None, None, T, q_out=q, q_scale=qs)
    torch.cuda.synchronize()
    for s in (slice(0, n), slice(T - n, T)):
        xs = x[s].double()
        v = xs / ((xs ** 2).mean(1, keepdim=True) + 1e-6).sqrt()
        codes = q[s].view(torch.float8_e4m3fn)
        check_norm(dict(x=xs, d=None, w=None, xo=xs, xn=v.bfloat16().double(),
                        q=codes.float().double(), qs=qs[s].double(), alpha=1.0, eps=1e-6), H, False)
    assert int((qs[n:T - n] != 0).sum()) == 0 and int((q[n:T - n] != 0).sum()) == 0
    assert (qs[T:] == -1.0).all() and (q[T:] == 77).all()
    del x, q, qs
    torch.cuda.empty_cache()
