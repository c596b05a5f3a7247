"""Calls of the rotary store whose output would overwrite what other threads still read: refused
before the launch, so that their addresses are never used."""
import ctypes

import pytest

import bit_grouped_gemm_gb300 as bg
from bit_grouped_gemm_gb300 import binding

pytestmark = pytest.mark.gpu
A, FAR = 1 << 30, 1 << 36


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_grouped_gemm_gb300 import build
    build.build()


@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (4, 4)])
@pytest.mark.parametrize("same", ["k", "v", "k v", "slot", "position", "k slot"])
def test_in_place_is_for_the_queries_alone(heads, kv_heads, same):
    """q_out = q, and another input at the same address."""
    lib = binding.load_library()
    q = A + 4 * FAR
    at = {n: A + (5 + i) * FAR for i, n in enumerate(("k", "v", "position", "slot"))}
    at.update({n: q for n in same.split()})
    cache = bg.MoeKvCache(A, A + FAR, None, None, 10)
    a = bg.moe_attn_create(bg.attn_desc(heads, kv_heads, 64, 16, max_tokens=32, max_requests=4), 0)
    try:
        assert lib.moe_rope_store(a, q, 0, at["k"], 0, at["v"], 0, 4, at["position"], at["slot"], q, 0,
                                  ctypes.byref(cache), None) == 1
    finally:
        bg.moe_attn_destroy(a)
