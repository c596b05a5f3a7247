"""Refusals of the operators around the expert block: every wrong argument is
found on the host, before any CUDA call, so these run without a GPU. Addresses
are made up and never read."""
import ctypes

import pytest

import bit_grouped_gemm_gb300 as bg
from bit_grouped_gemm_gb300 import binding

INVALID, UNSUPPORTED, CAPACITY = 1, 2, 4
A = 1 << 30            # an aligned address, and others far from it
FAR = 1 << 33


@pytest.fixture(scope="module")
def lib():
    from bit_grouped_gemm_gb300 import build
    build.build()
    return binding.load_library()


def norm_call(lib, T=4, x=A, delta=A + FAR, w=A + 2 * FAR, xo=A + 3 * FAR, xn=A + 4 * FAR,
              q=A + 5 * FAR, qs=A + 6 * FAR, hidden=2048, **desc):
    d = bg.norm_desc(hidden, **desc)
    return lib.moe_norm_quant(ctypes.byref(d), x, delta, w, T, xo, xn, q, qs, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), INVALID), (dict(x=None), INVALID), (dict(hidden=0), INVALID),
    (dict(hidden=12), INVALID), (dict(hidden=16392), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(alpha=float("nan")), INVALID),
    (dict(alpha=float("inf")), INVALID), (dict(quant_group=64), INVALID),
    (dict(x_stride=2040), INVALID), (dict(x_stride=2052), INVALID),
    (dict(delta_stride=100), INVALID), (dict(out_stride=2049), INVALID),
    (dict(xo=None, xn=None, q=None, qs=None), INVALID), (dict(qs=None), INVALID),
    (dict(q=None), INVALID), (dict(x=A + 8), INVALID), (dict(delta=A + FAR + 4), INVALID),
    (dict(xn=A), INVALID),                          # overlaps x
    (dict(xo=A + 16), INVALID),                     # x_out shifted against x
    (dict(xn=A + 3 * FAR + 64), INVALID),           # overlaps x_out
    (dict(q=A + FAR), INVALID),                     # overlaps delta
    (dict(qs=A + 4 * FAR), INVALID),                # scales overlap xn_out
])
def test_norm_refusals(lib, kw, status):
    assert norm_call(lib, **kw) == status


def test_norm_null_description(lib):
    assert lib.moe_norm_quant(None, A, None, None, 1, A + FAR, None, None, None, None) == INVALID


@pytest.mark.parametrize("field,value,status", [
    ("in_features", 0, INVALID), ("in_features", 100, INVALID), ("in_features", 16448, UNSUPPORTED),
    ("out_features", 0, INVALID), ("out_features", (1 << 20) + 1, UNSUPPORTED),
    ("max_tokens", 0, INVALID), ("max_tokens", (1 << 20) + 1, UNSUPPORTED),
    ("max_rank", -8, INVALID), ("max_rank", 12, INVALID), ("max_rank", 136, UNSUPPORTED),
    ("wait_limit_ms", -1, INVALID),
])
def test_linear_descriptions(lib, field, value, status):
    d = bg.linear_desc(2048, 2048, 64, 16)
    setattr(d, field, value)
    with pytest.raises(bg.MoeError) as ei:
        bg.moe_linear_scratch_bytes(d)
    assert ei.value.status == status
    with pytest.raises(bg.MoeError) as ei:
        bg.moe_linear_create(d, 0)
    assert ei.value.status == status


def test_linear_scratch(lib):
    n = bg.moe_linear_scratch_bytes(bg.linear_desc(2048, 4096, 4096, 32))
    assert n >= 4096 * 32 * 4
    assert n < 64 * 2 ** 20


def test_null_handles(lib):
    w, d, r = bg.MoeW4(A, A, A), bg.score_desc(), bg.MoeRouting()
    assert lib.moe_linear_forward(None, A, 0, 0, None, 1, ctypes.byref(w), None, None, A, 0,
                                  None) == INVALID
    assert lib.moe_linear_destroy(None) == INVALID
    assert lib.moe_linear_get_error(None) == INVALID
    assert lib.moe_linear_create(None, 0, None) == INVALID
    assert lib.moe_route_scored(None, A, 1, ctypes.byref(d), ctypes.byref(r), None) == INVALID
    assert lib.moe_router_logits(None, A, 1, A, None, A, None) == INVALID


def test_struct_sizes(lib):
    assert ctypes.sizeof(bg.MoeNormDesc) == 48
    assert ctypes.sizeof(bg.MoeScoreDesc) == 32
    assert ctypes.sizeof(bg.MoeLinearDesc) == 20
    assert ctypes.sizeof(bg.MoeLora) == 32
