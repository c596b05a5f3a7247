"""Refusals of the operators of attention over a paged cache: every wrong argument is found on the
host, before any CUDA call, so these run without a GPU. Addresses are made up and never read."""
import ctypes

import pytest

import bit_grouped_gemm_gb300 as bg
from bit_grouped_gemm_gb300 import binding

INVALID, UNSUPPORTED, CAPACITY = 1, 2, 4
A, FAR = 1 << 30, 1 << 33      # an aligned address, and others far from it


@pytest.fixture(scope="module")
def lib():
    from bit_grouped_gemm_gb300 import build
    build.build()
    return binding.load_library()


NAMES = ("table", "ring", "owned", "owned_out", "ring_pos", "ring_pos_out", "length", "offsets",
         "slot", "position", "mask", "status", "context", "added", "parent")


def page_call(lib, desc=None, **at):
    d = dict(requests=4, page_size=16, table_width=8, max_tokens=64, ring_size=32, mask_words=1)
    d.update(desc or {})
    a = {n: A + i * FAR for i, n in enumerate(NAMES)}
    a.update(at)
    pool = bg.MoePagePool(*(a[n] for n in NAMES[:6]))
    out = bg.MoeTokenMap(*(a[n] for n in NAMES[6:12]))
    return lib.moe_page_map(ctypes.byref(bg.page_desc(**d)), a["context"], a["added"], a["parent"],
                            ctypes.byref(pool), ctypes.byref(out), None)


@pytest.mark.parametrize("desc,status", [
    (dict(requests=0), INVALID), (dict(requests=4097), UNSUPPORTED), (dict(page_size=0), INVALID),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED),
    (dict(table_width=0), INVALID), (dict(table_width=(1 << 18) + 1), UNSUPPORTED),
    (dict(max_tokens=0), INVALID), (dict(max_tokens=(1 << 20) + 1), UNSUPPORTED),
    (dict(ring_size=0), INVALID), (dict(ring_size=(1 << 30) + 1), UNSUPPORTED),
    (dict(mask_words=-1), INVALID), (dict(mask_words=5), UNSUPPORTED), (dict(mask_words=0), INVALID),
])
def test_page_descriptions(lib, desc, status):
    assert page_call(lib, desc) == status


@pytest.mark.parametrize("name", [n for n in NAMES if n not in ("mask", "parent")])
def test_page_null_pointers(lib, name):
    assert page_call(lib, **{name: None}) == INVALID


@pytest.mark.parametrize("at", [
    dict(mask=None), dict(mask=A + 4 + 90 * FAR), dict(slot=A + 90 * FAR + 2), dict(context=A + 90 * FAR + 1),
    dict(table=A + FAR), dict(slot=A + 9 * FAR + 252), dict(length=A + 2 * FAR), dict(length=A + 12 * FAR),
    dict(owned_out=A + 2 * FAR + 4), dict(ring_pos_out=A + 4 * FAR + 4), dict(owned_out=A + 4 * FAR),
    dict(status=A + 7 * FAR + 16), dict(parent=A + 8 * FAR), dict(offsets=A + 6 * FAR + 12),
    dict(ring=A + 124), dict(mask=A + 13 * FAR),
])
def test_page_pointers(lib, at):
    assert page_call(lib, **at) == INVALID


def test_page_parent_needs_masks(lib):
    assert page_call(lib, dict(mask_words=0), mask=None) == INVALID
    assert lib.moe_page_map(None, A, A, None, None, None, None) == INVALID


@pytest.mark.parametrize("field,value,status", [
    ("heads", 0, INVALID), ("heads", 15, INVALID), ("kv_heads", 0, INVALID), ("heads", 258, UNSUPPORTED),
    ("head_dim", 0, INVALID), ("head_dim", 96, UNSUPPORTED), ("head_dim", 512, UNSUPPORTED),
    ("page_size", 0, INVALID), ("page_size", 8, UNSUPPORTED), ("page_size", 100, UNSUPPORTED),
    ("cache_type", 2, INVALID), ("cache_type", -1, INVALID), ("max_tokens", 0, INVALID),
    ("max_tokens", (1 << 20) + 1, UNSUPPORTED), ("max_requests", 0, INVALID), ("max_requests", 4097, UNSUPPORTED),
    ("softmax_scale", -1.0, INVALID), ("softmax_scale", float("nan"), INVALID),
    ("softmax_scale", float("inf"), INVALID), ("rotary_dim", -16, INVALID), ("rotary_dim", 144, INVALID),
    ("rotary_dim", 63, INVALID), ("rotary_dim", 24, UNSUPPORTED), ("rope_layout", 2, INVALID),
    ("rope_scaling", 3, INVALID), ("rope_theta", 0.5, INVALID), ("rope_theta", float("nan"), INVALID),
    ("rope_factor", 0.5, INVALID), ("rope_factor", float("inf"), INVALID), ("rope_low", 32.0, INVALID),
    ("rope_high", float("nan"), INVALID), ("rope_original", 0, INVALID), ("rope_gain", float("nan"), INVALID),
    ("wait_limit_ms", -1, INVALID),
])
def test_attention_descriptions(lib, field, value, status):
    d = bg.attn_desc(16, 2, 128, 64, rope_scaling="by_parts", rotary_dim=64)
    setattr(d, field, value)
    with pytest.raises(bg.MoeError) as ei:
        bg.moe_attn_scratch_bytes(d)
    assert ei.value.status == status
    with pytest.raises(bg.MoeError) as ei:
        bg.moe_attn_create(d, 0)
    assert ei.value.status == status


def test_attention_scratch_does_not_grow_with_tokens(lib):
    small = bg.moe_attn_scratch_bytes(bg.attn_desc(16, 2, 256, 64, max_tokens=1))
    assert small == bg.moe_attn_scratch_bytes(bg.attn_desc(16, 2, 256, 64, max_tokens=1 << 20))
    assert small < 64 * 2 ** 20


def test_null_handles(lib):
    c = bg.MoeKvCache(A, A, None, None, 1)
    assert lib.moe_attn_destroy(None) == INVALID
    assert lib.moe_attn_get_error(None) == INVALID
    assert lib.moe_attn_create(None, 0, None) == INVALID
    assert lib.moe_rope_store(None, A, 0, A, 0, A, 0, 1, A, A, A, 0, ctypes.byref(c), None) == INVALID
    assert lib.moe_tree_attention(None, A, 0, 1, ctypes.byref(c), A, 1, 1, A, A, None, 0, A, 0,
                                  None) == INVALID


def test_struct_sizes(lib):
    assert ctypes.sizeof(bg.MoeAttnDesc) == 96
    assert ctypes.sizeof(bg.MoeKvCache) == 40
    assert ctypes.sizeof(bg.MoePagePool) == 48
    assert ctypes.sizeof(bg.MoeTokenMap) == 48
    assert ctypes.sizeof(bg.MoePageDesc) == 24


def test_binding_checks_types():
    import torch
    i, f = torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    for bad in (f, i.long()):
        with pytest.raises(bg.MoeError):
            bg.page_pool(bad, i, i, i)
        with pytest.raises(bg.MoeError):
            bg.token_map(i, i, bad, i, i)
    with pytest.raises(bg.MoeError):
        bg.token_map(i, i, i, i, i, mask=i)
    k = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    k8, s = k.to(torch.float8_e4m3fn), torch.ones(2)
    bg.kv_cache(k, k.clone())
    bg.kv_cache(k8, k8.clone(), s, s)
    for args in ((k, k8), (k8, k8), (k, k, s, s), (k8, k8, s), (k8, k8, s, torch.ones(3)), (k[0], k[0]),
                 (k, k[:, :, :8]), (k.transpose(1, 2), k.transpose(1, 2)), (k.float(), k.float())):
        with pytest.raises(bg.MoeError):
            bg.kv_cache(*args)
