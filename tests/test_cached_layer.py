"""PagedBatch's and CachedAttention's refusals: a wrong argument is found before the
first launch. The library's calls are recorded in place of being made, so these run
without a GPU."""
import pytest
import torch

from bit_grouped_gemm_gb300 import binding, stack

INVALID, CAPACITY = 1, 4
T, H, B, PAGE = 6, 128, 3, 16


class Calls(list):
    def __init__(self, monkeypatch):
        for name in ("moe_norm_quant", "moe_linear_forward", "moe_rope_store", "moe_tree_attention",
                     "moe_page_map", "moe_linear_destroy"):
            monkeypatch.setattr(binding, name, lambda *a, n=name, **k: self.append(n))
        monkeypatch.setattr(binding, "moe_linear_create", lambda *a: 1)


def triple(n, k):
    return (torch.zeros(n, k // 8, dtype=torch.int32), *(torch.zeros(n, k // 64, dtype=torch.bfloat16),) * 2)


def make(monkeypatch, cache="bf16", page=PAGE, adapters=True, **kw):
    calls = Calls(monkeypatch)
    d = binding.attn_desc(4, 2, 64, page, cache=cache, max_tokens=T, max_requests=B)
    k = torch.zeros(5, 2, page, 64, dtype=torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn)
    scale = None if cache == "bf16" else torch.ones(2)
    lora = binding.lora(torch.zeros(2, 8, H, dtype=torch.bfloat16),
                        torch.zeros(2, 512, 8, dtype=torch.bfloat16)) if adapters else None
    arg = dict(k=k, v=k.clone(), k_scale=scale, v_scale=scale, adapters=lora)
    arg.update(kw)
    layer = stack.CachedAttention(1, d, torch.ones(H, dtype=torch.bfloat16), triple(512, H), triple(H, 256),
                                  max_tokens=T, **arg)
    return calls, layer


def batch(requests=B, page=PAGE, tokens=T, words=0):
    return stack.PagedBatch(requests, page, 4, 5, tokens, words, device="cpu")


def rows(n=T, h=H, dtype=torch.bfloat16):
    return torch.ones(n, h, dtype=dtype)


def ids(n=T, dtype=torch.int32):
    return torch.zeros(n, dtype=dtype)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_right_call_goes_through(monkeypatch, cache):
    calls, layer = make(monkeypatch, cache)
    x, p = rows(), batch()
    p.step(ids(B), ids(B))
    assert layer(x, rows(dtype=torch.float32), p, ids()) is x
    layer(rows(1), None, p)
    one = ["moe_norm_quant", "moe_linear_forward", "moe_rope_store", "moe_tree_attention",
           "moe_linear_forward", "moe_norm_quant"]
    assert calls == ["moe_page_map"] + 2 * one
    layer.close()
    layer.close()
    assert calls[-2:] == ["moe_linear_destroy"] * 2 and len(calls) == 15
    with pytest.raises(binding.MoeError):
        layer(x, None, p)


@pytest.mark.parametrize("args,status", [
    ((rows(T + 1), None, batch(tokens=T + 1)), CAPACITY),
    ((rows(), None, batch(requests=B + 1)), CAPACITY),
    ((rows(0), None, batch()), INVALID),
    ((rows(), None, batch(tokens=T - 1)), INVALID),          # more rows than the batch has
    ((rows(), None, batch(page=32)), INVALID),
    ((rows(T, H + 8), None, batch()), INVALID),
    ((rows(dtype=torch.float16), None, batch()), INVALID),
    ((rows(2 * T)[::2], None, batch()), INVALID),
    ((rows(), rows(), batch()), INVALID),                    # y in bf16
    ((rows(), rows(T - 1, dtype=torch.float32), batch()), INVALID),
    ((rows(), None, batch(), ids(T - 1)), INVALID),
    ((rows(), None, batch(), ids(dtype=torch.int64)), INVALID),
    ((rows().to("meta"), None, batch()), INVALID),
])
def test_a_wrong_call_launches_nothing(monkeypatch, args, status):
    calls, layer = make(monkeypatch)
    with pytest.raises(binding.MoeError) as e:
        layer(*args)
    assert e.value.status == status and not calls


def test_adapters_are_the_layers(monkeypatch):
    calls, layer = make(monkeypatch, adapters=False)
    with pytest.raises(binding.MoeError):
        layer(rows(), None, batch(), ids())
    assert not calls


@pytest.mark.parametrize("kw", [
    dict(k=torch.zeros(5, 2, 32, 64, dtype=torch.bfloat16)),       # another page size
    dict(k=torch.zeros(5, 4, PAGE, 64, dtype=torch.bfloat16)),
    dict(v=torch.zeros(4, 2, PAGE, 64, dtype=torch.bfloat16)),     # fewer pages than k
    dict(k_scale=torch.ones(2), v_scale=torch.ones(2)),            # scales of a bf16 cache
])
def test_wrong_caches_are_refused(monkeypatch, kw):
    with pytest.raises(binding.MoeError):
        make(monkeypatch, **kw)


@pytest.mark.parametrize("args", [
    (ids(B + 1), ids(B)), (ids(B), ids(B, torch.int64)), (ids(B), ids(2 * B)[::2]),
    (ids(B), ids(B), ids(T)),                                      # a tree without masks
])
def test_steps_are_checked(monkeypatch, args):
    calls = Calls(monkeypatch)
    with pytest.raises(binding.MoeError):
        batch().step(*args)
    assert not calls
    p = batch(words=1)
    p.step(ids(B), ids(B), ids(T))
    with pytest.raises(binding.MoeError):
        p.step(ids(B), ids(B), ids(T - 1))
    assert calls == ["moe_page_map"]


def test_another_current_device_is_refused(monkeypatch):
    dev = torch.device("cuda", 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert not stack._here(dev) and stack._here(torch.device("cuda", 0)) and stack._here(torch.device("cpu"))
    calls, layer = make(monkeypatch)
    p = batch()
    monkeypatch.setattr(stack, "_here", lambda d: False)
    for call in (lambda: layer(rows(), None, p), lambda: p.step(ids(B), ids(B))):
        with pytest.raises(binding.MoeError):
            call()
    assert not calls


@pytest.mark.parametrize("pages,fits", [(4, True), (5, True), (6, False)])
def test_a_batch_with_more_pages_than_the_cache_is_refused(monkeypatch, pages, fits):
    calls, layer = make(monkeypatch)
    p = stack.PagedBatch(B, PAGE, 4, pages, T, device="cpu")
    if fits:
        layer(rows(), None, p)
        assert len(calls) == 6
        return
    with pytest.raises(binding.MoeError) as e:
        layer(rows(), None, p)
    assert e.value.status == INVALID and not calls


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("bad", [
    dict(qkv=triple(256, H)), dict(qkv=triple(512, 2 * H)), dict(out=triple(2 * H, 256)), dict(out=triple(H, 128)),
    dict(qkv=(triple(512, H)[0], bf16(512, 1), bf16(512, 2))),
    dict(out=(triple(H, 256)[0], bf16(H, 4), bf16(H, 8)[:, ::2])),
    dict(out=tuple(t.to("meta") for t in triple(H, 256))), dict(norm=bf16(H).float()),
    dict(norm=bf16(2 * H)[::2]), dict(norm=bf16(2 * H)), dict(k=bf16(5, 2, PAGE, 64).to("meta")),
    dict(v=bf16(5, 2, PAGE, 64).to("meta")), dict(v=bf16(5, PAGE, 2, 64).transpose(1, 2)),
])
def test_a_layers_tensors_have_its_sizes(monkeypatch, bad):
    """Kernels read these by the layer's sizes: others would be read behind their ends."""
    calls = Calls(monkeypatch)
    d = binding.attn_desc(4, 2, 64, PAGE, max_tokens=T, max_requests=B)
    arg = dict(norm=bf16(H), qkv=triple(512, H), out=triple(H, 256), k=bf16(5, 2, PAGE, 64), v=bf16(5, 2, PAGE, 64))
    stack.CachedAttention(1, d, **arg, max_tokens=T)
    with pytest.raises(binding.MoeError) as e:
        stack.CachedAttention(1, d, **{**arg, **bad}, max_tokens=T)
    assert e.value.status == INVALID and not calls


@pytest.mark.parametrize("scale", [torch.ones(3), torch.ones(4)[::2], torch.ones(2).to("meta")])
def test_scales_have_a_value_per_head(monkeypatch, scale):
    for kw in (dict(k_scale=scale), dict(v_scale=scale)):
        with pytest.raises(binding.MoeError):
            make(monkeypatch, "e4m3", **kw)


def test_a_layer_that_is_refused_keeps_no_handle(monkeypatch):
    made, gone = [], []

    def create(desc, device):
        if made:
            raise binding.MoeError(3, "moe_linear_create")
        made.append(7)
        return 7
    calls = Calls(monkeypatch)
    monkeypatch.setattr(binding, "moe_linear_create", create)
    monkeypatch.setattr(binding, "moe_linear_destroy", gone.append)
    d = binding.attn_desc(4, 2, 64, PAGE, max_tokens=T, max_requests=B)
    with pytest.raises(binding.MoeError):
        stack.CachedAttention(1, d, bf16(H), triple(512, H), triple(H, 256), bf16(5, 2, PAGE, 64),
                              bf16(5, 2, PAGE, 64), max_tokens=T)
    assert made == gone and not calls
