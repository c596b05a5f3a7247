"""AdaptedLayer's refusals: a wrong argument is found before the first launch.
The library's calls are recorded in place of being made, so these run without a
GPU."""
from types import SimpleNamespace

import pytest
import torch

from bit_grouped_gemm_gb300 import binding, stack

INVALID, CAPACITY = 1, 4
T, H, E = 5, 64, 8


class Calls(list):
    """Records every call of the binding; the plan takes `capacity` tokens."""

    def __init__(self, monkeypatch, capacity):
        for name in ("moe_norm_quant", "moe_linear_forward", "moe_router_logits",
                     "moe_grouped_w4_ffn", "moe_linear_destroy"):
            monkeypatch.setattr(binding, name, lambda *a, n=name, **k: self.append(n))
        monkeypatch.setattr(binding, "moe_linear_create", lambda *a: 1)

        def route(plan, logits, tokens, *a, **k):
            if tokens > capacity:
                raise binding.MoeError(CAPACITY, "moe_route_scored")
            if logits is None:
                raise binding.MoeError(INVALID, "moe_route_scored")
            self.append("moe_route_scored")
        monkeypatch.setattr(binding, "moe_route_scored", route)


def make(monkeypatch, adapters=True, capacity=T, max_tokens=T):
    calls = Calls(monkeypatch, capacity)
    ones = torch.ones(H, dtype=torch.bfloat16)
    layer = SimpleNamespace(router_w=torch.zeros(H, E, dtype=torch.bfloat16), router_bias=None,
                            routed_c=None, shared_c=None)
    proj = (torch.zeros(H, H // 8, dtype=torch.int32), *(torch.zeros(H, 1, dtype=torch.bfloat16),) * 2)
    lora = binding.lora(torch.zeros(2, 8, H, dtype=torch.bfloat16),
                        torch.zeros(2, H, 8, dtype=torch.bfloat16)) if adapters else None
    return calls, stack.AdaptedLayer(1, layer, ones, ones, proj, binding.score_desc(), lora, max_tokens)


def rows(n=T, h=H, dtype=torch.bfloat16):
    return torch.ones(n, h, dtype=dtype)


def f32(n=T, h=H):
    return rows(n, h, torch.float32)


def ids(n=T, dtype=torch.int32):
    return torch.zeros(n, dtype=dtype)


def test_a_right_call_goes_through(monkeypatch):
    calls, layer = make(monkeypatch)
    for n in (1, T):
        assert layer(rows(n), f32(n), ids(n)).shape == (n, H)
    layer(rows(), None)
    assert len(calls) == 3 * 6


@pytest.mark.parametrize("args,status", [
    ((rows(T + 1), f32(T + 1), ids(T + 1)), CAPACITY),       # would write past the layer's buffers
    ((rows(0), None), INVALID),
    ((rows(T, H + 8), None), INVALID),
    ((rows(dtype=torch.float16), None), INVALID),
    ((rows(2 * T)[::2], None), INVALID),                     # strided rows
    ((torch.ones(T, 2, H, dtype=torch.bfloat16), None), INVALID),
    ((rows(), f32(T - 1)), INVALID),                         # fewer rows than x
    ((rows(), f32(T, H - 8)), INVALID),
    ((rows(), rows()), INVALID),                             # y in bf16
    ((rows(), f32(H, T).T), INVALID),
    ((rows(), f32(), ids(T - 1)), INVALID),
    ((rows(), f32(), ids(dtype=torch.int64)), INVALID),
    ((rows(), f32(), ids(2 * T)[::2]), INVALID),
    ((rows(), f32(), [0] * T), INVALID),
    ((rows().to("meta"), f32(), ids()), INVALID),            # another device
])
def test_refusals_come_before_any_launch(monkeypatch, args, status):
    calls, layer = make(monkeypatch)
    with pytest.raises(binding.MoeError) as ei:
        layer(*args)
    assert ei.value.status == status and calls == []


def test_ids_without_adapters_are_refused(monkeypatch):
    calls, layer = make(monkeypatch, adapters=False)
    with pytest.raises(binding.MoeError) as ei:
        layer(rows(), f32(), ids())
    assert ei.value.status == INVALID and calls == []


@pytest.mark.parametrize("capacity", [1, 3])
def test_more_tokens_than_the_plan_takes(monkeypatch, capacity):
    calls, layer = make(monkeypatch, capacity=capacity)
    layer(rows(capacity), None)
    calls.clear()
    for n in (capacity + 1, T):
        with pytest.raises(binding.MoeError) as ei:
            layer(rows(n), f32(n), ids(n))
        assert ei.value.status == CAPACITY and calls == []


def test_a_closed_layer_is_refused(monkeypatch):
    calls, layer = make(monkeypatch)
    layer.close()
    calls.clear()
    with pytest.raises(binding.MoeError) as ei:
        layer(rows(), f32(), ids())
    assert ei.value.status == INVALID and calls == []
