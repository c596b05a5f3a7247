"""The binding's check of tensor types: the library gets addresses alone, so a
tensor of another type has to be refused before them. No GPU: the library's calls
are recorded in place of being made."""
import pytest
import torch

import bit_grouped_gemm_gb300 as bg
from bit_grouped_gemm_gb300 import binding

BF, F32, I32, E4 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn
H = 64


def t(dtype, *shape):
    return torch.zeros(*(shape or (4, H)), dtype=torch.uint8 if dtype is E4 else dtype).view(dtype)


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(binding, "_status", lambda name, *a: made.append(name))
    monkeypatch.setattr(binding, "_stream", lambda s: 0)
    return made


def refused(calls, f, *a, **k):
    with pytest.raises(bg.MoeError) as ei:
        f(*a, **k)
    assert ei.value.status == 1 and calls == []


def wrong(*right):
    return [d for d in (BF, torch.float16, F32, torch.float64, I32, torch.int64, E4,
                        torch.float8_e5m2, torch.bool) if d not in right]


def linear(x=BF, ids=I32, y=BF, xs=None):
    w = bg.w4(t(I32, H, H // 8), t(BF, H, 1), t(BF, H, 1))
    lora = bg.lora(t(BF, 2, 8, H), t(BF, 2, H, 8))
    bg.moe_linear_forward(1, t(x), 4, w, t(y), x_scale=None if xs is None else t(xs, 4), lora=lora,
                          adapter=t(ids, 4))


def test_right_types_go_through(calls):
    linear()
    linear(x=E4, xs=F32)
    linear(x=torch.uint8, xs=F32)
    linear(x=torch.int16, y=torch.uint16)        # bit patterns
    bg.moe_norm_quant(bg.norm_desc(H), t(BF), t(BF), t(BF, H), 4, t(BF), t(BF), t(E4), t(F32, 4))
    bg.moe_norm_quant(bg.norm_desc(H, delta_f32=True), t(BF), t(F32), None, 4, xn_out=t(BF))
    bg.moe_router_logits(1, t(BF), 4, t(BF, H, 8), t(F32, 8), t(F32, 4, 8))
    bg.moe_route_scored(1, t(F32, 4, 8), 4, bg.score_desc(bias=t(F32, 8)))
    bg.moe_route_scored(1, 1 << 20, 4, bg.score_desc())
    assert len(calls) == 9


@pytest.mark.parametrize("arg,types", [("x", wrong(BF, E4)), ("ids", wrong(I32)), ("y", wrong(BF)),
                                       ("xs", wrong(F32))])
def test_linear_types(calls, arg, types):
    for d in types:
        refused(calls, linear, **{arg: d})


def test_norm_types(calls):
    right = dict(x=BF, delta=BF, weight=BF, x_out=BF, xn_out=BF, q_out=E4, q_scale=F32)
    for f32 in (False, True):
        right["delta"] = F32 if f32 else BF
        for arg in right:
            for d in wrong(right[arg]):
                got = {n: t(d if n == arg else v) for n, v in right.items()}
                refused(calls, bg.moe_norm_quant, bg.norm_desc(H, delta_f32=f32), T=4, **got)


def test_routing_types(calls):
    for d in wrong(F32):
        refused(calls, bg.moe_route_scored, 1, t(d, 4, 8), 4, bg.score_desc())
        refused(calls, bg.score_desc, "sigmoid", t(d, 8))
    right = dict(x=BF, router_w=BF, router_bias=F32, logits=F32)
    for arg in right:
        for d in wrong(right[arg]):
            refused(calls, bg.moe_router_logits, 1, T=4, **{n: t(d if n == arg else v) for n, v in right.items()})


def test_weights_and_adapters(calls):
    for d in wrong(I32):
        refused(calls, bg.w4, t(d), t(BF), t(BF))
    for d in wrong(BF):
        refused(calls, bg.w4, t(I32), t(d), t(BF))
        refused(calls, bg.w4, t(I32), t(BF), t(d))
        refused(calls, bg.lora, t(d, 2, 8, H), t(BF, 2, H, 8))
        refused(calls, bg.lora, t(BF, 2, 8, H), t(d, 2, H, 8))
    for d in wrong(F32):
        refused(calls, bg.lora, t(BF, 2, 8, H), t(BF, 2, H, 8), t(d, 2))
    refused(calls, bg.lora, t(BF, 2, 8, H), t(BF, 2, 8, H))          # B as [n, r, N]
    refused(calls, bg.lora, t(BF, 2, 8, H), t(BF, 3, H, 8))
    refused(calls, bg.lora, t(BF, 2, 8, H), t(BF, 2, 8, H).transpose(1, 2))
    refused(calls, bg.lora, t(BF, 2, 8, H), t(BF, 2, H, 8), t(F32, 3))
