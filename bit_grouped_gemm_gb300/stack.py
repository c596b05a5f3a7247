"""Device-resident synthetic layers and the stacked-layer driver.

``make_layer`` materialises one layer's tensors (router, routed experts,
shared expert) on a device from the seeded generator in ``synth`` and keeps
the ``MoeExperts`` structs the C ABI takes. ``run_stack`` chains layers with
the residual update ``x <- bf16(x + alpha * moe(rmsnorm(x)))``, every step
through the C ABI. ``AdaptedLayer`` is a served layer around the block: a 4-bit
projection with per-request adapters, then the experts on a scored routing.
"""
from __future__ import annotations

import dataclasses
import math
from typing import List, Optional

import torch

from . import binding, synth


@dataclasses.dataclass
class DeviceLayer:
    router_w: torch.Tensor
    router_bias: Optional[torch.Tensor]
    routed: dict            # name -> (q, s, b)
    shared: Optional[dict]
    routed_c: binding.MoeExperts = None
    shared_c: Optional[binding.MoeExperts] = None

    def __post_init__(self):
        r = self.routed
        self.routed_c = binding.experts(r["gate"], r["up"], r["down"])
        if self.shared is not None:
            s = self.shared
            self.shared_c = binding.experts(s["gate"], s["up"], s["down"])

    def nbytes(self) -> int:
        n = self.router_w.numel() * 2
        for d in (self.routed, self.shared or {}):
            for m in d.values():
                n += sum(t.numel() * t.element_size() for t in m)
        return n


def make_layer(w: synth.Workload, layer: int, device="cuda") -> DeviceLayer:
    p = synth.layer_params(w, layer, device)
    return DeviceLayer(p["router_w"], p["router_bias"], p["routed"], p["shared"])


def make_layers(w: synth.Workload, device="cuda") -> List[DeviceLayer]:
    return [make_layer(w, l, device) for l in range(w.layers)]


def residual_alpha(num_layers: int) -> float:
    """Scale of each layer's output in the residual stream (1/sqrt(L))."""
    return 1.0 / math.sqrt(num_layers)


def run_stack(plan: int, x: torch.Tensor, xn: torch.Tensor, layers: List[DeviceLayer], T: int,
              y_buf: torch.Tensor, alpha: float, stream=None, fused: bool = True) -> torch.Tensor:
    """Run the layers in order on the residual stream ``x`` (bf16, updated in
    place) and return it. Every layer sees the RMS-normalised stream ``xn``
    (bf16 scratch of x's shape); ``y_buf`` is the fp32 [T, H] layer output
    (written only when ``fused`` is False).

        xn = rmsnorm(x)
        for each layer: y = moe(xn); x = bf16(x + alpha * y); xn = rmsnorm(x)

    ``fused`` takes each layer and its update in one call
    (moe_forward_layer_residual, y never written); otherwise
    moe_forward_layer then moe_residual_add. Both give identical bits.
    """
    binding.moe_residual_add(plan, x, None, T, 0.0, x, xn, stream)
    for L in layers:
        if fused:
            binding.moe_forward_layer_residual(plan, xn, T, L.router_w, L.router_bias,
                                               L.routed_c, L.shared_c, alpha, x, xn, stream)
        else:
            binding.moe_forward_layer(plan, xn, T, L.router_w, L.router_bias, L.routed_c,
                                      L.shared_c, y_buf, stream)
            binding.moe_residual_add(plan, x, y_buf, T, alpha, x, xn, stream)
    return x


class AdaptedLayer:
    """A pre-norm layer for the batch of many requests, each with its own
    low-rank adapter or none, on the residual stream x (bf16 [T, H], in place):

        h8, hs = e4m3(rmsnorm(x + alpha * y) * w1)   y: the last layer's output
        d = projection(h8) with adapters             4-bit weights, H -> H
        x = x + d;  xn = rmsnorm(x) * w2
        y = experts(xn) on moe_route_scored's choice

    The experts' FP32 output y is returned and joins the stream in the next
    layer's first norm. ``norm1`` and ``norm2`` are bf16 [H]; ``proj`` is a
    (qweight, scales, biases) triple of an H x H matrix; ``adapters`` a
    ``binding.MoeLora`` (its tensors must outlive the layer) or None;
    ``score`` a ``binding.MoeScoreDesc``. A call takes up to ``max_tokens`` tokens,
    or the plan's if these are fewer; wrong arguments are refused before the
    first launch, so x is then as it was.
    """

    def __init__(self, plan: int, layer: DeviceLayer, norm1, norm2, proj, score,
                 adapters=None, max_tokens: int = 4096, alpha: float = 1.0):
        H = layer.router_w.shape[0]
        dev = layer.router_w.device
        self.plan, self.layer, self.score, self.adapters = plan, layer, score, adapters
        self.norm1, self.norm2, self.proj = norm1, norm2, proj
        self.alpha, self.max_tokens = alpha, max_tokens
        self.plan_tokens = 0    # the largest T that the plan is known to take
        self.proj_c = binding.w4(*proj)
        rank = adapters.rank if adapters is not None else 0
        self.linear = binding.moe_linear_create(binding.linear_desc(H, H, max_tokens, rank),
                                                dev.index or 0)
        empty = lambda *shape, dt: torch.empty(shape, dtype=dt, device=dev)
        self.h8 = empty(max_tokens, H, dt=torch.float8_e4m3fn)
        self.hs = empty(max_tokens, 1, dt=torch.float32)
        self.d = empty(max_tokens, H, dt=torch.bfloat16)
        self.xn = empty(max_tokens, H, dt=torch.bfloat16)
        self.logits = empty(max_tokens, layer.router_w.shape[1], dt=torch.float32)
        self.y = empty(max_tokens, H, dt=torch.float32)

    def close(self) -> None:
        if self.linear:
            binding.moe_linear_destroy(self.linear)
            self.linear = None

    def _check(self, x, y, adapter) -> None:
        H, dev = self.h8.shape[1], self.h8.device
        rows = lambda t, dtype, shape: (isinstance(t, torch.Tensor) and t.dtype == dtype and
                                        t.shape == shape and t.device == dev and t.is_contiguous())
        T = x.shape[0] if isinstance(x, torch.Tensor) and x.dim() == 2 else 0
        if T > self.max_tokens:
            raise binding.MoeError(binding.MOE_ERR_CAPACITY, "AdaptedLayer")
        if T > self.plan_tokens:
            # A call without logits tells of a T above the plan's before it looks
            # at them, and launches nothing.
            try:
                binding.moe_route_scored(self.plan, None, T, self.score, stream=0)
            except binding.MoeError as e:
                if e.status == binding.MOE_ERR_CAPACITY:
                    raise
            self.plan_tokens = T
        ok = self.linear is not None and T > 0 and rows(x, torch.bfloat16, (T, H))
        ok = ok and (y is None or rows(y, torch.float32, (T, H)))
        if adapter is not None:
            ok = ok and self.adapters is not None and rows(adapter, torch.int32, (T,))
        if not ok:
            raise binding.MoeError(binding.MOE_ERR_INVALID_ARG, "AdaptedLayer")

    def __call__(self, x: torch.Tensor, y: Optional[torch.Tensor], adapter=None,
                 stream=None) -> torch.Tensor:
        """One pass over T = len(x) tokens; ``adapter`` is int32 [T] (-1: none)."""
        self._check(x, y, adapter)
        T, H = x.shape
        L = self.layer
        first = binding.norm_desc(H, alpha=self.alpha, delta_f32=True)
        binding.moe_norm_quant(first, x, y, self.norm1, T, x_out=x, q_out=self.h8, q_scale=self.hs,
                               stream=stream)
        binding.moe_linear_forward(self.linear, self.h8, T, self.proj_c, self.d, x_scale=self.hs,
                                   lora=self.adapters if adapter is not None else None,
                                   adapter=adapter, stream=stream)
        binding.moe_norm_quant(binding.norm_desc(H), x, self.d, self.norm2, T, x_out=x,
                               xn_out=self.xn, stream=stream)
        binding.moe_router_logits(self.plan, self.xn, T, L.router_w, L.router_bias, self.logits,
                                  stream)
        routing = binding.moe_route_scored(self.plan, self.logits, T, self.score, None, stream)
        binding.moe_grouped_w4_ffn(self.plan, self.xn, T, routing, L.routed_c, L.shared_c, self.y,
                                   stream)
        return self.y[:T]
