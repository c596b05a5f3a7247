"""Device-resident synthetic layers and the stacked-layer driver.

``make_layer`` materialises one layer's tensors (router, routed experts,
shared expert) on a device from the seeded generator in ``synth`` and keeps
the ``MoeExperts`` structs the C ABI takes. ``run_stack`` chains layers with
the residual update ``x <- bf16(x + alpha * moe(rmsnorm(x)))``, every step
through the C ABI. ``AdaptedLayer`` is a served layer around the block: a 4-bit
projection with per-request adapters, then the experts on a scored routing.
``PagedBatch`` keeps the cache pages of a batch of requests, and
``CachedAttention`` is the attention half of a layer over them.
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


def _rows(t, dtype, shape, dev) -> bool:
    return (isinstance(t, torch.Tensor) and t.dtype == dtype and tuple(t.shape) == tuple(shape) and
            t.device == dev and t.is_contiguous())


def _here(dev) -> bool:
    """Whether calls that run on the current device run on ``dev``."""
    return dev.type != "cuda" or dev.index == torch.cuda.current_device()


def _settle(dev) -> None:
    """Waits for what the current stream still has to fill: the first call may come on another."""
    if dev.type == "cuda":
        torch.cuda.current_stream(dev).synchronize()


class PagedBatch:
    """The cache pages of up to ``requests`` requests, ``table_width`` each at most, and
    what a step's kernels need to know of its tokens; all of it on the device, where
    moe_page_map keeps it, so that a captured step follows lengths that change. Calls
    are made with its device as the current one.

    Pages 0..``pages``-1 are free at first. ``offsets``, ``length``, ``slot``,
    ``position``, ``mask`` (None without ``mask_words``) and ``status`` hold the last
    step's.
    """

    def __init__(self, requests: int, page_size: int, table_width: int, pages: int,
                 max_tokens: int, mask_words: int = 0, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.desc = binding.page_desc(requests, page_size, table_width, max_tokens, pages, mask_words)
        self.table = torch.zeros(requests, table_width, **i32)
        self.ring = torch.arange(pages, **i32)
        self.owned = torch.zeros(requests, **i32)
        self.ring_pos = torch.tensor([0, pages], **i32)
        self.length = torch.zeros(requests, **i32)
        self.offsets = torch.zeros(requests + 1, **i32)
        self.slot = torch.full((max_tokens,), -1, **i32)
        self.position = torch.zeros(max_tokens, **i32)
        self.status = torch.zeros(5, **i32)
        self.mask = torch.zeros(max_tokens, mask_words, dtype=torch.int64,
                                device=device) if mask_words else None
        self.pool = binding.page_pool(self.table, self.ring, self.owned, self.ring_pos)
        self.map = binding.token_map(self.length, self.offsets, self.slot, self.position,
                                     self.status, self.mask)
        _settle(self.table.device)

    def step(self, context: torch.Tensor, added: torch.Tensor,
             parent: Optional[torch.Tensor] = None, stream=None) -> None:
        """The next step: request b holds ``context[b]`` tokens and adds ``added[b]``
        (negative: it ends); ``parent`` int32 [max_tokens] makes trees of the new ones."""
        B, M, dev = self.desc.requests, self.desc.max_tokens, self.table.device
        ok = _here(dev) and _rows(context, torch.int32, (B,), dev) and _rows(added, torch.int32, (B,), dev)
        if parent is not None:
            ok = ok and self.mask is not None and _rows(parent, torch.int32, (M,), dev)
        if not ok:
            raise binding.MoeError(binding.MOE_ERR_INVALID_ARG, "PagedBatch")
        binding.moe_page_map(self.desc, context, added, parent, self.pool, self.map, stream)


class CachedAttention:
    """The attention half of a pre-norm layer on the residual stream x (bf16 [T, H],
    in place), with keys and values of a ``PagedBatch`` in a cache of its own:

        x = x + alpha * y;  h8, hs = e4m3(rmsnorm(x) * norm)   y: the last layer's output
        q, k, v = projection(h8) with adapters    4-bit, H -> (heads + 2 kv_heads) D
        q, k turned by their positions;  cache[slot] = k, v
        a = attention of q over the requests' pages
        x = x + output(a)                         4-bit, heads D -> H

    ``attn`` is a handle of ``desc`` (layers of one shape may share it), ``qkv`` and
    ``out`` are (qweight, scales, biases) triples, ``norm`` bf16 [H], ``k`` and ``v``
    the cache [pages, kv_heads, page_size, D], with scales for e4m3; ``adapters`` a
    ``binding.MoeLora`` of the first projection, or None. What a caller passes must
    outlive the layer. The cache has at least the batch's pages. Rows of x behind the
    batch's last token are changed, but no other row depends on them; tokens of the step
    past the rows of x store nothing. A call takes up to ``max_tokens`` rows, with the
    layer's device as the current one; wrong arguments are refused before the first
    launch, so x is then as it was.
    """

    def __init__(self, attn: int, desc, norm, qkv, out, k, v, k_scale=None, v_scale=None,
                 adapters=None, max_tokens: int = 4096, alpha: float = 1.0):
        H, dev = norm.shape[0], norm.device
        self.attn, self.desc, self.norm, self.adapters = attn, desc, norm, adapters
        self.max_tokens, self.alpha = min(max_tokens, desc.max_tokens), alpha
        self.q_cols, self.kv_cols = desc.heads * desc.head_dim, desc.kv_heads * desc.head_dim
        cols = self.q_cols + 2 * self.kv_cols
        shape = (k.shape[0], desc.kv_heads, desc.page_size, desc.head_dim)
        # (types are checked where the structs are made; an address has no size)
        fits = lambda t, n: isinstance(t, int) or (t.numel() == n and t.device == dev and t.is_contiguous())
        ok = fits(norm, H) and norm.dtype == torch.bfloat16 and tuple(k.shape) == shape
        ok = ok and fits(k, k.numel()) and fits(v, k.numel()) and (k_scale is not None) == (desc.cache_type != 0)
        ok = ok and all(s is None or fits(s, desc.kv_heads) for s in (k_scale, v_scale))
        for w, n, m in ((qkv, cols, H), (out, H, self.q_cols)):
            ok = ok and fits(w[0], n * m // 8) and fits(w[1], n * m // 64) and fits(w[2], n * m // 64)
        if not ok:
            raise binding.MoeError(binding.MOE_ERR_INVALID_ARG, "CachedAttention")
        self.kept = (qkv, out, k, v, k_scale, v_scale)
        self.qkv_c, self.out_c = binding.w4(*qkv), binding.w4(*out)
        self.cache = binding.kv_cache(k, v, k_scale, v_scale)
        rank, M = adapters.rank if adapters is not None else 0, self.max_tokens
        self.project = binding.moe_linear_create(binding.linear_desc(H, cols, M, rank), dev.index or 0)
        try:
            self.output = binding.moe_linear_create(binding.linear_desc(self.q_cols, H, M), dev.index or 0)
        except binding.MoeError:
            binding.moe_linear_destroy(self.project)
            raise
        empty = lambda *shape, dt: torch.empty(shape, dtype=dt, device=dev)
        self.h8 = empty(M, H, dt=torch.float8_e4m3fn)
        self.hs = empty(M, 1, dt=torch.float32)
        self.qkv = empty(M, cols, dt=torch.bfloat16)
        # (attention leaves rows behind the last token as they are)
        self.a = torch.zeros(M, self.q_cols, dtype=torch.bfloat16, device=dev)
        self.d = empty(M, H, dt=torch.bfloat16)
        _settle(dev)

    def close(self) -> None:
        for name in ("project", "output"):
            if getattr(self, name):
                binding.moe_linear_destroy(getattr(self, name))
                setattr(self, name, None)

    def _check(self, x, y, batch, adapter) -> None:
        H, dev = self.h8.shape[1], self.h8.device
        T = x.shape[0] if isinstance(x, torch.Tensor) and x.dim() == 2 else 0
        if T > self.max_tokens or batch.desc.requests > self.desc.max_requests:
            raise binding.MoeError(binding.MOE_ERR_CAPACITY, "CachedAttention")
        ok = self.project is not None and _here(dev) and T > 0 and _rows(x, torch.bfloat16, (T, H), dev)
        ok = ok and (y is None or _rows(y, torch.float32, (T, H), dev))
        ok = ok and batch.table.device == dev and T <= batch.desc.max_tokens
        ok = ok and batch.desc.page_size == self.desc.page_size
        ok = ok and batch.desc.ring_size <= self.cache.pages
        if adapter is not None:
            ok = ok and self.adapters is not None and _rows(adapter, torch.int32, (T,), dev)
        if not ok:
            raise binding.MoeError(binding.MOE_ERR_INVALID_ARG, "CachedAttention")

    def __call__(self, x: torch.Tensor, y: Optional[torch.Tensor], batch: PagedBatch, adapter=None,
                 stream=None) -> torch.Tensor:
        """One pass over the rows of ``batch``'s last step, T = len(x) of them with what
        pads them; ``adapter`` is int32 [T] (-1: none)."""
        self._check(x, y, batch, adapter)
        T, H = x.shape
        row, heads = self.qkv.shape[1], self.q_cols
        q, k, v = (self.qkv.data_ptr() + 2 * c for c in (0, heads, heads + self.kv_cols))
        binding.moe_norm_quant(binding.norm_desc(H, alpha=self.alpha, delta_f32=True), x, y, self.norm,
                               T, x_out=x, q_out=self.h8, q_scale=self.hs, stream=stream)
        binding.moe_linear_forward(self.project, self.h8, T, self.qkv_c, self.qkv, x_scale=self.hs,
                                   lora=self.adapters if adapter is not None else None,
                                   adapter=adapter, stream=stream)
        binding.moe_rope_store(self.attn, q, k, v, T, batch.position, batch.slot, q, self.cache,
                               q_stride=row, k_stride=row, v_stride=row, out_stride=row, stream=stream)
        binding.moe_tree_attention(self.attn, q, T, self.cache, batch.table, batch.offsets,
                                   batch.length, self.a, mask=batch.mask, q_stride=row, stream=stream)
        binding.moe_linear_forward(self.output, self.a, T, self.out_c, self.d, stream=stream)
        binding.moe_norm_quant(binding.norm_desc(H), x, self.d, None, T, x_out=x, stream=stream)
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
