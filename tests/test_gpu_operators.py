"""The operators around the expert block against plain 64-bit implementations.

Tolerances count roundings: half a step of the output type relative to the
value (bf16 2^-8, fp16 2^-11, e4m3 2^-4), and of the FP32 sums and functions
before it.
"""
import numpy as np
import pytest
import torch

import bit_grouped_gemm_gb300 as bg
from tests import parity

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_grouped_gemm_gb300 import build
    build.build()
    bg.load_library()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


# --------------------------------------------------------------------- norm
def norm_case(T, H, delta, group, weight=True, seed=0, x_pad=0, d_pad=0, o_pad=0, alpha=0.37,
              eps=1e-6, x=None, stream=None):
    """Runs the operator on padded rows; returns inputs and outputs as rows of H."""
    g = gen(seed)
    buf = lambda pad, dt: torch.zeros(T, H + pad, dtype=dt, device="cuda")
    xb = buf(x_pad, torch.bfloat16)
    xb[:, :H] = randn(g, T, H) if x is None else x
    d = None
    if delta:
        d = buf(d_pad, torch.float32 if delta == "f32" else torch.bfloat16)
        d[:, :H] = 2.0 * randn(g, T, H)
    w = (1.0 + 0.3 * randn(g, H)).bfloat16() if weight else None
    xo, xn = buf(x_pad, torch.bfloat16), buf(o_pad, torch.bfloat16)
    q = buf(o_pad, torch.uint8).view(torch.float8_e4m3fn)
    qs = torch.full((T, -(-H // 128) if group else 1), -1.0, device="cuda")
    desc = bg.norm_desc(H, eps=eps, alpha=alpha, delta_f32=delta == "f32",
                        quant_group=128 if group else 0, x_stride=H + x_pad,
                        delta_stride=H + d_pad, out_stride=H + o_pad)
    bg.moe_norm_quant(desc, xb, d, w, T, xo, xn, q, qs, stream)
    torch.cuda.synchronize()
    cut = lambda t: None if t is None else t[:, :H].double() if t.element_size() > 1 else t[:, :H].float().double()
    return dict(x=cut(xb), d=cut(d), w=None if w is None else w.double(), xo=cut(xo), xn=cut(xn),
                q=cut(q), qs=qs.double(), raw=(xo, xn, q), alpha=float(np.float32(alpha)),
                eps=float(np.float32(eps)))


def check_norm(r, H, group):
    e = r["x"] if r["d"] is None else r["x"] + r["alpha"] * r["d"]
    # x_out: one FP32 fused multiply-add and the bf16 rounding
    assert ((r["xo"] - e).abs() <= e.abs() * (2.0 ** -8 + 2 * U32) + 1e-38).all()
    v = r["xo"] / ((r["xo"] ** 2).mean(1, keepdim=True) + r["eps"]).sqrt()
    if r["w"] is not None:
        v = v * r["w"]
    # FP32 chain of v: the sum of squares (at most 64 terms a thread, 16 steps
    # across threads; halved by the root), the mean, eps, root, reciprocal and
    # two products
    chain = (0.5 * (64 + 16) + 6) * U32
    assert ((r["xn"] - v).abs() <= v.abs() * (2.0 ** -8 + chain) + 1e-38).all()
    step = 128 if group else H
    for i, c0 in enumerate(range(0, H, step)):
        p, s = v[:, c0:c0 + step], r["qs"][:, i]
        want = p.abs().amax(1) / 448.0
        assert ((s - want).abs() <= want * (chain + 2 * U32)).all()
        got = r["q"][:, c0:c0 + step] * s[:, None]
        # e4m3: half a step of the value, or of the smallest subnormal 2^-9
        tol = torch.maximum(p.abs() * 2.0 ** -4, s[:, None] * 2.0 ** -10)
        assert ((got - p).abs() <= tol * (1 + 2.0 ** -4) * (1 + 4 * chain) + p.abs() * 2 * chain).all()


@pytest.mark.parametrize("T,H", [(1, 2048), (1, 8), (3, 136), (5, 2056), (333, 5000), (2, 16384),
                                 (64, 4096), (1000, 256), (17, 8200), (4096, 2048)])
@pytest.mark.parametrize("delta", [None, "bf16", "f32"])
@pytest.mark.parametrize("group", [False, True])
def test_norm(T, H, delta, group):
    check_norm(norm_case(T, H, delta, group), H, group)


def test_norm_strides_keep_the_padding():
    r = norm_case(37, 520, "f32", True, x_pad=24, d_pad=8, o_pad=56, weight=False)
    check_norm(r, 520, True)
    for t in r["raw"]:
        assert (t[:, 520:].float() == 0).all()


def test_norm_empty_and_extreme_rows():
    H = 640
    x = torch.ones(6, H, device="cuda")
    x[0] = 0.0                       # zero row: scale and codes 0
    x[1] = 1e-30                     # v below 1e-26: still scaled
    x[2, 128:256] = 0.0              # one group of zeros
    x[3] = 3e4
    x[4, 7] = float("nan")
    x[5, 7] = float("inf")
    r = norm_case(6, H, None, True, x=x, weight=False)
    assert (r["qs"][0] == 0).all() and (r["q"][0] == 0).all() and (r["xn"][0] == 0).all()
    assert r["qs"][2, 1] == 0 and (r["q"][2, 128:256] == 0).all()
    ok = {k: (v[:4] if k in ("x", "xo", "xn", "q", "qs") else v) for k, v in r.items()}
    check_norm(ok, H, True)
    assert torch.isnan(r["xn"][4]).all() and torch.isnan(r["qs"][4]).all()
    assert torch.isnan(r["xn"][5, 7]) and (r["xn"][5, :7] == 0).all()
    assert torch.isnan(r["qs"][5, 0]) and (r["qs"][5, 1:] == 0).all()


def test_norm_in_place_and_partial_outputs():
    T, H = 19, 1024
    a = norm_case(T, H, "bf16", False, seed=3)
    g = gen(3)
    x = randn(g, T, H).bfloat16()
    d = (2.0 * randn(g, T, H)).bfloat16()
    w = (1.0 + 0.3 * randn(g, H)).bfloat16()
    desc = bg.norm_desc(H, alpha=0.37)
    bg.moe_norm_quant(desc, x, d, w, T, x_out=x)
    assert torch.equal(x.double(), a["xo"])
    xn = torch.zeros_like(x)
    bg.moe_norm_quant(desc, x, None, w, T, xn_out=xn)
    assert torch.equal(xn.double(), a["xn"])


# ------------------------------------------------------------------ routing
def ref_route(logits, bias, E, k, score, groups, topk_groups, renorm, scale):
    """Scores, choice and weights in numpy's 64 bits, one row at a time."""
    l = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64)) + 0.0
    T = l.shape[0]
    b = None if bias is None else np.where(np.isnan(bias), -np.inf, bias.astype(np.float64))
    idx, w = np.zeros((T, k), np.int64), np.zeros((T, k))
    with np.errstate(over="ignore", invalid="ignore"):
        for t in range(T):
            if score == "sigmoid":
                p = 1.0 / (1.0 + np.exp(-l[t]))
            else:
                m = l[t].max()
                p = np.exp(l[t] - m) / np.exp(l[t] - m).sum() if np.isfinite(m) else np.zeros(E)
            c = l[t] if b is None else p + b
            out = np.zeros(E, bool)
            if groups > 1:
                gc = (p if b is None else c).reshape(groups, -1)
                gs = -np.sort(-gc, axis=1)[:, :2].sum(1)
                best = np.argsort(-gs, kind="stable")[:topk_groups]
                out[:] = True
                for g in best:
                    out[g * (E // groups):(g + 1) * (E // groups)] = False
            order = np.lexsort((np.arange(E), -c, out))
            idx[t] = order[:k]
            q = p[idx[t]]
            if b is not None:
                q = np.where(np.isneginf(b[idx[t]]), 0.0, q)
            if renorm:
                q = q / q.sum() if q.sum() > 0 else np.zeros(k)
            w[t] = q * float(np.float32(scale))
    return idx, w


def ref_maps(idx, E):
    T, k = idx.shape
    flat = idx.reshape(-1)
    perm = np.argsort(flat, kind="stable")
    inv = np.empty_like(perm)
    inv[perm] = np.arange(T * k)
    counts = np.bincount(flat, minlength=E)
    off = np.concatenate([[0], np.cumsum(counts)])
    toff = np.concatenate([[0], np.cumsum(-(-counts // 128))])
    bmap = [(e, off[e] + r, min(128, counts[e] - r)) for e in range(E)
            for r in range(0, counts[e], 128)]
    return dict(counts=counts, offsets=off, tile_offsets=toff, perm=perm, inv=inv,
                block_map=np.array(bmap).reshape(-1, 3))


def route(logits, E, k, stream=None, max_tokens=None, **kw):
    T = logits.shape[0]
    plan = bg.moe_plan_create(bg.plan_desc(hidden=256, inter=256, num_experts=E, top_k=k,
                                           max_tokens=max_tokens or T), 0)
    try:
        r = bg.moe_route_scored(plan, logits, T, bg.score_desc(**kw), None, stream)
        out = parity.routing_to_numpy(r, T, k, E)
        assert bg.moe_get_error(plan) == 0
        return out
    finally:
        bg.moe_plan_destroy(plan)


def check_route(logits, E, k, bias=None, score="sigmoid", groups=1, topk_groups=1, renorm=True,
                scale=1.0, **kw):
    got = route(logits, E, k, bias=bias, score=score, groups=groups, topk_groups=topk_groups,
                renormalise=renorm, scale=scale, **kw)
    ln = logits.cpu().numpy()
    bn = None if bias is None else bias.cpu().numpy()
    idx, w = ref_route(ln, bn, E, k, score, groups, topk_groups, renorm, scale)
    assert np.array_equal(got["topk_idx"], idx)
    # FP32: exponential 2 ulp, its argument's difference half an ulp of a value
    # up to the logits' spread, sums of k or E / 32 + 5 terms, a division
    fin = ln[np.isfinite(ln)]
    spread = float(fin.max() - fin.min()) if fin.size else 0.0
    rel = (2 * (8 + min(spread, 100.0)) + k + 32) * U32
    assert (np.abs(got["topk_w"] - w) <= np.abs(w) * rel + 1e-37).all()
    for n, v in ref_maps(idx, E).items():
        assert np.array_equal(got[n], v), n
    return got


@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (2, 8, 1), (7, 24, 5), (31, 96, 6), (32, 256, 8),
                                   (33, 160, 32), (777, 512, 10), (1000, 256, 8), (5000, 64, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route(T, E, k, score, biased):
    g = gen(T + E)
    logits = randn(g, T, E)
    bias = 0.1 * randn(g, E) if biased else None
    check_route(logits, E, k, bias=bias, score=score, renorm=True, scale=2.5)
    check_route(logits, E, k, bias=bias, score=score, renorm=False)


@pytest.mark.parametrize("E,k,groups,tg", [(256, 8, 8, 4), (256, 8, 8, 1), (256, 8, 8, 8),
                                           (160, 6, 8, 3), (96, 4, 4, 2), (512, 10, 32, 9),
                                           (24, 2, 24, 5), (16, 2, 8, 1), (512, 8, 2, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_groups(E, k, groups, tg, score, biased):
    g = gen(E + groups)
    logits = randn(g, 300, E)
    bias = 0.05 * randn(g, E) if biased else None
    check_route(logits, E, k, bias=bias, score=score, groups=groups, topk_groups=tg)


def test_route_long():
    g = gen(5)
    logits, bias = randn(g, 9001, 512), 0.01 * randn(g, 512)
    check_route(logits, 512, 10, bias=bias, score="softmax", renorm=False)


def test_route_beyond_a_byte_per_cta():
    """More tokens than the counts' byte table takes."""
    g = gen(7)
    check_route(randn(g, 36001, 32), 32, 3, bias=0.1 * randn(g, 32), score="sigmoid")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,tg", [(1, 1), (8, 4)])
def test_route_scores_that_32_bits_cannot_order(score, groups, tg):
    """The bias cancels the score down to the bias' own rounding (1e-8 and
    less), so FP32 sums cannot order the experts; 64-bit ones can."""
    T, E, k = 64, 256, 8
    g = gen(11)
    row = randn(g, E)
    l = row.cpu().numpy().astype(np.float64)
    p = 1 / (1 + np.exp(-l)) if score == "sigmoid" else np.exp(l - l.max()) / np.exp(l - l.max()).sum()
    bias = torch.from_numpy((0.5 - p).astype(np.float32)).cuda()
    check_route(row.repeat(T, 1), E, k, bias=bias, score=score, groups=groups, topk_groups=tg)


@pytest.mark.parametrize("E,groups,tg", [(256, 1, 1), (256, 8, 4), (320, 5, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_ties_go_to_the_lower_index(E, groups, tg, score, biased):
    g = gen(2)
    logits = torch.randint(-2, 3, (70, E), generator=g, device="cuda").float()
    logits[0] = 0.0
    logits[1] = -0.0
    logits[2, ::2] = -0.0
    logits[2, 1::2] = 0.0
    bias = torch.randint(0, 2, (E,), generator=g, device="cuda").float() if biased else None
    check_route(logits, E, 8, bias=bias, score=score, groups=groups, topk_groups=tg)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_masks_and_extremes(score, biased):
    T, E, k = 40, 64, 6
    g = gen(4)
    logits = randn(g, T, E)
    low = torch.finfo(torch.float32).min
    logits[0] = float("-inf")                  # an empty row
    logits[1, 3:] = float("-inf")              # fewer live experts than k
    logits[2] = low
    logits[3, 5:] = low
    logits[4] = float("nan")
    logits[5, ::3] = float("nan")
    logits[6] = -90.0 + randn(g, E)            # far below zero
    logits[7] = 60.0 + randn(g, E)
    logits[8, 0] = 88.0
    bias = None
    if biased:
        bias = 0.1 * randn(g, E)
        bias[::2] = float("-inf")              # closed experts
        bias[1] = float("nan")
    check_route(logits, E, k, bias=bias, score=score)


def test_route_all_but_few_closed():
    g = gen(9)
    E, k = 32, 8
    bias = torch.full((E,), float("-inf"), device="cuda")
    bias[[4, 9, 30]] = 0.1
    got = check_route(randn(g, 50, E), E, k, bias=bias, score="sigmoid")
    assert set(got["topk_idx"][:, :3].reshape(-1)) == {4, 9, 30}
    assert (got["topk_w"][:, 3:] == 0).all()
    bias[:] = float("-inf")
    got = check_route(randn(g, 5, E), E, k, bias=bias, score="softmax")
    assert (got["topk_w"] == 0).all()


def test_route_into_callers_buffers_and_repeat():
    T, E, k = 333, 256, 8
    g = gen(6)
    logits, bias = randn(g, T, E), 0.1 * randn(g, E)
    want = check_route(logits, E, k, bias=bias, groups=8, topk_groups=4)
    bufs, r = parity.caller_routing_buffers(T, k, E)
    plan = bg.moe_plan_create(bg.plan_desc(hidden=256, inter=256, num_experts=E, top_k=k,
                                           max_tokens=500), 0)
    d = bg.score_desc(score="sigmoid", bias=bias, groups=8, topk_groups=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for b in bufs.values():
            b.zero_()
        side.wait_stream(torch.cuda.current_stream())
        bg.moe_route_scored(plan, logits, T, d, r, side)
        got = parity.routing_to_numpy(r, T, k, E)
        for n in want:
            if n != "logits":
                assert np.array_equal(got[n], want[n]), n
    bg.moe_plan_destroy(plan)


def test_route_refusals_with_a_plan():
    import ctypes
    lib = bg.load_library()
    plan = bg.moe_plan_create(bg.plan_desc(hidden=256, inter=256, num_experts=64, top_k=8,
                                           max_tokens=16), 0)
    logits = torch.zeros(17, 64, device="cuda")

    def call(T=4, ptr=None, null_desc=False, **kw):
        d = bg.score_desc(score="sigmoid")
        for n, v in kw.items():
            setattr(d, n, v)
        r = bg.MoeRouting()
        return lib.moe_route_scored(plan, logits.data_ptr() if ptr is None else ptr, T,
                                    None if null_desc else ctypes.byref(d), ctypes.byref(r), None)
    assert call() == 0
    assert call(T=0) == 1 and call(T=17) == 4 and call(null_desc=True) == 1
    assert call(ptr=logits.data_ptr() + 4) == 1
    assert call(score=2) == 1 and call(score=-1) == 1 and call(renormalise=2) == 1
    assert call(groups=0) == 1 and call(groups=3) == 1 and call(groups=64) == 1
    assert call(groups=8, topk_groups=9) == 1 and call(groups=8, topk_groups=0) == 1
    assert call(groups=16, topk_groups=1) == 1        # 4 experts for k = 8
    assert call(groups=16, topk_groups=2) == 0
    assert call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(bias=logits.data_ptr() + 2) == 1
    torch.cuda.synchronize()
    bg.moe_plan_destroy(plan)


def test_router_logits_are_those_of_the_routing():
    g = gen(8)
    for T in (3, 200):
        x = randn(g, T, 512).bfloat16()
        w = (0.05 * randn(g, 512, 64)).bfloat16()
        b = randn(g, 64)
        plan = bg.moe_plan_create(bg.plan_desc(hidden=512, inter=256, num_experts=64, top_k=4,
                                               max_tokens=T), 0)
        out = torch.zeros(T, 64, device="cuda")
        bg.moe_router_logits(plan, x, T, w, b, out)
        r = bg.moe_route(plan, x, T, w, b)
        same = parity.routing_to_numpy(r, T, 4, 64)["logits"]
        assert np.array_equal(out.cpu().numpy(), same)
        bg.moe_plan_destroy(plan)


# --------------------------------------------------------------- projection
def w4_case(g, N, K):
    q = torch.randint(-(1 << 31), 1 << 31, (N, K // 8), generator=g, device="cuda",
                      dtype=torch.int64).to(torch.int32)
    s = (0.005 + 0.015 * torch.rand(N, K // 64, generator=g, device="cuda")).bfloat16()
    b = (-8.0 * s.float() + 1e-2 * randn(g, N, K // 64)).bfloat16()
    return q, s, b


def w4_values(q, s, b):
    N, K = q.shape[0], q.shape[1] * 8
    nib = torch.stack([(q.long() >> (4 * i)) & 15 for i in range(8)], 2).reshape(N, K).double()
    return nib * s.double().repeat_interleave(64, 1) + b.double().repeat_interleave(64, 1)


class Linear:
    """One projection's inputs on the GPU, and its outputs in 64 bits."""

    def __init__(self, T, K, N, x="bf16", rank=0, n=4, ids="mixed", seed=0, x_pad=0, y_pad=0,
                 scaled=True, lscale=True):
        g = gen(seed)
        self.T, self.K, self.N, self.rank = T, K, N, rank
        xv = randn(g, T, K)
        self.xs = None
        if x == "e4m3":
            self.xs = xv.abs().amax(1) / 448.0 if scaled else None
            xv = (xv / (self.xs[:, None] if scaled else 1.0)).to(torch.float8_e4m3fn)
            self.x = torch.zeros(T, K + x_pad, dtype=torch.uint8, device="cuda")
            self.x[:, :K] = xv.view(torch.uint8)
            self.x = self.x.view(torch.float8_e4m3fn)
        else:
            self.x = torch.zeros(T, K + x_pad, dtype=torch.bfloat16, device="cuda")
            self.x[:, :K] = xv
        self.w = w4_case(g, N, K)
        self.lora = self.ids = None
        if rank:
            self.a = (randn(g, n, rank, K) / K ** 0.5).bfloat16()
            self.b = (0.3 * randn(g, n, N, rank)).bfloat16()
            self.ls = 0.5 + torch.rand(n, generator=g, device="cuda") if lscale else None
            self.lora = bg.lora(self.a, self.b, self.ls)
            if ids == "mixed":
                self.ids = torch.randint(-1, n, (T,), generator=g, device="cuda")
            elif ids == "runs":
                self.ids = (torch.arange(T, device="cuda") * (n + 1) // T) - 1
            else:
                self.ids = torch.tensor(ids, device="cuda").repeat(-(-T // len(ids)))[:T]
            self.ids = self.ids.to(torch.int32)
        self.y = torch.full((T, N + y_pad), 7.0, dtype=torch.bfloat16, device="cuda")
        self.x_pad, self.y_pad = x_pad, y_pad

    def run(self, stream=None, max_tokens=None, handle=None):
        h = handle or bg.moe_linear_create(
            bg.linear_desc(self.K, self.N, max_tokens or self.T, self.rank), 0)
        try:
            bg.moe_linear_forward(h, self.x, self.T, bg.w4(*self.w), self.y, x_scale=self.xs,
                                  lora=self.lora, adapter=self.ids,
                                  x_stride=self.K + self.x_pad, y_stride=self.N + self.y_pad,
                                  stream=stream)
            torch.cuda.synchronize()
            return bg.moe_linear_get_error(h)
        finally:
            if handle is None:
                bg.moe_linear_destroy(h)

    def check(self, status=0):
        assert self.run() == status
        self.compare()

    def compare(self):
        x = self.x[:, :self.K].float().double()
        w = w4_values(*self.w)
        y = x @ w.T
        size = x.abs() @ w.abs().T                 # sum of the products' sizes
        lsize = torch.zeros_like(size)
        if self.lora is not None:
            for i in range(self.a.shape[0]):
                rows = (self.ids == i).nonzero().flatten()
                if rows.numel() == 0:
                    continue
                sc = 1.0 if self.ls is None else float(self.ls[i].double())
                a, b = self.a[i].double(), self.b[i].double()
                y[rows] += sc * (x[rows] @ a.T) @ b.T
                lsize[rows] += sc * (x[rows].abs() @ a.abs().T) @ b.abs().T
        if self.xs is not None:
            y, size, lsize = (t * self.xs.double()[:, None] for t in (y, size, lsize))
        got = self.y[:, :self.N].double()
        # weights rounded to fp16; FP32 sums over K (and the rank); x A^T kept
        # to 16 bits; the output's bf16
        K, r = self.K, self.rank
        tol = (y.abs() * 2.0 ** -8 * (1 + 2.0 ** -7) + size * (2.0 ** -11 + 2 * K * U32)
               + lsize * (2.0 ** -16 + 2 * (K + r) * U32) + 1e-30)
        bad = (got - y).abs() > tol
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst " \
                              f"{float(((got - y).abs() / tol).max()):.2f} x its tolerance"
        # the roundings are independent: together within half a step of bf16
        assert float((got - y).pow(2).mean().sqrt()) <= 2.0 ** -8 * float(y.pow(2).mean().sqrt()) + 1e-30
        if self.y_pad:
            assert (self.y[:, self.N:] == 7.0).all()


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 64, 65, 127, 128, 129, 257, 300, 700])
@pytest.mark.parametrize("K,N", [(2048, 512), (320, 200)])
def test_linear_tokens(T, K, N):
    Linear(T, K, N, rank=16).check()
    Linear(T, K, N, x="e4m3", rank=8, ids="runs").check()


@pytest.mark.parametrize("K", [64, 128, 192, 256, 1088, 4096])
@pytest.mark.parametrize("N", [1, 8, 100, 127, 129, 255, 1000])
@pytest.mark.parametrize("T", [3, 150])
def test_linear_odd_sizes(K, N, T):
    Linear(T, K, N, rank=8, y_pad=3, x_pad=16).check()


@pytest.mark.parametrize("rank", [8, 16, 24, 40, 64, 128])
@pytest.mark.parametrize("T", [5, 40, 260])
def test_linear_ranks(rank, T):
    Linear(T, 512, 384, rank=rank, n=3).check()
    Linear(T, 512, 384, rank=rank, n=3, ids="runs", lscale=False, x="e4m3").check()


@pytest.mark.parametrize("T", [4, 16, 48, 300])
def test_linear_without_adapters(T):
    Linear(T, 1024, 640).check()
    Linear(T, 1024, 640, x="e4m3").check()
    Linear(T, 1024, 640, x="e4m3", scaled=False).check()
    Linear(T, 1024, 640, rank=16, ids=[-1]).check()
    Linear(T, 1024, 640, rank=16, ids=[-5, 99, 4, 2 ** 31 - 1]).check()     # none of them exists


@pytest.mark.parametrize("T,n", [(16, 16), (100, 70), (256, 256), (600, 300)])
def test_linear_many_adapters(T, n):
    Linear(T, 256, 264, rank=8, n=n).check()


def test_linear_large():
    Linear(4096, 2048, 2048, rank=32, n=8, ids="runs").check()
    Linear(1031, 2048, 4096, x="e4m3", rank=16, n=8, ids="runs").check()


@pytest.mark.parametrize("T", [2047, 2049, 4500])
def test_linear_orders_mixed_blocks_of_tokens(T):
    # more adapters than bins, tokens without one, runs and random order block by block
    Linear(T, 192, 136, rank=8, n=300).check()
    g = gen(3)
    mixed = torch.randint(-2, 6, (2048,), generator=g, device="cuda").tolist()
    runs = [i // 300 for i in range(2048)]
    Linear(T, 128, 72, x="e4m3", rank=24, ids=runs + mixed, x_pad=16, y_pad=3).check()
    Linear(T, 128, 72, x="e4m3", rank=24, ids=mixed + runs).check()


def test_linear_mixed_then_runs_on_one_handle():
    h = bg.moe_linear_create(bg.linear_desc(256, 320, 4200, 16), 0)
    for T, ids in ((4200, "mixed"), (300, "runs"), (4100, "runs"), (90, "mixed"), (2100, "mixed")):
        c = Linear(T, 256, 320, rank=16, n=9, ids=ids)
        assert c.run(handle=h) == 0
        c.compare()
        first = c.y.clone()
        assert c.run(handle=h) == 0
        assert torch.equal(c.y, first)
    bg.moe_linear_destroy(h)


@pytest.mark.parametrize("T", [3, 40, 200])
def test_linear_repeats_bit_for_bit_on_one_handle(T):
    c = Linear(T, 1024, 1000, rank=16)
    h = bg.moe_linear_create(bg.linear_desc(1024, 1000, 512, 64), 0)
    assert c.run(handle=h) == 0
    c.compare()
    first = c.y.clone()
    other = Linear(97, 1024, 1000, x="e4m3", rank=64, seed=5)
    assert other.run(handle=h) == 0
    other.compare()
    side = torch.cuda.Stream()
    for _ in range(3):
        c.y.zero_()
        side.wait_stream(torch.cuda.current_stream())
        assert c.run(handle=h, stream=side) == 0
        assert torch.equal(c.y, first)
    bg.moe_linear_destroy(h)


@pytest.mark.parametrize("T", [2, 24, 200])
def test_linear_in_a_graph(T):
    c = Linear(T, 1024, 512, rank=16)
    h = bg.moe_linear_create(bg.linear_desc(1024, 512, T, 16), 0)
    assert c.run(handle=h) == 0
    first = c.y.clone()
    graph, w = torch.cuda.CUDAGraph(), bg.w4(*c.w)
    with torch.cuda.graph(graph):
        bg.moe_linear_forward(h, c.x, T, w, c.y, lora=c.lora, adapter=c.ids)
        bg.moe_linear_forward(h, c.x, T, w, c.y, lora=c.lora, adapter=c.ids)
    for _ in range(3):
        c.y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.y, first)
    # new rows and ids in place are seen by the next replay
    c.x.copy_(c.x.flip(0))
    c.ids.copy_(c.ids.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    c.compare()
    assert bg.moe_linear_get_error(h) == 0
    bg.moe_linear_destroy(h)


@pytest.mark.parametrize("T", [6, 40, 300])
@pytest.mark.parametrize("ids", ["mixed", "runs"])
def test_linear_keeps_broken_adapters_to_their_own_tokens(T, ids):
    clean = Linear(T, 256, 200, rank=16, n=4, ids=ids)
    assert clean.run() == 0
    c = Linear(T, 256, 200, rank=16, n=4, ids=ids)
    c.b[1, 5, 3], c.b[1, 77, 0], c.b[1, 150] = float("nan"), float("inf"), float("-inf")
    c.a[2, 4, 9], c.a[2, 0] = float("nan"), float("inf")
    c.ls[3] = float("nan")
    assert c.run() == 0
    rows = (c.ids <= 0)
    assert rows.any() and torch.equal(c.y[rows], clean.y[rows])
    # and a token whose scale is not a number
    e = Linear(T, 256, 200, x="e4m3", rank=16, n=4, ids=ids)
    assert e.run() == 0
    first = e.y.clone()
    e.xs[1] = float("nan")
    assert e.run() == 0
    assert torch.isnan(e.y[1]).all()
    keep = torch.arange(T, device="cuda") != 1
    assert torch.equal(e.y[keep], first[keep])


@pytest.mark.parametrize("T", [1, 200])
def test_linear_flags_values_beyond_the_operands(T):
    c = Linear(T, 256, 128)
    c.x[T - 1, 9] = 1e6
    assert c.run() == 6                            # MOE_ERR_OPERAND_RANGE
    c = Linear(T, 256, 128)
    c.w[1][5, 1] = 3e-6
    assert c.run() == 6


def test_linear_refusals_with_a_handle():
    import ctypes
    lib = bg.load_library()
    c = Linear(4, 256, 128, rank=8)
    h = bg.moe_linear_create(bg.linear_desc(256, 128, 8, 16), 0)
    w = bg.w4(*c.w)
    p = lambda t: t.data_ptr()

    def call(x=None, xt=0, xld=0, xs=None, T=4, wt=w, lora=c.lora, ids=p(c.ids), y=None, yld=0):
        return lib.moe_linear_forward(h, p(c.x) if x is None else x, xt, xld, xs, T,
                                      ctypes.byref(wt), None if lora is None else ctypes.byref(lora),
                                      ids, p(c.y) if y is None else y, yld, None)
    assert call() == 0
    assert call(T=0) == 1 and call(T=9) == 4
    assert call(x=0) == 1 and call(x=p(c.x) + 2) == 1 and call(y=0) == 1 and call(y=p(c.y) + 1) == 1
    assert call(xt=2) == 1 and call(xs=p(c.y)) == 1
    assert call(xld=248) == 1 and call(xld=264) == 1 and call(yld=127) == 1
    assert call(lora=None) == 1 and call(ids=None) == 1 and call(lora=None, ids=None) == 0
    assert call(wt=bg.MoeW4(None, w.scales, w.biases)) == 1
    assert call(wt=bg.MoeW4(w.qweight, w.scales + 2, w.biases)) == 1
    L = lambda **kw: [setattr(l := bg.lora(c.a, c.b, c.ls), k, v) for k, v in kw.items()] and l
    assert call(lora=L(rank=12)) == 1 and call(lora=L(rank=24)) == 4 and call(lora=L(rank=0)) == 1
    assert call(lora=L(n=0)) == 1 and call(lora=L(n=65537)) == 2 and call(lora=L(a=None)) == 1
    assert call(lora=L(b=p(c.b) + 2)) == 1
    assert call(y=p(c.x)) == 1                       # output over the input
    torch.cuda.synchronize()
    bg.moe_linear_destroy(h)


# ------------------------------------------------------- long and far offsets
def test_norm_beyond_31_bits():
    """More than 2^31 elements per tensor; the last rows are checked."""
    H, T = 16384, (1 << 31) // 16384 + 40
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    tail = slice(T - 24, T)
    x[tail] = randn(gen(1), 24, H)
    xo, xn = torch.empty_like(x), torch.empty_like(x)
    q = torch.empty(T, H, dtype=torch.float8_e4m3fn, device="cuda")
    qs = torch.empty(T, 128, device="cuda")
    bg.moe_norm_quant(bg.norm_desc(H, quant_group=128), x, None, None, T, xo, xn, q, qs)
    torch.cuda.synchronize()
    r = dict(x=x[tail].double(), d=None, w=None, xo=xo[tail].double(), xn=xn[tail].double(),
             q=q[tail].float().double(), qs=qs[tail].double(), alpha=1.0, eps=float(np.float32(1e-6)))
    check_norm(r, H, True)


@pytest.mark.parametrize("T", [9, 40])
def test_linear_rows_far_apart(T):
    """Row strides that put the last rows beyond 2^31 elements."""
    c = Linear(T, 128, 64, rank=8)
    ld = ((1 << 31) // (T - 1) + 64) // 16 * 16
    xs = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
    ys = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
    xs.view(T, ld)[:, :128] = c.x
    h = bg.moe_linear_create(bg.linear_desc(128, 64, T, 8), 0)
    bg.moe_linear_forward(h, xs, T, bg.w4(*c.w), ys, lora=c.lora, adapter=c.ids, x_stride=ld,
                          y_stride=ld)
    torch.cuda.synchronize()
    assert bg.moe_linear_get_error(h) == 0
    c.y = ys.view(T, ld)[:, :64].clone()
    c.compare()
    bg.moe_linear_destroy(h)


@pytest.mark.parametrize("T,K,N,rank,x", [
    (7100, 64, 72, 8, "bf16"), (7100, 64, 71, 0, "e4m3"), (2300, 128, 8, 64, "bf16"), (1500, 320, 201, 24, "e4m3"),
    (700, 1088, 999, 40, "bf16"), (520, 2048, 264, 16, "e4m3"), (257, 2048, 1032, 16, "bf16"),
    (150, 4096, 1000, 24, "e4m3"), (65, 4096, 4104, 16, "bf16"), (40, 4096, 4104, 0, "bf16")])
def test_linear_odd_sizes_beyond_decode_batches(T, K, N, rank, x):
    Linear(T, K, N, x=x, rank=rank, n=11, x_pad=16, y_pad=3).check()
    Linear(T, K, N, x=x, rank=rank, n=5, ids="runs", y_pad=8).check()


@pytest.mark.parametrize("ids", ["mixed", "runs"])
def test_linear_keeps_broken_adapters_apart_in_large_batches(ids):
    test_linear_keeps_broken_adapters_to_their_own_tokens(2500, ids)


def test_linear_large_batch_in_a_graph():
    test_linear_in_a_graph(1200)


def test_linear_flags_values_in_a_large_batch():
    test_linear_flags_values_beyond_the_operands(5000)


def test_linear_rows_far_apart_in_a_large_batch():
    test_linear_rows_far_apart(3000)


def test_linear_small_sizes_of_many_tokens():
    # several CTAs of tokens on the decode batches' kernels
    for T in (33, 40, 41, 63, 96, 129, 250):
        Linear(T, 256, 72, rank=24, n=5, y_pad=1, x_pad=32).check()
        Linear(T, 512, 1000, x="e4m3", rank=8).check()
        Linear(T, 1024, 264).check()


# --------------------------------------------------------------- all together
@pytest.mark.parametrize("T", [1, 5, 96])
def test_adapted_layer(T):
    """The operators in the order in which a served layer calls them, each
    step's output against the 64-bit step on the library's own input to it."""
    import dataclasses
    from bit_grouped_gemm_gb300 import stack, synth
    shape = synth.MoEShape(hidden=256, inter=256, num_experts=32, top_k=4)
    w = dataclasses.replace(synth.standard_workloads()["t128_uniform"], shape=shape, tokens=T)
    g = gen(T)
    H, E, k = 256, 32, 4
    L = stack.make_layer(w, 0, "cuda")
    proj = w4_case(g, H, H)
    a, b = (randn(g, 3, 16, H) / 16).bfloat16(), (0.3 * randn(g, 3, H, 16)).bfloat16()
    bias = 0.05 * randn(g, E)
    score = bg.score_desc("sigmoid", bias, groups=4, topk_groups=2, scale=1.5)
    n1, n2 = ((1 + 0.2 * randn(g, H)).bfloat16() for _ in range(2))
    plan = bg.moe_plan_create(bg.plan_desc(hidden=H, inter=256, num_experts=E, top_k=k,
                                           max_tokens=T), 0)
    layer = stack.AdaptedLayer(plan, L, n1, n2, proj, score, bg.lora(a, b), max_tokens=T, alpha=0.5)
    x0 = randn(g, T, H).bfloat16()
    y0 = randn(g, T, H)
    ids = torch.randint(-1, 3, (T,), generator=g, device="cuda").to(torch.int32)
    x = x0.clone()
    y = layer(x, y0, ids).double()
    torch.cuda.synchronize()
    assert bg.moe_get_error(plan) == 0 and bg.moe_linear_get_error(layer.linear) == 0
    # stream after the first norm, from its own rounding
    x1 = (x0.double() + 0.5 * y0.double()).float().bfloat16().double()
    d = layer.d[:T].double()
    want = x1 + d
    assert ((x.double() - want).abs() <= want.abs() * 2.0 ** -8 + x1.abs() * 2.0 ** -8 + 1e-30).all()
    # projection on the 8-bit rows
    c = Linear(T, H, H)
    c.x, c.xs, c.w, c.rank = layer.h8[:T], layer.hs[:T, 0], proj, 16
    c.lora, c.a, c.b, c.ls, c.ids, c.y = True, a, b, None, ids, layer.d[:T]
    c.compare()
    # routing on the library's logits, then the experts on that routing
    logits = layer.logits[:T].cpu().numpy()
    idx, wt = ref_route(logits, bias.cpu().numpy(), E, k, "sigmoid", 4, 2, True, 1.5)
    got = parity.routing_to_numpy(bg.moe_route_scored(plan, layer.logits, T, score), T, k, E)
    assert np.array_equal(got["topk_idx"], idx)
    xf = layer.xn[:T].double()

    def expert(sets, e, row):
        gate, up, down = (w4_values(*[m[e] for m in sets[n]]) for n in ("gate", "up", "down"))
        u = gate @ row
        return down @ (u / (1 + torch.exp(-u)) * (up @ row))
    rows = list(range(T) if T <= 5 else range(0, T, 24))
    ref = []
    for t in rows:
        out = expert(L.shared, 0, xf[t])
        for j in range(k):
            out = out + float(wt[t, j]) * expert(L.routed, int(idx[t, j]), xf[t])
        ref.append(out)
    parity.check_y(y[rows].cpu().numpy(), torch.stack(ref).cpu().numpy())
    layer.close()
    bg.moe_plan_destroy(plan)
