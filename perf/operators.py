"""The operators of a layer around the expert block, as cases that can be timed.

Three operators, in the order in which a served pre-norm layer calls them:

* ``norm``: the residual's addition and RMS norm, with the normalised row in
  bf16 and in 8 bits (e4m3) with its scales;
* ``linear``: a projection with shared 4-bit affine weights and, beside it,
  the low-rank adapters of many requests at once;
* ``route``: a router's choice of experts from its logits: softmax or sigmoid
  scores, a bias for balance, groups, top-k, renormalised weights, and the
  maps that the grouped expert GEMM reads.

``run`` computes each one in elementary torch operations, or, where ``own`` is
set, through this repository's library.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 64          # quantisation group of the 4-bit weights along K
QGROUP = 128        # columns per scale of the grouped 8-bit output
TILE = 128          # rows per tile of the expert GEMM's block map
E4M3_MAX = 448.0
EPS = 1e-6


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decoded token's row: the projection's bf16 output joins the stream
        dict(name="norm_token", op="norm", T=1, H=2048, delta="bf16", quant="row", weight=True),
        # a prompt chunk after the expert block: its fp32 output joins the stream
        dict(name="norm_prompt", op="norm", T=4096, H=2048, delta="f32", quant="row", weight=True),
        # a mixed batch of an odd size, a width that ends inside a scale's group
        dict(name="norm_ragged", op="norm", T=333, H=5000, delta="bf16", quant="group", weight=True),
        # the long prompt: 16k rows of a wider stream
        dict(name="norm_long", op="norm", T=16384, H=4096, delta="bf16", quant="group", weight=True),
        # one decoded token: sigmoid scores with a balance bias, 4 of 8 groups
        dict(name="route_token", op="route", T=1, E=256, k=8, score="sigmoid", bias=True,
             groups=8, topk_groups=4, renorm=True, scale=2.5, closed=0),
        # a mixed batch, softmax scores, no bias, some experts masked by -inf logits
        dict(name="route_ragged", op="route", T=777, E=96, k=6, score="softmax", bias=False,
             groups=1, topk_groups=1, renorm=True, scale=1.0, closed=7),
        # a prompt chunk: sigmoid, bias, groups
        dict(name="route_prompt", op="route", T=4096, E=256, k=8, score="sigmoid", bias=True,
             groups=8, topk_groups=4, renorm=True, scale=2.5, closed=0),
        # the long prompt, softmax scores with a bias over more experts
        dict(name="route_long", op="route", T=16384, E=512, k=10, score="softmax", bias=True,
             groups=1, topk_groups=1, renorm=False, scale=1.0, closed=0),
        # one decoded token with its adapter
        dict(name="linear_token", op="linear", T=1, K=2048, N=2048, x="bf16", rank=16,
             adapters=16, order="mixed"),
        # a decode batch: 16 requests, each with an adapter of its own or none, 8-bit rows
        dict(name="linear_decode", op="linear", T=16, K=2048, N=2048, x="e4m3", rank=16,
             adapters=16, order="mixed"),
        # a ragged batch of prompts and odd sizes
        dict(name="linear_ragged", op="linear", T=333, K=1088, N=1000, x="bf16", rank=8,
             adapters=5, order="runs"),
        # a prompt chunk of several requests, 8-bit rows from the norm
        dict(name="linear_prompt", op="linear", T=4096, K=2048, N=4096, x="e4m3", rank=32,
             adapters=8, order="runs"),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v))


def _plain_size(v):
    """Sizes next to 3 * 2^10 are moved off it."""
    return v + 8 if v == 3 << 10 else v


def draw(rng):
    op = rng.choice(("norm", "route", "linear"))
    if op == "norm":
        H = _plain_size(8 * _log_int(rng, 16, 1024))
        T = _plain_size(_log_int(rng, 1, min(16384, (16384 * 4096) // H)))
        return dict(op="norm", T=T, H=H, delta=rng.choice(("bf16", "f32", "none")),
                    quant=rng.choice(("row", "group", "none")), weight=rng.random() < 0.8)
    if op == "route":
        E = 8 * rng.choice((4, 8, 12, 16, 20, 32, 48, 64))
        T = _plain_size(_log_int(rng, 1, 16384))
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0])
        k = rng.randint(1, 10)
        tg = 1 if groups == 1 else rng.randint(1, groups)
        while tg * (E // groups) < k:
            tg += 1
        return dict(op="route", T=T, E=E, k=k, score=rng.choice(("sigmoid", "softmax")),
                    bias=rng.random() < 0.6, groups=groups, topk_groups=tg,
                    renorm=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)),
                    closed=rng.choice((0, 0, 3)))
    while True:
        K = _plain_size(GROUP * _log_int(rng, 2, 64))
        N = _plain_size(_log_int(rng, 64, 4096))
        T = _plain_size(_log_int(rng, 1, 4096))
        if T * K * N <= 4096 * 2048 * 4096:
            break
    return dict(op="linear", T=T, K=K, N=N, x=rng.choice(("bf16", "e4m3")),
                rank=8 * rng.choice((1, 2, 4, 8)), adapters=rng.randint(1, 16),
                order=rng.choice(("runs", "mixed")))


# --------------------------------------------------------------- the inputs
class _Handle:
    """A library handle that is given back when its state is dropped."""

    def __init__(self, value, destroy):
        self.value, self.destroy = value, destroy

    def __del__(self):
        self.destroy(self.value)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def prepare(case, seed):
    g = _gen(seed)
    s = _prepare_inputs(case, g)
    s["case"] = case
    if own:
        _prepare_own(case, s)
    return s


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _prepare_inputs(case, g):
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        # a residual stream: unit rows, a few channels that stand out, as trained models have
        x = _randn(g, T, H)
        x[:, :: max(1, H // 4)] *= 20.0
        d = None
        if case["delta"] != "none":
            d = _randn(g, T, H) * 3.0
            d = d.bfloat16() if case["delta"] == "bf16" else d
        w = (1.0 + 0.2 * _randn(g, H)).bfloat16() if case["weight"] else None
        return dict(x=x.bfloat16(), delta=d, weight=w, alpha=0.158 if d is not None else 0.0)
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        # logits of an RMS-normed row on a router weight of small entries; some experts are
        # favoured, as in a router without perfect balance
        logits = 0.9 * _randn(g, T, E) + 0.5 * _randn(g, E)
        if case["closed"]:
            shut = torch.randperm(E, generator=g, device=DEV)[: case["closed"]]
            logits[:, shut] = float("-inf")
        spread = 0.1 if case["score"] == "sigmoid" else 0.002
        bias = spread * _randn(g, E) if case["bias"] else None
        return dict(logits=logits, bias=bias)
    T, K, N, r, n = case["T"], case["K"], case["N"], case["rank"], case["adapters"]
    x = _randn(g, T, K)
    xs = None
    if case["x"] == "e4m3":
        xs = x.abs().amax(1) / E4M3_MAX
        x = (x / xs[:, None]).to(torch.float8_e4m3fn)
    else:
        x = x.bfloat16()
    q = torch.randint(-(1 << 31), 1 << 31, (N, K // 8), generator=g, device=DEV,
                      dtype=torch.int64).to(torch.int32)
    sc = (0.005 + 0.015 * torch.rand(N, K // GROUP, generator=g, device=DEV)).bfloat16()
    zb = (-8.0 * sc.float() + 1e-3 * _randn(g, N, K // GROUP)).bfloat16()
    a = (_randn(g, n, r, K) / math.sqrt(K)).bfloat16()
    b = (0.1 * _randn(g, n, N, r)).bfloat16()
    lscale = 0.5 + 1.5 * torch.rand(n, generator=g, device=DEV)
    # requests in runs of tokens (prompts) or one per token (decode); -1: no adapter
    if case["order"] == "runs":
        runs = min(T, 2 * n)
        cut = torch.arange(T, device=DEV) * runs // T
        ids = torch.randint(-1, n, (runs,), generator=g, device=DEV)[cut]
    else:
        ids = torch.randint(-1, n, (T,), generator=g, device=DEV)
        if T == 1:
            ids = ids.clamp_min(0)
    return dict(x=x, x_scale=xs, q=q, s=sc, b=zb, la=a, lb=b, lscale=lscale,
                ids=ids.to(torch.int32))


def _prepare_own(case, s):
    import bit_grouped_gemm_gb300 as bg
    e = lambda shape, dt: torch.zeros(shape, dtype=dt, device=DEV)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        s["x_out"] = e((T, H), torch.bfloat16)
        s["xn"] = e((T, H), torch.bfloat16)
        s["q8"] = s["q_scale"] = None
        if case["quant"] != "none":
            s["q8"] = e((T, H), torch.float8_e4m3fn)
            s["q_scale"] = e((T, _scales(case)), torch.float32)
        s["desc"] = bg.norm_desc(H, eps=EPS, alpha=s["alpha"], delta_f32=case["delta"] == "f32",
                                 quant_group=QGROUP if case["quant"] == "group" else 0)
    elif case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        plan = bg.moe_plan_create(bg.plan_desc(hidden=256, inter=256, num_experts=E, top_k=k,
                                               max_tokens=T), 0)
        s["plan"] = _Handle(plan, bg.moe_plan_destroy)
        o = dict(topk_idx=e((T, k), torch.int32), topk_w=e((T, k), torch.float32),
                 counts=e(E, torch.int32), offsets=e(E + 1, torch.int32),
                 tile_offsets=e(E + 1, torch.int32), perm=e(T * k, torch.int32),
                 inv=e(T * k, torch.int32), block_map=e((_max_tiles(case), 3), torch.int32),
                 num_tiles=e(1, torch.int32))
        s["out"] = o
        s["routing"] = bg.MoeRouting(**{n: t.data_ptr() for n, t in o.items()})
        s["desc"] = bg.score_desc(score=case["score"], bias=s["bias"], groups=case["groups"],
                                  topk_groups=case["topk_groups"], renormalise=case["renorm"],
                                  scale=case["scale"])
    else:
        d = bg.linear_desc(case["K"], case["N"], max_tokens=case["T"], max_rank=case["rank"])
        s["linear"] = _Handle(bg.moe_linear_create(d, 0), bg.moe_linear_destroy)
        s["w4"] = bg.w4(s["q"], s["s"], s["b"])
        s["lora"] = bg.lora(s["la"], s["lb"], s["lscale"])
        s["y"] = e((case["T"], case["N"]), torch.bfloat16)


def _scales(case):
    return -(-case["H"] // QGROUP) if case["quant"] == "group" else 1


def _max_tiles(case):
    return -(-case["T"] * case["k"] // TILE) + case["E"]


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    return {"norm": _plain_norm, "route": _plain_route, "linear": _plain_linear}[case["op"]](
        case, state)


def _run_own(case, s):
    import bit_grouped_gemm_gb300 as bg
    if case["op"] == "norm":
        bg.moe_norm_quant(s["desc"], s["x"], s["delta"], s["weight"], case["T"], s["x_out"],
                          s["xn"], s["q8"], s["q_scale"])
        out = [s["x_out"], s["xn"]]
        return out if s["q8"] is None else out + [s["q8"], s["q_scale"]]
    if case["op"] == "route":
        bg.moe_route_scored(s["plan"].value, s["logits"], case["T"], s["desc"], s["routing"])
        return list(s["out"].values())
    bg.moe_linear_forward(s["linear"].value, s["x"], case["T"], s["w4"], s["y"],
                          x_scale=s["x_scale"], lora=s["lora"], adapter=s["ids"])
    return s["y"]


def _plain_norm(case, s):
    T, H = case["T"], case["H"]
    xo = s["x"]
    if s["delta"] is not None:
        xo = (s["x"].float() + s["alpha"] * s["delta"].float()).bfloat16()
    v = xo.float()
    y = v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    if s["weight"] is not None:
        y = y * s["weight"].float()
    out = [xo, y.bfloat16()]
    if case["quant"] == "none":
        return out
    n = _scales(case)
    width = H if n == 1 else QGROUP
    yp = torch.zeros(T, n * width, device=y.device)
    yp[:, :H] = y
    amax = yp.view(T, n, width).abs().amax(2)
    inv = torch.where(amax > 0, E4M3_MAX / amax, torch.zeros_like(amax))
    code = (yp.view(T, n, width) * inv[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    code = code.view(T, n * width)[:, :H].to(torch.float8_e4m3fn)
    return out + [code, amax / E4M3_MAX]


def _plain_route(case, s):
    T, E, k = case["T"], case["E"], case["k"]
    low = float("-inf")
    # 64 bits: the order of neighbouring scores decides the choice
    l = torch.where(torch.isnan(s["logits"]), low, s["logits"]).double()
    if case["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
    else:
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = torch.nan_to_num(p / p.sum(1, keepdim=True), nan=0.0)
    # without a bias the scores rank as their logits do
    c = l if s["bias"] is None else p + s["bias"].double()
    shut = torch.zeros(T, E, dtype=torch.bool, device=l.device)
    if case["groups"] > 1:
        gs = E // case["groups"]
        gc = (p if s["bias"] is None else c).view(T, case["groups"], gs)
        score = gc.sort(dim=2, descending=True).values[:, :, :min(2, gs)].sum(2)
        best = score.sort(dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        keep = torch.zeros(T, case["groups"], dtype=torch.bool, device=l.device)
        keep.scatter_(1, best, True)
        shut = ~keep.repeat_interleave(gs, 1)
    order = c.sort(dim=1, descending=True, stable=True).indices
    late = shut.gather(1, order).to(torch.uint8).sort(dim=1, stable=True).indices
    idx = order.gather(1, late)[:, :k]
    w = p.gather(1, idx)
    if case["renorm"]:
        tot = w.sum(1, keepdim=True)
        w = torch.where(tot > 0, w / tot, torch.zeros_like(w))
    w = w * case["scale"]
    flat = idx.reshape(-1)
    perm = flat.sort(stable=True).indices
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device=l.device)
    counts = (flat[:, None] == torch.arange(E, device=l.device)).sum(0)
    zero = counts.new_zeros(1)
    off = torch.cat([zero, counts.cumsum(0)])
    tiles = (counts + TILE - 1) // TILE
    toff = torch.cat([zero, tiles.cumsum(0)])
    # every tile slot of the buffer, the unused ones zero
    slot = torch.arange(_max_tiles(case), device=l.device)
    e = (slot[:, None] >= toff[None, 1:]).sum(1)
    used = e < E
    e = e.clamp_max(E - 1)
    part = (slot - toff[e]) * TILE
    rows = torch.minimum(counts[e] - part, torch.full_like(e, TILE))
    bmap = torch.stack([e, off[e] + part, rows], 1) * used[:, None]
    i32 = lambda t: t.to(torch.int32)
    return [i32(idx), w.float(), i32(counts), i32(off), i32(toff), i32(perm), i32(inv),
            i32(bmap), i32(toff[E:])]


def _plain_linear(case, s):
    K, N, r, n = case["K"], case["N"], case["rank"], case["adapters"]
    shift = 4 * torch.arange(8, device=s["q"].device, dtype=torch.int32)
    q = ((s["q"][:, :, None] >> shift) & 15).view(N, K // GROUP, GROUP).float()
    w = (q * s["s"].float()[:, :, None] + s["b"].float()[:, :, None]).view(N, K)
    x = s["x"].float()
    # every adapter's products side by side; a token keeps those of its own
    h = x @ s["la"].float().reshape(n * r, K).T
    mine = s["ids"][:, None] == torch.arange(n, device=x.device)
    h = h * (mine * s["lscale"]).repeat_interleave(r, 1)
    y = x @ w.T + h @ s["lb"].float().transpose(1, 2).reshape(n * r, N)
    if s["x_scale"] is not None:
        y = y * s["x_scale"][:, None]
    return y.bfloat16()


# --------------------------------------------- what a pass cannot do without
def work(case):
    T = case["T"]
    if case["op"] == "norm":
        H, d = case["H"], {"none": 0, "bf16": 2, "f32": 4}[case["delta"]]
        q = 0 if case["quant"] == "none" else T * H + 4 * T * _scales(case)
        return {"bytes": T * H * (2 + d + 2 + 2) + q + (2 * H if case["weight"] else 0),
                "flops": T * H * 8}
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        out = T * k * 16 + (3 * E + 3) * 4 + _max_tiles(case) * 12
        return {"bytes": T * E * 4 + (4 * E if case["bias"] else 0) + out,
                "flops": T * E * (8 + k)}
    K, N, r = case["K"], case["N"], case["rank"]
    n = min(T, case["adapters"])
    xb = 1 if case["x"] == "e4m3" else 2
    return {"bytes": T * K * xb + (4 * T if xb == 1 else 0) + N * K // 2 + N * (K // GROUP) * 4
            + n * r * (K + N) * 2 + 4 * T + T * N * 2,
            "flops": 2 * T * K * N + 2 * T * r * (K + N)}


# ------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = _prepare_inputs(case, _gen(seed))
    f = {"norm": _exact_norm, "route": _exact_route, "linear": _exact_linear}[case["op"]]
    return f(case, s)


def _exact_norm(case, s):
    T, H = case["T"], case["H"]
    stream = s["x"].double()
    if s["delta"] is not None:
        stream = stream + s["alpha"] * s["delta"].double()
    # the norm is that of the stored stream
    kept = stream.float().bfloat16().double() if s["delta"] is not None else stream
    rms = (kept.pow(2).sum(1) / H + EPS).sqrt()
    normed = kept / rms[:, None]
    if s["weight"] is not None:
        normed = normed * s["weight"].double()
    out = [stream, normed]
    if case["quant"] == "none":
        return out
    step = H if case["quant"] == "row" else QGROUP
    scales, codes = [], []
    for c0 in range(0, H, step):
        part = normed[:, c0:c0 + step]
        sc = part.abs().max(1).values / E4M3_MAX
        scales.append(sc)
        codes.append(part / sc.clamp_min(1e-300)[:, None])
    return out + [torch.cat(codes, 1), torch.stack(scales, 1)]


def _exact_route(case, s):
    """The weights of the choice; the choice and its maps are whole numbers."""
    idx = _plain_route(case, s)[0].long()
    l = s["logits"].double()
    if case["score"] == "sigmoid":
        w = torch.sigmoid(torch.gather(l, 1, idx))
    else:
        w = torch.exp(torch.gather(torch.log_softmax(l, 1), 1, idx))
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return [None, w * case["scale"]] + [None] * 7


def _exact_linear(case, s):
    T, K, N = case["T"], case["K"], case["N"]
    nib = torch.stack([(s["q"].long() >> (4 * i)) & 15 for i in range(8)], -1).reshape(N, K)
    grp = torch.arange(K, device=nib.device) // GROUP
    w = nib.double() * s["s"].double()[:, grp] + s["b"].double()[:, grp]
    x = s["x"].float().double()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].double()[:, None]
    y = torch.matmul(x, w.transpose(0, 1))
    for a in range(case["adapters"]):
        rows = torch.nonzero(s["ids"] == a).flatten()
        if rows.numel():
            low = torch.matmul(x[rows], s["la"][a].double().transpose(0, 1))
            y[rows] += s["lscale"][a].double() * torch.matmul(low, s["lb"][a].double().transpose(0, 1))
    return y
