"""Attention over a paged cache, as cases that can be timed.

Three operators, in the order in which a served layer calls them before the
projection back to the stream:

* ``pages``: from the lengths of a batch's requests, the pages that they need
  (taken from a ring of free ones), and for every new token its slot in the
  cache, its position and, for trees of drafted tokens, its ancestors' mask;
* ``rope``: rotary positions of queries and keys, and the store of keys and
  values into their slots, in bf16 or in 8 bits (e4m3);
* ``attn``: the attention of new tokens, as chains or as drafted trees, over
  the requests' pages.

``run`` computes each one in elementary torch operations, or, where ``own`` is
set, through this repository's library.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
ROPE_LOW, ROPE_HIGH, ROPE_ORIGINAL = 1.0, 32.0, 32768


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decoded token of one request, the first on a new page
        dict(name="pages_token", op="pages", B=1, n=1, tree=False, ctx=2048, page=64, done=0),
        # a full batch of drafted trees; a few requests have ended and give their pages back
        dict(name="pages_trees", op="pages", B=256, n=16, tree=True, ctx=32768, page=32, done=9),
        # prompts of odd lengths, cut into chunks, on small pages
        dict(name="pages_prompts", op="pages", B=37, n=443, tree=False, ctx=5000, page=16, done=0),
        # one decoded token: its query, its key and value into the cache
        dict(name="rope_token", op="rope", T=1, Hq=16, Hkv=2, D=128, R=128, layout="half",
             scaling="none", cache="bf16", page=64, far=4096),
        # a mixed batch at far positions: half of each head in neighbouring pairs, seven queries
        # to a key, 8-bit cache
        dict(name="rope_ragged", op="rope", T=333, Hq=28, Hkv=4, D=128, R=64, layout="interleaved",
             scaling="by_parts", cache="e4m3", page=16, far=1000000),
        # a prompt chunk: a quarter of a wide head
        dict(name="rope_prompt", op="rope", T=4096, Hq=16, Hkv=2, D=256, R=64, layout="half",
             scaling="none", cache="bf16", page=64, far=32768),
        # one decoded token of one request
        dict(name="attn_token", op="attn", B=1, n=1, tree=False, ctx=2000, ragged=False, Hq=16,
             Hkv=2, D=128, cache="bf16", page=64),
        # a decode batch of contexts of all lengths
        dict(name="attn_batch", op="attn", B=64, n=1, tree=False, ctx=16384, ragged=True, Hq=16,
             Hkv=2, D=128, cache="bf16", page=64),
        # drafted trees, wide heads
        dict(name="attn_trees", op="attn", B=32, n=16, tree=True, ctx=8192, ragged=True, Hq=16,
             Hkv=2, D=256, cache="bf16", page=64),
        # larger trees of odd sizes, three queries to a key, small pages, 8-bit cache
        dict(name="attn_ragged", op="attn", B=7, n=61, tree=True, ctx=3001, ragged=True, Hq=24,
             Hkv=8, D=64, cache="e4m3", page=16),
        # a few drafted tokens on two long contexts, 8-bit cache
        dict(name="attn_long", op="attn", B=2, n=8, tree=True, ctx=131072, ragged=False, Hq=16,
             Hkv=2, D=128, cache="e4m3", page=64),
        # a prompt chunk of three requests behind what the cache holds
        dict(name="attn_prompt", op="attn", B=3, n=1365, tree=False, ctx=4096, ragged=False,
             Hq=16, Hkv=2, D=128, cache="bf16", page=64),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("pages", "rope", "attn", "attn"))
    page = rng.choice((16, 32, 64, 128))
    if op == "pages":
        tree = rng.random() < 0.5
        B = _log_int(rng, 1, 512)
        n = _log_int(rng, 1, 128 if tree else 2048)
        n = min(n, 16384 // B)
        return dict(op="pages", B=B, n=n, tree=tree, ctx=_log_int(rng, 1, 65536), page=page,
                    done=rng.choice((0, 0, B // 16)))
    Hkv, G = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 7, 8))
    D = rng.choice((64, 128, 256))
    kind = rng.choice(("bf16", "e4m3"))
    if op == "rope":
        row = (G * Hkv + 2 * Hkv) * D
        return dict(op="rope", T=_log_int(rng, 1, min(16384, 4096 * 5120 // row)), Hq=G * Hkv,
                    Hkv=Hkv, D=D, R=rng.choice((D, D // 2, D // 4)),
                    layout=rng.choice(("half", "interleaved")),
                    scaling=rng.choice(("none", "linear", "by_parts")), cache=kind, page=page,
                    far=_log_int(rng, 64, 1000000))
    while True:
        tree = rng.random() < 0.5
        B = _log_int(rng, 1, 128)
        n = _log_int(rng, 1, 64) if tree else rng.choice((1, _log_int(rng, 1, 2048)))
        c = dict(op="attn", B=B, n=n, tree=tree, ctx=_log_int(rng, 1, 131072),
                 ragged=rng.random() < 0.7, Hq=G * Hkv, Hkv=Hkv, D=D, cache=kind, page=page)
        # no more keys to read, products or scores than the largest listed ones
        keys = B * (c["ctx"] + n)
        if keys * Hkv * D <= 2 ** 27 and keys * n * G * Hkv * D <= 2 ** 35.4:
            return c


# --------------------------------------------------------------- the inputs
class _Handle:
    """A library handle that is given back when its state is dropped."""

    def __init__(self, value, destroy):
        self.value, self.destroy = value, destroy

    def __del__(self):
        self.destroy(self.value)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _host(seed):
    return torch.Generator().manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _dev(v):
    return torch.as_tensor(v, dtype=torch.int32).to(DEV)


def _lengths(h, B, most, ragged):
    """Context lengths of a batch: all of them, or spread over their logarithm."""
    if not ragged:
        return torch.full((B,), most, dtype=torch.int64)
    spread = torch.rand(B, generator=h, dtype=torch.float64)
    return torch.exp(spread * math.log(most)).round().long().clamp(1, most)


def _new_tokens(case, h):
    """New tokens of each request: n, n - 1 and so on down to three quarters of n, in any order."""
    B, n = case["B"], case["n"]
    new = n - torch.arange(B) % (n - (3 * n + 3) // 4 + 1)
    return new[torch.randperm(B, generator=h)]


def _parents(h, new):
    """Trees of drafted tokens in level order: each token hangs below one of the eight before
    it; the first ones, and now and then another, below the context itself (-1)."""
    start = torch.cumsum(new, 0) - new
    i = torch.arange(int(new.sum())) - start.repeat_interleave(new)
    back = torch.randint(1, 9, i.shape, generator=h)
    return (i - back).clamp_min(-1)


def prepare(case, seed):
    s = {"pages": _prepare_pages, "rope": _prepare_rope, "attn": _prepare_attn}[case["op"]](
        case, seed)
    s["case"] = case
    if own:
        _prepare_own(case, s)
    return s


def _words(case):
    return -(-case["n"] // 64)


def _prepare_pages(case, seed):
    h = _host(seed)
    B, P = case["B"], case["page"]
    ctx = _lengths(h, B, case["ctx"], B > 1)
    new = _new_tokens(case, h)
    parent = _dev(_parents(h, new)) if case["tree"] else None
    owned = (ctx + P - 1) // P
    width = int((case["ctx"] + case["n"] + P - 1) // P + 1)
    add = new.clone()
    if case["done"]:
        add[torch.randperm(B, generator=h)[:case["done"]]] = -1
        # the tokens' rows are those of the requests that go on
        if parent is not None:
            parent = _dev(_parents(h, add.clamp_min(0)))
    need = int(((ctx + new + P - 1) // P - owned).sum())
    held = int(owned.sum())
    pool = B * width
    ids = torch.randperm(pool, generator=h)[:held + need + 64]
    free = len(ids) - held
    table = torch.full((B, width), -1, dtype=torch.int64)
    inside = torch.arange(width)[None] < owned[:, None]
    table[inside] = ids[:held]
    ring = torch.full((pool,), -1, dtype=torch.int64)
    head = int(torch.randint(0, pool, (1,), generator=h))
    ring[(head + torch.arange(free)) % pool] = ids[held:]
    # rows for every token, and the padding of a batch that a graph was captured for
    rows = int(new.sum()) + 5
    s = dict(ctx=_dev(ctx), add=_dev(add), parent=parent, owned=_dev(owned), table=_dev(table),
             ring=_dev(ring), ring_pos=_dev([head, free]), rows=rows)
    return s


def _rope_freqs(case):
    """Angular frequencies of the rotated pairs, in 64 bits on the GPU."""
    R = case["R"]
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R)
    if case["scaling"] == "linear":
        return f / 4.0
    if case["scaling"] == "by_parts":
        turns = ROPE_ORIGINAL * f / (2 * math.pi)
        keep = ((turns - ROPE_LOW) / (ROPE_HIGH - ROPE_LOW)).clamp(0.0, 1.0)
        return f * (keep + (1.0 - keep) / 4.0)
    return f


def _gain(case):
    return 1.1386 if case["scaling"] == "by_parts" else 1.0


def _cache(case, g, pages):
    shape = (pages, case["Hkv"], case["page"], case["D"])
    k, v = _randn(g, *shape), _randn(g, *shape)
    if case["cache"] == "bf16":
        return dict(kc=k.bfloat16(), vc=v.bfloat16(), ks=None, vs=None)
    ks = 0.01 + 0.01 * torch.rand(case["Hkv"], generator=g, device=DEV)
    vs = 0.01 + 0.01 * torch.rand(case["Hkv"], generator=g, device=DEV)
    code = lambda x, s: (x / s[:, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return dict(kc=code(k, ks), vc=code(v, vs), ks=ks, vs=vs)


def _prepare_rope(case, seed):
    g, h = _gen(seed), _host(seed)
    T, P = case["T"], case["page"]
    # the rows of one fused projection: queries, keys and values side by side
    row = (case["Hq"] + 2 * case["Hkv"]) * case["D"]
    qkv = (1.5 * _randn(g, T, row)).bfloat16()
    pages = 2 * (-(-T // P)) + 2
    slot = torch.randperm(pages * P, generator=h)[:T]
    if T > 8:
        slot[torch.randperm(T, generator=h)[:T // 64]] = -1      # rows that are padding
    position = torch.randint(0, case["far"], (T,), generator=h)
    return dict(qkv=qkv, slot=_dev(slot), position=_dev(position), **_cache(case, g, pages),
                freqs=_rope_freqs(case))


def _prepare_attn(case, seed):
    g, h = _gen(seed), _host(seed)
    B, P, T1 = case["B"], case["page"], case["Hq"] * case["D"]
    ctx = _lengths(h, B, case["ctx"], case["ragged"])
    new = _new_tokens(case, h)
    length = ctx + new
    held = (length + P - 1) // P
    pool, width = int(held.sum()) + 8, int(held.max())
    table = torch.zeros((B, width), dtype=torch.int64)
    ids = torch.randperm(pool, generator=h)
    table[torch.arange(width)[None] < held[:, None]] = ids[:int(held.sum())]
    T = int(new.sum())
    off = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(new, 0)])
    mask = None
    if case["tree"]:
        mask = _ancestors(_dev(_parents(h, new)).long(), _dev(off).long(), _dev(new).long(),
                          case["n"])[1]
    return dict(q=(1.5 * _randn(g, T, T1)).bfloat16(), **_cache(case, g, pool), table=_dev(table),
                offsets=_dev(off), length=_dev(length), mask=mask, T=T, most=int(length.max()))


def _prepare_own(case, s):
    import bit_grouped_gemm_gb300 as bg
    e = lambda *shape, dt=torch.int32: torch.zeros(shape, dtype=dt, device=DEV)
    if case["op"] == "pages":
        B, M, w = case["B"], s["rows"], _words(case) if case["tree"] else 0
        s["desc"] = bg.page_desc(B, case["page"], s["table"].shape[1], M, s["ring"].shape[0],
                                 mask_words=w)
        s["owned_out"], s["ring_out"] = e(B), e(2)
        s["pool"] = bg.page_pool(s["table"], s["ring"], s["owned"], s["ring_pos"],
                                 owned_out=s["owned_out"], ring_pos_out=s["ring_out"])
        o = dict(length=e(B), offsets=e(B + 1), slot=e(M), position=e(M),
                 mask=e(M, w, dt=torch.int64) if w else None, status=e(5))
        s["out"], s["map"] = o, bg.token_map(**o)
        return
    rope = case["op"] == "rope"
    T = case["T"] if rope else s["T"]
    d = bg.attn_desc(case["Hq"], case["Hkv"], case["D"], case["page"], cache=case["cache"],
                     max_tokens=T, max_requests=1 if rope else case["B"],
                     rotary_dim=case["R"] if rope else 0,
                     rope_layout=case["layout"] if rope else "half",
                     rope_scaling=case["scaling"] if rope else "none", rope_factor=4.0,
                     rope_low=ROPE_LOW, rope_high=ROPE_HIGH, rope_original=ROPE_ORIGINAL,
                     rope_gain=_gain(case) if rope else 1.0)
    s["attn"] = _Handle(bg.moe_attn_create(d, 0), bg.moe_attn_destroy)
    s["cache"] = bg.kv_cache(s["kc"], s["vc"], s["ks"], s["vs"])
    s["out"] = e(T, case["Hq"] * case["D"], dt=torch.bfloat16)


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    return {"pages": _plain_pages, "rope": _plain_rope, "attn": _plain_attn}[case["op"]](
        case, state)


def _run_own(case, s):
    import bit_grouped_gemm_gb300 as bg
    if case["op"] == "pages":
        bg.moe_page_map(s["desc"], s["ctx"], s["add"], s["parent"], s["pool"], s["map"])
        o = s["out"]
        return [s["owned_out"], s["ring_out"], s["table"], s["ring"], o["length"], o["offsets"],
                o["slot"], o["position"], o["status"]] + ([] if o["mask"] is None else [o["mask"]])
    if case["op"] == "rope":
        q, k, v = _split(case, s)
        row = s["qkv"].shape[1]
        bg.moe_rope_store(s["attn"].value, q, k, v, case["T"], s["position"], s["slot"], s["out"],
                          s["cache"], q_stride=row, k_stride=row, v_stride=row)
        return [s["out"], s["kc"], s["vc"]]
    bg.moe_tree_attention(s["attn"].value, s["q"], s["T"], s["cache"], s["table"], s["offsets"],
                          s["length"], s["out"], mask=s["mask"])
    return s["out"]


def _split(case, s):
    a, b = case["Hq"] * case["D"], case["Hkv"] * case["D"]
    return s["qkv"][:, :a], s["qkv"][:, a:a + b], s["qkv"][:, a + b:]


def _ancestors(parent, off, new, most):
    """Depth of every token in its tree and the bits of its ancestors and itself, in 64-bit
    words, by doubling the step up the tree."""
    T = parent.shape[0]
    row = torch.arange(T, device=parent.device)
    b = (row[:, None] >= off[None, 1:-1]).sum(1)
    first = off[b]
    words = -(-most // 64)
    top = T                                       # a row above all roots: no bits, depth 0
    up = torch.cat([torch.where(parent < 0, top, first + parent), parent.new_full((1,), top)])
    i = row - first
    bits = torch.zeros(T + 1, words, dtype=torch.int64, device=parent.device)
    bits[row, i // 64] = torch.ones_like(i) << (i % 64)
    depth = torch.cat([torch.ones_like(row), row.new_zeros(1)])
    for _ in range(max(1, (most - 1).bit_length())):
        bits = bits | bits[up]
        depth = depth + depth[up]
        up = up[up]
    return depth[:T] - 1, bits[:T]


def _plain_pages(case, s):
    P, M = case["page"], s["rows"]
    B, width = s["table"].shape
    cap = s["ring"].shape[0]
    ctx, add, owned = s["ctx"].long(), s["add"].long(), s["owned"].long()
    head, free = s["ring_pos"][0].long(), s["ring_pos"][1].long()
    new = add.clamp_min(0)
    ends = torch.cumsum(new, 0)
    off = torch.cat([ends.new_zeros(1), ends]).clamp_max(M)
    want = (ctx + new + P - 1) // P
    fits = (add >= 0) & (want <= width) & (ctx <= owned * P) & (ends <= M)
    need = torch.where(fits, (want - owned).clamp_min(0), 0)
    upto = torch.cumsum(need, 0)
    served = fits & ((need == 0) | (upto <= free))
    taken = torch.where(served, need, 0)
    first = upto - need
    # pages of the served requests, from the ring's head on
    col = torch.arange(width, device=ctx.device)
    fresh = served[:, None] & (col >= owned[:, None]) & (col < want[:, None])
    at = (head + first[:, None] + col - owned[:, None]) % cap
    pages = torch.where(fresh, s["ring"].long()[at], s["table"].long())
    # pages of the requests that ended, to the ring's tail
    gone = add < 0
    back = torch.where(gone, owned, 0)
    backto = torch.cumsum(back, 0)
    fit = gone & (backto + free <= cap)
    back = torch.where(fit, back, 0)
    left = fit[:, None] & (col < owned[:, None])
    to = (head + free + (backto - back)[:, None] + col) % cap
    ring = torch.cat([s["ring"], s["ring"].new_zeros(1)])
    ring[torch.where(left, to, cap).flatten()] = s["table"].flatten()
    ring = ring[:cap]
    # the tokens' rows
    row = torch.arange(M, device=ctx.device)
    b = (row[:, None] >= off[None, 1:]).sum(1)
    live = b < B
    b = b.clamp_max(B - 1)
    live = live & served[b]
    i = row - off[b]
    at = ctx[b] + i
    page = pages[b, torch.where(live, at // P, 0)]
    slot = torch.where(live, page * P + at % P, -1)
    out = []
    if case["tree"]:
        parent = s["parent"].long()
        T = parent.shape[0]
        depth, bits = _ancestors(parent, off, new, case["n"])
        i = torch.cat([depth, depth.new_zeros(M - T)])
        bits = torch.cat([bits, bits.new_zeros(M - T, bits.shape[1])])
        out = [torch.where(live[:, None], bits, 0)]
    position = torch.where(live, ctx[b] + i, 0)
    keep = torch.where(fit, 0, torch.where(served, torch.maximum(owned, want), owned))
    length = torch.where(served, ctx + new, 0)
    used, came = taken.sum(), back.sum()
    refused = (~served & ~fit).sum()
    status = torch.stack([off[-1], used, refused, (upto[-1] - free).clamp_min(0), 0 * used])
    pos = torch.stack([(head + used) % cap, free - used + came])
    i32 = lambda t: t.to(torch.int32)
    return [i32(keep), i32(pos), i32(pages), i32(ring), i32(length), i32(off), i32(slot),
            i32(position), i32(status)] + out


def _plain_rope(case, s):
    T, D, R, P = case["T"], case["D"], case["R"], case["page"]
    # far positions: the angle in 64 bits
    angle = s["position"].double()[:, None] * s["freqs"]
    cos = (torch.cos(angle) * _gain(case)).float()[:, None]
    sin = (torch.sin(angle) * _gain(case)).float()[:, None]

    def turn(x):
        x = x.float().view(T, -1, D)
        if case["layout"] == "half":
            a, b = x[..., :R // 2], x[..., R // 2:R]
            return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., R:]], 2)
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
        return torch.cat([y, x[..., R:]], 2)

    q, k, v = _split(case, s)
    k, v = turn(k), v.float().view(T, -1, D)
    if s["ks"] is not None:
        k = (k / s["ks"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / s["vs"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    # rows without a slot go to a page behind the last one
    pages = s["kc"].shape[0]
    slot = torch.where(s["slot"] < 0, pages * P, s["slot"]).long()

    def store(cache, x):
        # bytes: 8-bit floats have no scatter of their own
        raw = torch.uint8 if cache.dtype == torch.float8_e4m3fn else torch.int16
        c = torch.cat([cache.view(raw), cache.view(raw)[:1]])
        c[slot // P, :, slot % P] = x.to(cache.dtype).view(raw)
        return c[:pages].view(cache.dtype)

    return [turn(q).view(T, -1).bfloat16(), store(s["kc"], k), store(s["vc"], v)]


def _plain_attn(case, s):
    B, Hkv, D, P = case["B"], case["Hkv"], case["D"], case["page"]
    G, L, n, T = case["Hq"] // Hkv, s["most"], case["n"], s["T"]
    off, length = s["offsets"].long(), s["length"].long()
    new = off[1:] - off[:-1]
    ctx = length - new
    # every request's keys side by side, the shorter ones padded
    j = torch.arange(L, device=off.device)
    page = s["table"].long()[:, j // P]

    def rows(c, scale):
        raw = c.view(torch.uint8 if c.dtype == torch.float8_e4m3fn else torch.int16)
        x = raw[page, :, (j % P)[None]].view(c.dtype).float()
        x = x if scale is None else x * scale[:, None]
        return x.permute(0, 2, 1, 3)                     # [B, Hkv, L, D]

    t = (off[:-1, None] + torch.arange(n, device=off.device)).clamp_max(T - 1)
    q = s["q"].float().view(T, Hkv, G, D)[t]             # [B, n, Hkv, G, D]
    q = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    score = q @ rows(s["kc"], s["ks"]).transpose(2, 3) / math.sqrt(D)
    i = torch.arange(n, device=off.device)
    node = j[None] - ctx[:, None]                        # a key's place among the new tokens
    see = (node[:, None] <= i[:, None]) & (j[None] < length[:, None])[:, None]
    if s["mask"] is not None:
        at = node.clamp(0, n - 1)
        word = s["mask"][t].gather(2, (at // 64)[:, None].expand(B, n, L))
        see = see & ((node < 0)[:, None] | ((word >> (at % 64)[:, None]) & 1).bool())
    score = score.view(B, Hkv, n, G, L).masked_fill_(~see[:, None, :, None], float("-inf"))
    p = torch.exp(score - score.amax(4, keepdim=True))
    p = p / p.sum(4, keepdim=True)
    v = rows(s["vc"], s["vs"])
    # the padding's places hold other requests' values
    v = v * (j[None] < length[:, None])[:, None, :, None]
    o = (p.view(B, Hkv, n * G, L) @ v).view(B, Hkv, n, G, D).permute(0, 2, 1, 3, 4)
    return o[i[None] < new[:, None]].reshape(T, -1).bfloat16()


# --------------------------------------------- what a pass cannot do without
def work(case):
    """Bytes and products of a case, its ragged lengths at what they come to on average."""
    if case["op"] == "pages":
        B, n = case["B"], case["n"]
        T = B * n if n == 1 or B == 1 else B * n * 7 // 8
        w = _words(case) if case["tree"] else 0
        fresh = B * -(-n // case["page"])
        return {"bytes": 4 * (6 * B + 2 * T + 2 * fresh + 10) + T * (8 * w + (4 if w else 0)),
                "flops": 8 * T}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    e = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "rope":
        T = case["T"]
        return {"bytes": T * (4 * Hq * D + Hkv * D * (4 + 2 * e) + 8),
                "flops": T * (Hq + Hkv) * case["R"] * 3}
    B, n, ctx = case["B"], case["n"], case["ctx"]
    if case["ragged"] and ctx > 1:
        ctx = int((ctx - 1) / math.log(ctx))
    new = n if n == 1 or B == 1 else n * 7 // 8
    keys = ctx + new / 2 if not case["tree"] else ctx + min(new, 6)
    return {"bytes": int(B * (ctx + new) * Hkv * D * 2 * e + 4 * B * new * Hq * D),
            "flops": int(4 * B * new * keys * Hq * D)}


# ------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    if case["op"] == "pages":
        return None                                      # whole numbers throughout
    if case["op"] == "rope":
        return _exact_rope(case, _prepare_rope(case, seed))
    return _exact_attn(case, _prepare_attn(case, seed))


def _exact_rope(case, s):
    T, D, R, P, Hq, Hkv = (case[k] for k in ("T", "D", "R", "page", "Hq", "Hkv"))
    x = s["qkv"].double().view(T, Hq + 2 * Hkv, D)
    pair = torch.arange(R // 2, device=x.device)
    one, two = (pair, pair + R // 2) if case["layout"] == "half" else (2 * pair, 2 * pair + 1)
    z = torch.complex(x[:, :Hq + Hkv, one], x[:, :Hq + Hkv, two])
    angle = s["position"].double()[:, None, None] * s["freqs"]
    z = z * torch.polar(torch.full_like(angle, _gain(case)), angle)
    x[:, :Hq + Hkv, one], x[:, :Hq + Hkv, two] = z.real, z.imag
    caches = []
    for c, sc, rows in ((s["kc"], s["ks"], x[:, Hq:Hq + Hkv]), (s["vc"], s["vs"], x[:, Hq + Hkv:])):
        c = c.float().double()
        if sc is not None:
            rows = (rows / sc.double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        kept = torch.nonzero(s["slot"] >= 0).flatten()
        slot = s["slot"][kept].long()
        c[slot // P, :, slot % P] = rows[kept]
        caches.append(c)
    return [x[:, :Hq].reshape(T, -1)] + caches


def _exact_attn(case, s):
    Hkv, D, P = case["Hkv"], case["D"], case["page"]
    G = case["Hq"] // Hkv
    out = torch.zeros(s["T"], Hkv, G, D, dtype=torch.float64, device=DEV)
    off, length = s["offsets"].tolist(), s["length"].tolist()
    for b in range(case["B"]):
        new, total = off[b + 1] - off[b], length[b]
        ctx = total - new
        pages = s["table"][b, :-(-total // P)].long()
        see = torch.ones(new, total, dtype=torch.bool, device=DEV)
        see[:, ctx:] = torch.ones(new, new, dtype=torch.bool, device=DEV).tril()
        if s["mask"] is not None:
            word = s["mask"][off[b]:off[b + 1]]
            bits = (word[:, :, None] >> torch.arange(64, device=DEV)) & 1
            see[:, ctx:] &= bits.reshape(new, -1)[:, :new].bool()
        for h in range(Hkv):
            flat = lambda c, sc: (c[pages, h].float().double().reshape(-1, D)[:total] *
                                  (1.0 if sc is None else sc[h].double()))
            k, v = flat(s["kc"], s["ks"]), flat(s["vc"], s["vs"])
            q = s["q"][off[b]:off[b + 1]].double().view(new, Hkv, G, D)[:, h]
            for c0 in range(0, new, 256):
                rows = slice(c0, min(new, c0 + 256))
                score = torch.einsum("igd,kd->igk", q[rows], k) / math.sqrt(D)
                score = torch.where(see[rows, None], score, -math.inf)
                out[off[b] + rows.start:off[b] + rows.stop, h] = torch.einsum(
                    "igk,kd->igd", torch.softmax(score, 2), v)
    return out.view(s["T"], -1)
