"""The operators of attention over a paged cache against plain 64-bit forms, at the
sizes, masks and values where they can go wrong."""
import itertools
import math

import pytest
import torch

import bit_grouped_gemm_gb300 as bg
from tests import attention_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
i32 = ref.i32


@pytest.fixture(scope="module", autouse=True)
def built():
    from bit_grouped_gemm_gb300 import build
    build.build()
    bg.load_library()


# ----------------------------------------------------------------- page map
class PageCase:
    """Lists of one step's state, and the call on device copies of them."""

    def __init__(self, page, width, M, cap, words, context, added, owned, ring_pos, parent=None,
                 seed=0):
        self.page, self.width, self.M, self.cap, self.words = page, width, M, cap, words
        self.context, self.added, self.owned, self.ring_pos = context, added, owned, ring_pos
        self.parent = parent
        h = torch.Generator().manual_seed(seed)
        B = len(context)
        ids = torch.randperm(B * width + cap, generator=h).tolist()
        self.table = [[ids.pop() for _ in range(width)] for _ in range(B)]
        self.ring = [ids.pop() for _ in range(cap)]

    def want(self):
        return ref.page_map(len(self.context), self.page, self.width, self.M, self.cap, self.words,
                            self.context, self.added, self.parent, self.table, self.ring,
                            self.owned, self.ring_pos)

    def got(self, in_place=False, stream=None):
        B, M = len(self.context), self.M
        table, ring, owned, pos = (i32(x) for x in (self.table, self.ring, self.owned, self.ring_pos))
        fill = lambda *s: torch.full(s, 12345, dtype=torch.int32, device=DEV)
        o = dict(length=fill(B), offsets=fill(B + 1), slot=fill(M), position=fill(M), status=fill(5))
        o["mask"] = fill(M, self.words).long() if self.words else None
        owned_out, pos_out = (owned, pos) if in_place else (fill(B), fill(2))
        d = bg.page_desc(B, self.page, self.width, M, self.cap, self.words)
        pool = bg.page_pool(table, ring, owned, pos, owned_out, pos_out)
        parent = None
        if self.parent is not None:
            parent = i32((self.parent + [0] * M)[:M])
        bg.moe_page_map(d, i32(self.context), i32(self.added), parent, pool, bg.token_map(**o),
                        stream)
        torch.cuda.synchronize()
        r = dict(table=table, ring=ring, owned=owned_out, ring_pos=pos_out, **o)
        if not self.words:
            r["mask"] = torch.zeros(M, 0)
        return {k: v.tolist() for k, v in r.items()}

    def check(self, **kw):
        want, got = self.want(), self.got(**kw)
        for k in want:
            assert got[k] == want[k], k


def random_pages(seed, B, page, most_ctx, most_new, words=0, tree=False, ended=0, spare=0, pad=3):
    h = torch.Generator().manual_seed(seed)
    r = lambda hi, n=B: torch.randint(0, hi + 1, (n,), generator=h).tolist()
    context, added = r(most_ctx), r(most_new)
    for b in torch.randperm(B, generator=h)[:ended].tolist():
        added[b] = -1 - b
    owned = [-(-c // page) + x for c, x in zip(context, r(2))]
    width = max(-(-(most_ctx + most_new) // page), max(owned)) + 1
    need = sum(max(0, -(-(c + max(a, 0)) // page) - o) for c, a, o in zip(context, added, owned))
    rows = sum(max(a, 0) for a in added)
    parent = None
    if tree:
        parent = [int(torch.randint(-1, i, (1,), generator=h)) if i else -1
                  for a in added for i in range(max(a, 0))]
    cap = need + sum(owned) + 7
    return PageCase(page, width, max(rows, 1) + pad, cap, words, context, added, owned,
                    [cap - 3, max(0, min(need + spare, cap))], parent, seed)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seed,B,page,ctx,new,words,tree,ended", [
    (0, 1, 16, 0, 1, 0, False, 0), (1, 1, 64, 63, 1, 0, False, 0), (2, 1, 256, 1000, 700, 0, False, 0),
    (3, 2, 16, 5, 40, 1, True, 0), (4, 31, 32, 200, 64, 1, True, 3), (5, 7, 16, 90, 128, 2, True, 0),
    (6, 5, 128, 700, 256, 4, True, 1), (7, 300, 16, 300, 3, 1, False, 20), (8, 513, 64, 999, 1, 0, False, 50),
    (9, 40, 16, 100, 130, 3, False, 0), (10, 1025, 32, 60, 9, 1, True, 100), (11, 17, 16, 2000, 900, 0, False, 2),
    (12, 9, 16, 0, 0, 0, False, 0),
])
def test_page_map(seed, B, page, ctx, new, words, tree, ended, in_place):
    random_pages(seed, B, page, ctx, new, words, tree, ended).check(in_place=in_place)


@pytest.mark.parametrize("short", [1, 3, 20, 10 ** 6])
def test_page_map_runs_out_of_pages(short):
    """Requests are served in order as far as the ring goes; those without need all the same."""
    for seed in range(4):
        c = random_pages(seed, 12, 16, 64, 40, spare=-short, ended=2)
        c.check(in_place=True)
        assert c.want()["status"][3] > 0 and c.want()["status"][2] > 0


def test_page_map_refuses_requests():
    """Unsound lengths, one kind each; their neighbours are served."""
    ok = (10, 5, 1)
    bad = [(-1, 5, 1), (10, 5, -1), (10, 5, 9), (33, 5, 2), (100, 100, 7), (2 ** 31 - 1, 2 ** 31 - 1, 1),
           (0, 65, 0), (10, -1, 9), (10, -1, -2)]
    for x in bad:
        for order in ([ok, x, ok], [x, ok], [ok, x]):
            context, added, owned = (list(v) for v in zip(*order))
            c = PageCase(16, 8, 200, 30, 1, context, added, owned, [28, 12])
            c.check()
            assert c.want()["status"][2] >= 1
    # rows past the capacity, and everything behind them
    PageCase(16, 8, 12, 30, 0, [0, 3, 4, 0], [5, 8, 1, 0], [0, 1, 1, 0], [0, 12]).check()
    # a ring too full to take the pages back, a state out of range
    PageCase(16, 8, 12, 10, 0, [20, 30, 4], [-1, -1, 2], [2, 3, 1], [4, 7]).check()
    PageCase(16, 8, 12, 10, 0, [20, 30, 4], [-1, 3, 2], [2, 2, 1], [-3 % 2 ** 31, 2 ** 31 - 1]).check()
    PageCase(16, 8, 12, 10, 0, [20, 30, 4], [-1, 3, 2], [2, 2, 1], [25, -1]).check()


def test_page_map_wrong_parents_are_roots():
    parent = [-1, 0, 2, -2, 5, 3, 2 ** 31 - 1, -2 ** 31, 0]
    PageCase(16, 8, 9, 30, 1, [3, 7], [4, 5], [1, 1], [0, 12], parent).check()
    assert PageCase(16, 8, 9, 30, 1, [3, 7], [4, 5], [1, 1], [0, 12], parent).want()["status"][4] == 6


def test_page_map_pages_circulate():
    """Steps in place, ends and starts of requests among them: no page is lost or held twice."""
    h = torch.Generator().manual_seed(5)
    B, page, width, cap, M = 24, 16, 12, 150, 400
    context, owned = [0] * B, i32([0] * B)
    table, ring, pos = i32([[-1] * width] * B), i32(list(range(cap))), i32([0, cap])
    out = dict(length=i32([0] * B), offsets=i32([0] * (B + 1)), slot=i32([0] * M),
               position=i32([0] * M), status=i32([0] * 5))
    d, pool = bg.page_desc(B, page, width, M, cap), bg.page_pool(table, ring, owned, pos)
    tm = bg.token_map(**out)
    for step in range(60):
        added = [-1 if c and int(torch.randint(0, 9, (1,), generator=h)) == 0 else
                 int(torch.randint(0, 17, (1,), generator=h)) for c in context]
        bg.moe_page_map(d, i32(context), i32(added), None, pool, tm)
        length, have = out["length"].tolist(), owned.tolist()
        head, free = pos.tolist()
        ids = [ring.tolist()[(head + i) % cap] for i in range(free)]
        ids += [p for b in range(B) for p in table.tolist()[b][:have[b]]]
        assert sorted(ids) == list(range(cap)), step
        context = [n if a >= 0 and n else 0 if a < 0 else c for c, a, n in zip(context, added, length)]


# ------------------------------------------------------------- rotary, store
def run_rope(T, Hq, Hkv, D, R, page, layout="half", cache="bf16", scaling="none", far=5000, seed=0,
             gain=1.0, fused=True, in_place=False, stream=None, x=None, position=None):
    g, h = torch.Generator(device=DEV).manual_seed(seed), torch.Generator().manual_seed(seed)
    cols = (Hq + 2 * Hkv) * D
    if x is None:
        x = (1.5 * torch.randn(T, cols, generator=g, device=DEV)).bfloat16()
    q, k, v = x[:, :Hq * D], x[:, Hq * D:(Hq + Hkv) * D], x[:, (Hq + Hkv) * D:]
    ld = dict(q_stride=cols, k_stride=cols, v_stride=cols)
    if not fused:
        q, k, v, ld = q.contiguous(), k.contiguous(), v.contiguous(), {}
    pages = -(-T // page) + 2
    slot = torch.randperm(pages * page, generator=h)[:T]
    slot[::7] = torch.tensor([-1, pages * page, -2 ** 31, 2 ** 31 - 1])[torch.arange(len(slot[::7])) % 4]
    if position is None:
        position = torch.randint(0, far, (T,), generator=h)
        position[0] = 0
    kc, vc, ks, vs = ref.cache_of(g, pages, Hkv, page, D, cache)
    arg = dict(rope_theta=10000.0, rope_scaling=scaling, rope_factor=8.0, rope_low=1.0, rope_high=4.0,
               rope_original=2048)
    freqs = ref.frequencies(R, 10000.0, scaling, 8.0, 1.0, 4.0, 2048)
    xin = [t.double().view(T, -1, D) for t in (q.clone(), k.clone(), v.clone())]
    yq, yk = (ref.turn(t, position, freqs, layout, gain) for t in xin[:2])
    yv = xin[2]
    wk, wv = kc.float().double(), vc.float().double()
    keep = ((slot >= 0) & (slot < pages * page)).to(DEV)
    at = slot.to(DEV)[keep]
    if cache == "e4m3":
        yk, yv = yk / ks.double()[:, None], yv / vs.double()[:, None]
    wk[at // page, :, at % page] = yk[keep]
    wv[at // page, :, at % page] = yv[keep]
    out = q if in_place else torch.full((T, Hq * D), float("nan"), dtype=torch.bfloat16, device=DEV)
    d = bg.attn_desc(Hq, Hkv, D, page, cache=cache, max_tokens=T, rotary_dim=R, rope_layout=layout,
                     rope_gain=gain, **arg)
    a = bg.moe_attn_create(d, 0)
    try:
        bg.moe_rope_store(a, q, k, v, T, i32(position), i32(slot), out, bg.kv_cache(kc, vc, ks, vs),
                          out_stride=cols if in_place and fused else 0, stream=stream, **ld)
        torch.cuda.synchronize()
        assert bg.moe_attn_get_error(a) == 0
    finally:
        bg.moe_attn_destroy(a)
    # sizes of the pairs that turn: a turned element is off by the rotation's FP32 error times the
    # pair's size (angle 2^-31 turns and sincospi's 2 units: 2^-21 in all with the products)
    size = [t.abs().amax(2, keepdim=True) * 2.0 ** -21 for t in xin[:2]]
    return out.double().view(T, -1, D), kc, vc, yq, wk, wv, size[0], float(size[1].max()), at


def check_rope(cache="bf16", **kw):
    out, kc, vc, yq, wk, wv, slack, kslack, at = run_rope(cache=cache, **kw)
    assert ((out - yq).abs() <= 2.0 ** -8 * yq.abs() + slack).all()
    if cache == "bf16":
        assert ((kc.double() - wk).abs() <= 2.0 ** -8 * wk.abs() + kslack).all()
        assert torch.equal(vc.double(), wv)
        return
    # e4m3: half a step, 2^-4 relative or 2^-10 among the subnormals; the scale is at least 0.01
    for got, want, s in ((kc, wk, 100 * kslack), (vc, wv, 0.0)):
        want = want.clamp(-448.0, 448.0)
        tol = torch.maximum(2.0 ** -4 * want.abs(), torch.full_like(want, 2.0 ** -10))
        assert ((got.float().double() - want).abs() <= tol * (1 + 2.0 ** -20) + s).all()


@pytest.mark.parametrize("cache,layout", list(itertools.product(["bf16", "e4m3"], ["half", "interleaved"])))
@pytest.mark.parametrize("T,Hq,Hkv,D,R,page", [
    (1, 16, 2, 128, 128, 64), (3, 1, 1, 64, 16, 16), (17, 28, 4, 128, 64, 16), (130, 8, 8, 256, 256, 256),
    (333, 6, 2, 64, 64, 32), (40, 16, 2, 256, 64, 128), (5, 3, 1, 128, 0, 16), (64, 5, 1, 256, 240, 64),
])
def test_rope_store(T, Hq, Hkv, D, R, page, cache, layout):
    check_rope(T=T, Hq=Hq, Hkv=Hkv, D=D, R=R, page=page, cache=cache, layout=layout, seed=T)


@pytest.mark.parametrize("scaling,gain", [("linear", 1.0), ("by_parts", 1.25), ("none", -0.5)])
def test_rope_scaling(scaling, gain):
    check_rope(T=50, Hq=4, Hkv=2, D=128, R=128, page=16, scaling=scaling, gain=gain, far=100000)


def test_rope_far_and_negative_positions():
    """The angle is exact modulo a turn, to the ends of int32."""
    pos = torch.tensor([0, 1, -1, 2 ** 20, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, 123456789])
    check_rope(T=9, Hq=2, Hkv=1, D=64, R=64, page=16, position=pos)


@pytest.mark.parametrize("fused", [True, False])
def test_rope_in_place(fused):
    check_rope(T=29, Hq=8, Hkv=2, D=128, R=96, page=16, fused=fused, in_place=True)


def test_rope_extreme_values():
    """e4m3 saturates infinities and large values and keeps NaNs; bf16 passes them."""
    T, Hq, Hkv, D = 8, 1, 1, 64
    x = torch.ones(T, 3 * D, dtype=torch.bfloat16, device=DEV)
    x[0, 2 * D:] = float("inf")
    x[1, 2 * D:] = -1e30
    x[2, 2 * D:] = float("nan")
    x[3, D:2 * D] = float("nan")
    for cache in ("bf16", "e4m3"):
        g = torch.Generator(device=DEV).manual_seed(0)
        kc, vc, ks, vs = ref.cache_of(g, 1, 1, 16, D, cache)
        a = bg.moe_attn_create(bg.attn_desc(1, 1, D, 16, cache=cache, max_tokens=T, rotary_dim=0), 0)
        out = torch.empty(T, D, dtype=torch.bfloat16, device=DEV)
        bg.moe_rope_store(a, x, x[:, D:], x[:, 2 * D:], T, i32(range(T)), i32(range(T)), out,
                          bg.kv_cache(kc, vc, ks, vs), q_stride=3 * D, k_stride=3 * D, v_stride=3 * D)
        torch.cuda.synchronize()
        bg.moe_attn_destroy(a)
        v, k = vc[0, 0].float(), kc[0, 0].float()
        assert (v[0] == (float("inf") if cache == "bf16" else 448.0)).all()
        assert (v[1] <= -440).all() and torch.isnan(v[2]).all() and torch.isnan(k[3]).all()
        assert torch.equal(out, x[:, :D])


# ----------------------------------------------------------------- attention
def run_attention(lengths, news, Hq, Hkv, D, page, cache="bf16", words=0, seed=0, scale=0.0, masks=None,
                  pad=2, lead=0, spread=1.5, edit=None, q_extra=0, o_extra=0, calls=1, width_extra=1,
                  stream=None, limit=None):
    """One call on random inputs, checked against the 64-bit definition. `edit(d)` may change the
    inputs before the call."""
    g, h = torch.Generator(device=DEV).manual_seed(seed), torch.Generator().manual_seed(seed)
    T = lead + sum(news) + pad
    cols = Hq * D
    held = [max(n, 0) for n in lengths]
    table, pages = ref.table_of(h, held, page, width_extra=width_extra)
    kc, vc, ks, vs = ref.cache_of(g, pages, Hkv, page, D, cache)
    qbuf = (spread * torch.randn(T, cols + q_extra, generator=g, device=DEV)).bfloat16()
    if words and masks is None:
        masks = [ref.random_tree(h, n, words) for n in news]
    d = dict(q=qbuf, kc=kc, vc=vc, ks=ks, vs=vs, table=table, masks=masks, lengths=lengths)
    if edit:
        edit(d)
    mask = None
    if masks is not None:
        rows = [[0] * words] * lead + [r for m in masks for r in m] + [[-1] * words] * pad
        mask = torch.tensor(rows, dtype=torch.int64, device=DEV)
    off = [lead]
    for n in news:
        off.append(off[-1] + n)
    q = qbuf[:, :cols].view(T, Hq, D) if not q_extra else qbuf[:, :cols].reshape(T, Hq, D)
    sc = scale or 1.0 / math.sqrt(D)
    want, bound = ref.attention(q, d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["lengths"], news,
                                masks, sc, lead)
    out = torch.full((T, cols + o_extra), 7.0, dtype=torch.bfloat16, device=DEV)
    a = bg.moe_attn_create(bg.attn_desc(Hq, Hkv, D, page, cache=cache, max_tokens=T,
                                        max_requests=len(lengths), softmax_scale=scale, rotary_dim=0), 0)
    try:
        for _ in range(calls):
            bg.moe_tree_attention(a, qbuf, T, bg.kv_cache(kc, vc, ks, vs), d["table"], i32(off),
                                  i32(d["lengths"]), out, mask=mask, q_stride=cols + q_extra,
                                  out_stride=cols + o_extra, stream=stream)
        torch.cuda.synchronize()
        assert bg.moe_attn_get_error(a) == 0
    finally:
        bg.moe_attn_destroy(a)
    got = out[:, :cols].double().view(T, Hq, D)
    assert (out[:lead] == 7).all() and (out[off[-1]:] == 7).all() and (out[:, cols:] == 7).all()
    live = slice(lead, off[-1])
    g_, w_, b_ = got[live], want[live], bound[live]
    fine = torch.isfinite(w_)
    other = ((torch.isnan(w_) != torch.isnan(g_)) | (fine != torch.isfinite(g_)) |
             (torch.isinf(w_) & torch.isinf(g_) & (w_ != g_))).nonzero()
    assert other.numel() == 0, other[:4].tolist()
    off_by = ((g_ - w_).abs() - b_)[fine]
    assert (off_by <= 0).all(), float(((g_ - w_).abs() / b_.clamp_min(1e-30))[fine].max())
    return out


SHAPES = [(16, 2, 128), (1, 1, 64), (8, 1, 256), (6, 2, 64), (7, 1, 128), (4, 4, 256), (24, 8, 64), (64, 1, 64),
          (128, 1, 64)]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
def test_attention_single_tokens(Hq, Hkv, D, cache):
    """One new token per request, contexts from none on, across page and tile ends."""
    ctx = [0, 1, 15, 16, 17, 63, 64, 126, 127, 128, 129, 255, 256, 511, 1000]
    run_attention([c + 1 for c in ctx], [1] * len(ctx), Hq, Hkv, D, 16, cache, seed=D + Hq)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_pages(D, page, cache):
    run_attention([700, 3, 257, 128], [5, 3, 1, 128], 4, 2, D, page, cache, seed=page)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 128), (8, 1, 256), (6, 2, 64), (5, 1, 128)])
def test_attention_chains(Hq, Hkv, D, cache):
    """Prompts: whole ones and chunks behind a context."""
    run_attention([1, 33, 200, 513, 300], [1, 33, 130, 257, 1], Hq, Hkv, D, 32, cache, seed=Hq)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("words,new", [(1, [1, 2, 33, 64]), (2, [65, 128, 7]), (4, [256, 200, 3]), (1, [5, 80, 64])])
def test_attention_trees(words, new, cache):
    """Trees of all word counts; the last case has tokens past the words, seen by none."""
    h = torch.Generator().manual_seed(words)
    ctx = torch.randint(0, 400, (len(new),), generator=h).tolist()
    masks = [ref.random_tree(h, n, max(words, -(-n // 64))) for n in new]
    masks = [[r[:words] for r in m] for m in masks]
    run_attention([c + n for c, n in zip(ctx, new)], new, 6, 2, 128, 16, cache, words, masks=masks)


def test_attention_empty_rows():
    """Masks that leave a row nothing (no context), requests that are not served, idle ones."""
    n = [4, 3, 0, 5, 2]
    masks = [[[0], [2], [0], [8]], [[0], [0], [0]], [], [[0]] * 5, [[1], [2]]]
    out = run_attention([4, 3, 50, 4, 302], n, 4, 2, 64, 16, words=1, masks=masks)
    assert (out[0] == 0).all() and (out[2] == 0).all() and (out[4:7] == 0).all() and (out[7:12] == 0).all()
    run_attention([0, 0, 30], [3, 1, 0], 4, 2, 128, 32)
    run_attention([0], [1], 4, 2, 256, 32, cache="e4m3")


@pytest.mark.parametrize("D,cache", [(64, "bf16"), (128, "bf16"), (256, "e4m3"), (128, "e4m3")])
def test_attention_garbage_behind_the_length(D, cache):
    """The rest of the last page and unused pages hold NaNs and infinities."""
    def edit(d):
        bad = torch.tensor([float("nan")], device=DEV).to(d["kc"].dtype)
        page = 64
        used = torch.zeros(d["kc"].shape[0], page, dtype=torch.bool)
        for b, L in enumerate(d["lengths"]):
            for j in range(L):
                used[int(d["table"][b, j // page]), j % page] = True
        raw = torch.uint8 if d["kc"].dtype == torch.float8_e4m3fn else torch.int16
        for c in (d["kc"], d["vc"]):
            c.view(raw).permute(0, 2, 1, 3)[~used.to(DEV)] = bad.view(raw)
    run_attention([100, 1, 129, 64, 300], [1, 1, 5, 64, 170], 8, 2, D, 64, cache, edit=edit)


@pytest.mark.parametrize("D,cache", [(64, "bf16"), (128, "e4m3"), (256, "bf16")])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_attention_masked_infinities(D, cache, value):
    """A new token's key or value that is no number reaches the rows that see it and no others."""
    if cache == "e4m3" and not math.isnan(value):
        pytest.skip("e4m3 has no infinities")
    n, L = 40, 140
    h = torch.Generator().manual_seed(9)

    def edit(d):
        put = lambda c, j, h_: c.view(raw)[int(d["table"][0, j // 16]), h_, j % 16].copy_(bad)
        raw = torch.uint8 if cache == "e4m3" else torch.int16
        row = torch.zeros(D, device=DEV)
        row[3::5] = value
        bad = row.to(d["kc"].dtype).view(raw)
        put(d["vc"], L - n + 5, 0)
        put(d["vc"], L - n + 30, 1)
        if math.isnan(value):
            put(d["kc"], L - n + 9, 1)
    for masks, words in ((None, 0), ([ref.random_tree(h, n, 1)], 1)):
        run_attention([L], [n], 4, 2, D, 16, cache, words, masks=masks, edit=edit)


def test_attention_infinities_in_context():
    """Every row sees the context's: infinite values, and keys whose scores are -inf."""
    def edit(d):
        d["vc"][int(d["table"][0, 1]), 0, 3, 5] = float("inf")
        d["vc"][int(d["table"][0, 1]), 1, 3, 6] = -float("inf")
        d["kc"][int(d["table"][0, 2]), 0, 4, :] = 0
        d["kc"][int(d["table"][0, 2]), 0, 4, 0] = -float("inf")
        d["q"][:, 0::128] = d["q"][:, 0::128].abs() + 0.5
    run_attention([150], [20], 2, 2, 128, 16, edit=edit)


@pytest.mark.parametrize("spread,scale", [(60.0, 0.0), (1e-3, 0.0), (1.5, 3.0), (1.5, 1e-6)])
def test_attention_scores_of_all_sizes(spread, scale):
    """Flat and peaked softmaxes; running maxima that grow late."""
    run_attention([600, 1500], [70, 9], 4, 1, 128, 64, spread=spread, scale=scale)


def test_attention_maximum_at_the_end():
    """Scores that rise along the keys by far more than an exponent's range."""
    def edit(d):
        for b, L in enumerate(d["lengths"]):
            j = torch.arange(L, device=DEV)
            at = d["table"][b].long()[j // 32]
            d["kc"][at, :, j % 32, 0] = (j * 2.0).bfloat16()[:, None]
        d["q"][:, 0::64] = 20.0
    run_attention([900, 40], [3, 40], 2, 1, 64, 32, edit=edit)


def test_attention_tail_of_many_small_weights():
    """One key far above thousands of equal ones, which hold most of the weight together."""
    for cache in ("bf16", "e4m3"):
        def edit(d):
            d["kc"].zero_()
            d["q"].zero_()
            d["q"][:, 0::128] = 8.0
            first = int(d["table"][0, 0])
            d["kc"][first, 0, 0, 0] = 14.0 if cache == "bf16" else 448.0
            if d["ks"] is not None:
                d["ks"].fill_(14.0 / 448.0)
        run_attention([9000], [1], 1, 1, 128, 64, cache, edit=edit)


def test_attention_strides_and_leading_rows():
    run_attention([50, 90], [3, 20], 4, 2, 64, 16, lead=5, pad=4, q_extra=72, o_extra=8)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_attention_many_requests(cache):
    h = torch.Generator().manual_seed(1)
    new = torch.randint(0, 4, (700,), generator=h).tolist()
    lengths = [n + int(torch.randint(0, 40, (1,), generator=h)) for n in new]
    run_attention(lengths, new, 4, 2, 64, 16, cache)


@pytest.mark.parametrize("Hq,Hkv,D,n,words", [(16, 2, 128, 1, 0), (8, 1, 256, 16, 1), (4, 4, 64, 64, 1), (2, 1, 128, 300, 0)])
def test_attention_long_context_is_shared_by_sms(Hq, Hkv, D, n, words):
    run_attention([20011], [n], Hq, Hkv, D, 64, words=words, calls=2)


def test_attention_refuses_pages_outside_the_cache():
    """A wrong table entry and a length past the table set the error and read nothing."""
    g = torch.Generator(device=DEV).manual_seed(0)
    kc, vc, _, _ = ref.cache_of(g, 4, 1, 16, 64, "bf16")
    q = torch.randn(2, 64, generator=g, device=DEV).bfloat16()
    out = torch.zeros(2, 64, dtype=torch.bfloat16, device=DEV)
    a = bg.moe_attn_create(bg.attn_desc(1, 1, 64, 16, max_tokens=2, rotary_dim=0), 0)
    cache = bg.kv_cache(kc, vc)
    run = lambda table, off, length: bg.moe_tree_attention(a, q, 2, cache, i32(table), i32(off),
                                                           i32(length), out)
    try:
        for page in (4, -1, 2 ** 31 - 1, -2 ** 31):
            run([[0, page, 1]], [0, 2], [40])
            assert bg.moe_attn_get_error(a) == 6
            assert torch.isfinite(out.float()).all()
        assert bg.moe_attn_get_error(a) == 0
        run([[0, 2, 1]], [0, 2], [49])
        assert bg.moe_attn_get_error(a) == 6
        # wrong entries behind the length are not looked at; wrong offsets stay within the rows
        run([[0, -5, 99]], [0, 2], [16])
        run([[0, 2, 1]], [-3, 2 ** 31 - 1], [16])
        run([[0, 2, 1], [0, 1, 2]], [2, 0, 2 ** 31 - 1], [16, 30])
        assert bg.moe_attn_get_error(a) == 0
    finally:
        bg.moe_attn_destroy(a)


def test_attention_repeats_and_graphs():
    """The same bits on every run, on another stream, and in a replayed graph with new lengths."""
    g = torch.Generator(device=DEV).manual_seed(3)
    B, Hq, Hkv, D, page = 3, 8, 2, 128, 16
    lengths, off = i32([700, 90, 40]), i32([0, 1, 3, 10])
    table, pages = ref.table_of(torch.Generator().manual_seed(0), [800] * B, page)
    kc, vc, _, _ = ref.cache_of(g, pages, Hkv, page, D, "bf16")
    q = torch.randn(10, Hq * D, generator=g, device=DEV).bfloat16()
    out = torch.zeros_like(q)
    a = bg.moe_attn_create(bg.attn_desc(Hq, Hkv, D, page, max_tokens=16, rotary_dim=0), 0)
    cache = bg.kv_cache(kc, vc)
    run = lambda: bg.moe_tree_attention(a, q, 10, cache, table, off, lengths, out)
    try:
        run()
        first = out.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(3):
                out.zero_()
                run()
                assert torch.equal(out, first)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for new in ([700, 90, 40], [20, 799, 7], [3, 2, 650]):
            lengths.copy_(i32(new))
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone()
            out.zero_()
            run()
            torch.cuda.synchronize()
            assert torch.equal(out, got)
        assert bg.moe_attn_get_error(a) == 0
    finally:
        bg.moe_attn_destroy(a)


def test_refusals_with_a_handle():
    """Wrong arguments of the calls that need a handle: nothing is launched."""
    from bit_grouped_gemm_gb300 import binding
    import ctypes
    lib = binding.load_library()
    A, FAR = 1 << 30, 1 << 36
    handle = {k: bg.moe_attn_create(bg.attn_desc(8, 2, 64, 16, cache=k, max_tokens=32, max_requests=4), 0)
              for k in ("bf16", "e4m3")}

    def cache(kind, **kw):
        f = dict(k=A, v=A + FAR, k_scale=None, v_scale=None, pages=10)
        if kind == "e4m3":
            f.update(k_scale=A + 2 * FAR, v_scale=A + 3 * FAR)
        f.update(kw)
        return ctypes.byref(bg.MoeKvCache(**f))

    def rope(kind="bf16", q=A + 4 * FAR, ql=0, k=A + 5 * FAR, kl=0, v=A + 6 * FAR, vl=0, T=4, pos=A + 7 * FAR,
             slot=A + 8 * FAR, out=A + 9 * FAR, ol=0, **c):
        return lib.moe_rope_store(handle[kind], q, ql, k, kl, v, vl, T, pos, slot, out, ol, cache(kind, **c),
                                  None)

    def attn(kind="bf16", q=A + 4 * FAR, ql=0, T=4, table=A + 5 * FAR, width=4, B=2, off=A + 6 * FAR,
             length=A + 7 * FAR, mask=A + 8 * FAR, words=1, out=A + 9 * FAR, ol=0, **c):
        return lib.moe_tree_attention(handle[kind], q, ql, T, cache(kind, **c), table, width, B, off, length,
                                      mask, words, out, ol, None)

    try:
        for call in (rope, attn):
            for kw, status in [
                    (dict(k_scale=A), 1), (dict(kind="e4m3", v_scale=None), 1), (dict(pages=0), 1),
                    (dict(pages=1 << 27), 2), (dict(kind="e4m3", k_scale=A + 2 * FAR + 2), 1),
                    (dict(q=None), 1), (dict(q=A + 4 * FAR + 8), 1), (dict(T=0), 1), (dict(T=33), 4),
                    (dict(ql=504), 1), (dict(ql=516), 1), (dict(ol=8), 1), (dict(out=None), 1),
                    (dict(out=A), 1), (dict(out=A + FAR + 16), 1), (dict(out=A + 9 * FAR + 2), 1),
                    (dict(ql=1 << 31), 1)]:
                assert call(**kw) == status, (call, kw)
        for kw, status in [(dict(k=None), 1), (dict(v=None), 1), (dict(k=A + 8), 1), (dict(kl=120), 1),
                           (dict(vl=132), 1), (dict(pos=None), 1), (dict(slot=A + 2), 1), (dict(slot=None), 1),
                           (dict(out=A + 4 * FAR + 16), 1), (dict(out=A + 4 * FAR, ol=1024), 1),
                           (dict(out=A + 5 * FAR), 1), (dict(q=A + 9 * FAR, ql=768, ol=768, vl=768, k=A + 9 * FAR + 512), 1),
                           (dict(out=A + 7 * FAR), 1), (dict(kind="e4m3", out=A + 2 * FAR), 1)]:
            assert rope(**kw) == status, kw
        for kw, status in [(dict(table=None), 1), (dict(width=0), 1), (dict(width=(1 << 18) + 1), 2), (dict(B=0), 1),
                           (dict(B=5), 4), (dict(off=None), 1), (dict(length=None), 1), (dict(mask=None), 1),
                           (dict(words=0), 1), (dict(words=5), 1), (dict(mask=A + 8 * FAR + 4), 1),
                           (dict(table=A + 2), 1), (dict(out=A + 5 * FAR), 1), (dict(out=A + 8 * FAR), 1),
                           (dict(out=A + 4 * FAR), 1), (dict(v=A + 8), 1)]:
            assert attn(**kw) == status, kw
    finally:
        for a in handle.values():
            bg.moe_attn_destroy(a)


@pytest.mark.parametrize("Hq,Hkv,D,cache", [(2, 1, 64, "bf16"), (6, 2, 128, "e4m3"), (4, 1, 256, "bf16"), (16, 2, 128, "bf16")])
def test_attention_many_key_tiles_per_sm(Hq, Hkv, D, cache):
    """Batches in which every SM goes through many key tiles with few query rows."""
    B = 160 // Hkv
    h = torch.Generator().manual_seed(D)
    lengths = torch.randint(600, 1800, (B,), generator=h).tolist()
    run_attention(lengths, [1 + b % 3 for b in range(B)], Hq, Hkv, D, 64, cache)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_zero_rows_between_others(D, cache):
    """Requests without keys in long runs between served ones, on few and on many SMs."""
    for rep in (1, 40):
        lengths, news = [], []
        for i in range(rep):
            lengths += [200 + i, 0, 0, 0, 0, 0, 0, 33, 0, 5]
            news += [1, 1, 2, 1, 1, 1, 3, 2, 1, 5]
        run_attention(lengths, news, 4, 2, D, 16, cache)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 64), (16, 2, 128), (3, 1, 128), (4, 4, 64), (7, 1, 64)])
def test_attention_prompts_of_many_row_tiles(Hq, Hkv, D, cache):
    """Long chains, whose row tiles go two by two; odd ends of rows and of keys, several requests."""
    run_attention([900, 333, 1500], [900, 200, 517], Hq, Hkv, D, 32, cache, seed=Hq)


def test_attention_prompts_with_numbers_that_are_none():
    def edit(d):
        d["vc"][int(d["table"][0, 300 // 16]), 0, 300 % 16, 3::7] = float("nan")
        d["vc"][int(d["table"][0, 555 // 16]), 0, 555 % 16, 1::9] = float("inf")
    run_attention([600], [590], 4, 1, 64, 16, edit=edit)
    run_attention([600], [590], 4, 1, 128, 16, edit=edit)
