"""A batch served through CachedAttention on the pages of a PagedBatch, step after step
as it would be: a prompt's chunks, single tokens, drafted trees, requests that end and
others that take their pages; alone, replayed from a graph, and in a stack with experts."""
import dataclasses
import math

import pytest
import torch

import bit_grouped_gemm_gb300 as bg
from bit_grouped_gemm_gb300 import stack, synth

from . import attention_ref as ref
from .attention_ref import DEV, i32

pytestmark = pytest.mark.gpu

H, HQ, HKV, D, PAGE, M, B = 256, 8, 2, 64, 16, 160, 4
FREQS = ref.frequencies(D)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_grouped_gemm_gb300 import build
    build.build()


def weights(g, n, k):
    q = torch.randint(-2 ** 31, 2 ** 31 - 1, (n, k // 8), generator=g, device=DEV, dtype=torch.int64)
    s = (0.02 + 0.02 * torch.rand(n, k // 64, generator=g, device=DEV)).bfloat16()
    return q.to(torch.int32), s, (-7.5 * s.float()).bfloat16()


class Layer:
    """A layer with caches, and its attention's handle."""

    def __init__(self, seed, cache, pages, adapters=True, rows=M):
        g = torch.Generator(device=DEV).manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device=DEV)
        cols = (HQ + 2 * HKV) * D
        self.k, self.v, self.ks, self.vs = ref.cache_of(g, pages, HKV, PAGE, D, cache)
        self.a, self.b = (r(3, 16, H) / 16).bfloat16(), (0.2 * r(3, cols, 16)).bfloat16()
        d = bg.attn_desc(HQ, HKV, D, PAGE, cache=cache, max_tokens=rows, max_requests=B)
        self.attn = bg.moe_attn_create(d, 0)
        self.qkv_w, self.out_w = weights(g, cols, H), weights(g, H, HQ * D)
        self.norm = (1 + 0.2 * r(H)).bfloat16()
        self.layer = stack.CachedAttention(self.attn, d, self.norm, self.qkv_w, self.out_w, self.k, self.v,
                                           self.ks, self.vs, bg.lora(self.a, self.b) if adapters else None,
                                           rows, alpha=0.5)

    def close(self):
        self.layer.close()
        bg.moe_attn_destroy(self.attn)

    def errors(self):
        L = self.layer
        return [bg.moe_attn_get_error(self.attn)] + [bg.moe_linear_get_error(h) for h in (L.project, L.output)]


class Served:
    """What a host would know of the batch: contexts, and which requests go on."""

    def __init__(self, words=0, pages=40, rows=M):
        self.batch = stack.PagedBatch(B, PAGE, 12, pages, rows, words)
        self.context = [0] * B

    def step(self, added, parent=None):
        rows = sum(max(n, 0) for n in added)
        if parent is not None:
            parent = i32(parent + [-1] * (self.batch.desc.max_tokens - rows))
        self.batch.step(i32(self.context), i32(added), parent)
        self.context = [0 if n < 0 else c + n for c, n in zip(self.context, added)]
        return rows


def close(got, want, tol):
    assert ((got.double() - want).abs() <= tol).all()


def check_step(L, s, added, x0, y0, ids, masks, pad):
    """One step, each operator's output against the 64-bit one on the library's own input to it."""
    layer, batch = L.layer, s.batch
    rows = sum(max(n, 0) for n in added)
    T = rows + pad
    before = L.k.clone(), L.v.clone()
    x = x0.clone()
    layer(x, y0, batch, ids)
    torch.cuda.synchronize()
    assert L.errors() == [0, 0, 0]
    lengths = [0 if n < 0 else c for n, c in zip(added, s.context)]
    assert batch.length.tolist() == lengths and batch.status.tolist()[2:] == [0, 0, 0]
    # the rows before they are turned, by the same projection
    raw = torch.empty_like(layer.qkv)
    bg.moe_linear_forward(layer.project, layer.h8, T, layer.qkv_c, raw, x_scale=layer.hs,
                          lora=layer.adapters if ids is not None else None, adapter=ids)
    q, k, v = (t.double().view(T, -1, D) for t in raw[:T].split([HQ * D, HKV * D, HKV * D], 1))
    pos, slot = batch.position[:T], batch.slot[:T].long()
    assert (slot[:rows] >= 0).all() and (slot[rows:] == -1).all()
    assert len(set(slot[:rows].tolist())) == rows
    yq, yk = ref.turn(q, pos, FREQS, "half"), ref.turn(k, pos, FREQS, "half")
    tol = lambda y: 2.0 ** -8 * y.abs() + y.abs().amax(2, keepdim=True) * 2.0 ** -20
    close(layer.qkv[:T, :HQ * D].view(T, HQ, D), yq, tol(yq))
    at = slot[:rows]
    for now, old, want, scale in ((L.k, before[0], yk, L.ks), (L.v, before[1], v, L.vs)):
        rest = torch.ones(now.shape[0] * PAGE, dtype=torch.bool, device=DEV)
        rest[at] = False
        flat = lambda t: t.float().transpose(1, 2).reshape(-1, HKV, D)
        assert torch.equal(flat(now)[rest], flat(old)[rest])
        want, t = want[:rows], tol(want)[:rows]
        if scale is not None:
            want = (want / scale.double()[:, None]).clamp(-448, 448)
            t = torch.maximum(2.0 ** -4 * want.abs(), torch.full_like(want, 2.0 ** -10)) + 100 * t
        close(flat(now)[at], want, t)
    news = [max(n, 0) for n in added]
    want, bound = ref.attention(layer.qkv[:T, :HQ * D].reshape(T, HQ, D), L.k, L.v, L.ks, L.vs, batch.table,
                                lengths, news, masks, 1 / math.sqrt(D))
    close(layer.a[:rows].view(rows, HQ, D), want[:rows], bound[:rows])
    d = torch.empty_like(layer.d)
    bg.moe_linear_forward(layer.output, layer.a, T, layer.out_c, d)
    x1 = x0.double() + (0.5 * y0.double() if y0 is not None else 0.0)
    want = x1 + d[:T].double()
    close(x[:rows], want[:rows], (want.abs() * 2.0 ** -8 + x1.abs() * 2.0 ** -8 + 1e-30)[:rows])


STEPS = [  # new tokens of each request (negative: it ends), and whether they are trees
    ([37, 5, 64, 0], False), ([1, 1, 1, 20], False), ([1, -1, 1, 1], False), ([5, 33, 1, 7], True),
    ([1, 1, -1, 12], True), ([0, 2, 90, 0], False), ([1, 1, 1, 1], True), ([-1, -1, -1, -1], False),
    ([60, 1, 0, 30], False),
]


@pytest.mark.parametrize("adapters", [True, False])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("words", [0, 2])
def test_a_batch_from_prompts_to_the_end(cache, words, adapters):
    L, s = Layer(1, cache, 40, adapters), Served(words)
    g, h = torch.Generator(device=DEV).manual_seed(2), torch.Generator().manual_seed(2)
    for i, (added, tree) in enumerate(STEPS):
        parent = masks = None
        if words:
            parent = [int(torch.randint(-1, j, (1,), generator=h)) if j and tree else j - 1
                      for n in added for j in range(max(n, 0))]
        rows = s.step(added, parent)
        if words:
            masks, r = [], 0
            for n in added:
                m = []
                for j in range(max(n, 0)):
                    own = list(m[parent[r + j]]) if parent[r + j] >= 0 else [0] * words
                    own[j // 64] |= 1 << (j % 64)
                    m.append(own)
                masks.append(m)
                r += max(n, 0)
        pad = 3 if i % 2 else 0
        if rows + pad == 0:
            continue
        x = torch.randn(rows + pad, H, generator=g, device=DEV).bfloat16()
        y = torch.randn(rows + pad, H, generator=g, device=DEV) if i % 3 else None
        ids = torch.randint(-1, 3, (rows + pad,), generator=h).to(torch.int32).to(DEV) if adapters else None
        check_step(L, s, added, x, y, ids, masks, pad)
    free = int(s.batch.ring_pos[1]) + int(s.batch.owned.sum())
    assert free == 40
    L.close()


def test_requests_that_get_no_pages_wait_for_others():
    """Too few pages: a request is refused, its rows are zeros and store nothing, and it is
    served once another's end has freed some."""
    L, s = Layer(3, "bf16", 6), Served(pages=6)
    x = lambda n: torch.randn(n, H, device=DEV).bfloat16()
    s.batch.step(i32([0] * B), i32([60, 50, 0, 0]))
    L.layer(x(110), None, s.batch)
    torch.cuda.synchronize()
    assert s.batch.status.tolist()[:4] == [110, 4, 1, 2] and s.batch.length.tolist() == [60, 0, 0, 0]
    assert (L.layer.a[60:110] == 0).all() and (L.layer.a[:60] != 0).any() and L.errors() == [0] * 3
    s.batch.step(i32([60, 0, 0, 0]), i32([-1, 0, 0, 0]))
    s.batch.step(i32([0] * B), i32([0, 50, 0, 0]))
    L.layer(x(50), None, s.batch)
    torch.cuda.synchronize()
    assert s.batch.length.tolist() == [0, 50, 0, 0] and (L.layer.a[:50] != 0).any()
    L.close()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_two_layers_and_experts_in_one_graph(cache):
    """Attention, experts, attention on two layers' caches: a captured step, replayed on new
    lengths and tokens, gives the bits of calls one by one, on a state of its own."""
    shape = synth.MoEShape(hidden=H, inter=256, num_experts=16, top_k=2)
    w = dataclasses.replace(synth.standard_workloads()["t128_uniform"], shape=shape, tokens=M)
    plan = bg.moe_plan_create(bg.plan_desc(hidden=H, inter=256, num_experts=16, top_k=2, max_tokens=M), 0)
    experts = stack.make_layer(w, 0, "cuda")
    g = torch.Generator(device=DEV).manual_seed(7)
    one = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    proj = weights(g, H, H)

    class State:
        def __init__(self):
            self.at = [Layer(5, cache, 40), Layer(6, cache, 40)]
            self.ffn = stack.AdaptedLayer(plan, experts, one, one, proj, bg.score_desc(), max_tokens=M, alpha=0.5)
            self.batch = stack.PagedBatch(B, PAGE, 12, 40, M)
            self.context, self.added = i32([0] * B), i32([0] * B)
            self.x = torch.zeros(M, H, dtype=torch.bfloat16, device=DEV)
            self.ids = torch.full((M,), -1, dtype=torch.int32, device=DEV)

        def run(self):
            self.batch.step(self.context, self.added)
            self.at[0].layer(self.x, None, self.batch, self.ids)
            y = self.ffn(self.x, None)
            self.at[1].layer(self.x, y, self.batch, self.ids)

        def close(self):
            for a in self.at:
                a.close()
            self.ffn.close()

    eager, replayed = State(), State()
    replayed.run()                       # (an empty step: nothing is stored)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed.run()
    context = [0] * B
    for added in ([70, 9, 33, 2], [1, 1, 1, 1], [1, -1, 17, 1], [1, 40, 1, -1], [2, 2, 2, 2]):
        rows = sum(max(n, 0) for n in added)
        x = torch.randn(M, H, generator=g, device=DEV).bfloat16()
        ids = torch.randint(-1, 3, (M,), generator=g, device=DEV).to(torch.int32)
        for s in (eager, replayed):
            for to, new in ((s.x, x), (s.ids, ids), (s.context, i32(context)), (s.added, i32(added))):
                to.copy_(new)
        eager.run()
        graph.replay()
        torch.cuda.synchronize()
        context = [0 if n < 0 else c + n for c, n in zip(context, added)]
        assert torch.equal(eager.x[:rows], replayed.x[:rows]) and torch.isfinite(eager.x[:rows].float()).all()
        for a, b in zip(eager.at, replayed.at):
            assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8))
            assert torch.equal(a.v.view(torch.uint8), b.v.view(torch.uint8))
            assert a.errors() == [0] * 3 and b.errors() == [0] * 3
        assert torch.equal(eager.batch.table, replayed.batch.table)
        assert eager.batch.length.tolist() == context
    assert bg.moe_get_error(plan) == 0
    eager.close()
    replayed.close()
    bg.moe_plan_destroy(plan)


def test_two_layers_of_two_batches_on_two_streams():
    """Handles of their own: two batches' steps at once give the bits of one after the other."""
    added = [150, 3, 1, 1]
    g = torch.Generator(device=DEV).manual_seed(11)
    xs = [torch.randn(sum(added), H, generator=g, device=DEV).bfloat16() for _ in range(2)]

    def run(streams):
        out = []
        states = [(Layer(20 + i, "bf16", 40), Served()) for i in range(2)]
        for rep in range(4):
            got = []
            for (L, s), x0, st in zip(states, xs, streams):
                with torch.cuda.stream(st):
                    s.batch.step(i32([0, 0, 0, 0]), i32(added if rep % 2 == 0 else [-1] * B))
                    x = x0.clone()
                    if rep % 2 == 0:
                        L.layer(x, None, s.batch)
                    got.append(x)
            torch.cuda.synchronize()
            out.append(got)
        for L, _ in states:
            assert L.errors() == [0] * 3
            L.close()
        return out

    torch.cuda.synchronize()
    here = torch.cuda.current_stream()
    want = run([here, here])
    got = run([torch.cuda.Stream(), torch.cuda.Stream()])
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_the_first_step_may_come_on_another_stream():
    """A batch and a layer made on a stream that is busy, used at once on another one: their first
    state is there."""
    want = None
    x0 = torch.randn(70, H, generator=torch.Generator(device=DEV).manual_seed(13), device=DEV).bfloat16()
    context, added = i32([0] * B), i32([60, 3, 0, 2])
    for rep in range(3):
        torch.full((1 << 20,), 2 ** 30 + 5, dtype=torch.int32, device=DEV)     # (what the allocator hands out next)
        torch.cuda.synchronize()
        makes, runs = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(makes):
            torch.cuda._sleep(50 * 10 ** 6)
            s = Served()
        with torch.cuda.stream(runs):
            s.batch.step(context, added)
        torch.cuda.synchronize()
        assert s.batch.status.tolist() == [65, 6, 0, 0, 0] and s.batch.length.tolist() == [60, 3, 0, 2]
        assert s.batch.table[:, 0].tolist() == [0, 4, 0, 5] and s.batch.ring_pos.tolist() == [6, 34]
        with torch.cuda.stream(makes):
            L = Layer(1, "bf16", 40, adapters=False)
            torch.cuda._sleep(50 * 10 ** 6)
            layer = stack.CachedAttention(L.attn, L.layer.desc, L.norm, L.qkv_w, L.out_w, L.k, L.v, max_tokens=M)
        with torch.cuda.stream(runs):
            x = x0.clone()
            layer(x, None, s.batch)
        torch.cuda.synchronize()
        assert (layer.a[65:70] == 0).all()
        want = x if want is None else want
        assert torch.equal(x, want)
        layer.close()
        L.close()
