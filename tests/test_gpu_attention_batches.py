"""Attention over a paged cache where the call and the batch differ in size: fewer rows than the
batch's step has, and few requests with new tokens among many idle ones."""
import math

import pytest
import torch

import bit_grouped_gemm_gb300 as bg

from . import attention_ref as ref
from .attention_ref import DEV, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_grouped_gemm_gb300 import build
    build.build()


class Batch:
    """A call on random inputs, its rows checked against the 64-bit definition of the whole batch."""

    def __init__(self, lengths, news, Hq=4, Hkv=2, D=64, page=16, cache="bf16", words=0, limit=0, seed=0):
        g, h = torch.Generator(device=DEV).manual_seed(seed), torch.Generator().manual_seed(seed)
        self.lengths, self.news, self.Hq, self.D, self.T = lengths, news, Hq, D, sum(news)
        self.table, pages = ref.table_of(h, [max(n, 0) for n in lengths], page)
        self.kc, self.vc, self.ks, self.vs = ref.cache_of(g, pages, Hkv, page, D, cache)
        self.cache = bg.kv_cache(self.kc, self.vc, self.ks, self.vs)
        self.q = torch.randn(self.T, Hq * D, generator=g, device=DEV).bfloat16()
        self.out = torch.full_like(self.q, 7.0)
        self.masks = [ref.random_tree(h, n, words) for n in news] if words else None
        self.mask = torch.tensor([r for m in self.masks for r in m], dtype=torch.int64,
                                 device=DEV) if words else None
        off = [0]
        for n in news:
            off.append(off[-1] + n)
        self.off, self.length = i32(off), i32(lengths)
        self.attn = bg.moe_attn_create(bg.attn_desc(Hq, Hkv, D, page, cache=cache, max_tokens=self.T,
                                                    max_requests=len(lengths), rotary_dim=0,
                                                    wait_limit_ms=limit), 0)

    def __enter__(self):
        return self

    def __exit__(self, *_):
        bg.moe_attn_destroy(self.attn)

    def run(self, T=None):
        bg.moe_tree_attention(self.attn, self.q, T or self.T, self.cache, self.table, self.off, self.length,
                              self.out, mask=self.mask)

    def check(self, T=None):
        """The first T rows are the whole batch's, the others as they were."""
        T = T or self.T
        torch.cuda.synchronize()
        assert bg.moe_attn_get_error(self.attn) == 0
        want, bound = ref.attention(self.q.view(self.T, self.Hq, self.D), self.kc, self.vc, self.ks, self.vs,
                                    self.table, self.lengths, self.news, self.masks, 1 / math.sqrt(self.D))
        got = self.out.double().view(self.T, self.Hq, self.D)
        assert ((got - want).abs() <= bound)[:T].all()
        assert (self.out[T:] == 7.0).all()


@pytest.mark.parametrize("cache,D", [("bf16", 64), ("e4m3", 128), ("bf16", 256)])
@pytest.mark.parametrize("words", [0, 1])
@pytest.mark.parametrize("T", [1, 2, 30, 31, 42, 91])
def test_fewer_rows_than_the_batch_has(cache, D, words, T):
    """The batch has 92 rows, the call fewer: its rows keep their contexts."""
    with Batch([40, 30, 300, 60], [1, 30, 11, 50], D=D, cache=cache, words=words) as b:
        b.run(T)
        b.check(T)


def test_a_prompt_cut_after_some_row_tiles():
    with Batch([1100], [1000], Hq=8, Hkv=1, D=128) as b:
        b.run(333)
        b.check(333)


def idle_but(at, B, L, n=1):
    """Lengths and new tokens of a batch in which only the requests `at` have any."""
    lengths, news = [17 + b % 5 for b in range(B)], [0] * B
    for b in at:
        lengths[b], news[b] = L, n
    return lengths, news


@pytest.mark.parametrize("cache,D", [("bf16", 128), ("e4m3", 64)])
@pytest.mark.parametrize("at", [[0], [2100], [4095], [0, 4095], [0, 1, 33, 64, 66, 2000, 4094], list(range(3, 4096, 97)),
                                list(range(1000, 1300))])
def test_few_requests_among_4096(cache, D, at):
    """Idle requests in front, between and behind, under a wait limit of 1 ms."""
    lengths, news = idle_but(at, 4096, 500)
    lengths[at[-1]], news[at[-1]] = 1500, 3
    with Batch(lengths, news, D=D, cache=cache, limit=1) as b:
        b.run()
        b.check()


def test_served_and_unserved_requests_among_idle_ones():
    """Requests that get no keys (zeros) and idle ones, in runs of all lengths up to 40."""
    lengths, news = [], []
    for i in range(40):
        lengths += [300 + i, 1] + [9] * i
        news += [1 + i % 3, 2] + [0] * i
    with Batch(lengths, news, D=64, limit=1) as b:
        b.run()
        b.check()


def graph_ms(run):
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(10):
            run()
    times = []
    for _ in range(7):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        graph.replay()
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) / 10)
    return sorted(times)[3]


def test_idle_requests_behind_the_last_one_take_no_time():
    """One token takes the same time whether the idle requests of a batch come before or behind it:
    the SM that has it does not go through those behind, one after the other (717 against 79 us)."""
    took = []
    for at in (4095, 0):
        with Batch(*idle_but([at], 4096, 2000), Hq=16, Hkv=2, D=128, page=64) as b:
            took.append(graph_ms(b.run))
            b.check()
    assert took[1] < 3 * took[0], took


@pytest.mark.parametrize("idle,n", [(100000, 0), (9000, 0), (0, 3)])
def test_requests_without_keys_to_read_do_not_change_the_split(idle, n):
    """A token beside a long idle context, or beside rows without keys, is shared by the SMs as
    alone: the same sums in the same order."""
    with Batch([2000], [1], Hq=16, Hkv=2, D=128, page=64) as b:
        b.run()
        b.check()
        want = b.out.clone()
    with Batch([2000, idle], [1, n], Hq=16, Hkv=2, D=128, page=64) as b:
        # the same inputs
        with Batch([2000], [1], Hq=16, Hkv=2, D=128, page=64) as one:
            b.q[:1] = one.q
            for mine, its in ((b.kc, one.kc), (b.vc, one.vc)):
                mine[b.table[0, :32].long()] = its[one.table[0, :32].long()]
        b.run()
        b.check()
        assert torch.equal(b.out[:1], want)
