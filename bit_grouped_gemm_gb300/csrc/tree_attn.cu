// tree_attn.cu -- attention of new tokens, chains or drafted trees, over a paged
// cache, on the 5th-generation tensor cores (moe_tree_attention).
//
//   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  s_j = scale q . k_j
//
// in one pass over the keys with a running maximum m.
//
//   * A row tile is up to 128 query rows of one request and key-value head: R =
//     128 / G tokens times the G query heads that share the head's keys, so one
//     read of a key serves all of them. Its keys come in tiles of 128.
//   * Scores: S = Q K^T (M 128, N 128, K head_dim), Q and K in shared memory as
//     chunks of 64 columns (128-byte rows, 128-byte swizzle), S in tensor memory,
//     two buffers. Two groups of 4 warps take 64 columns each of every row, one
//     row per thread; the weights go back into the scores' place as bf16, and
//     O += P V takes them from there (V as stored: its keys are the product's K,
//     so it is the operand with the other major order). The product of the next
//     tile's scores runs while a tile's weights are computed.
//   * The maximum that weights refer to is moved, and O in tensor memory scaled,
//     only when a row's maximum has grown by 2^8: weights stay below 2^8, far
//     from overflow, and the sums are exact in the same way.
//   * Keys and values arrive by TMA, a box per page. An 8-bit cache is converted
//     to bf16 (exact) by 4 further warps between its own ring and the operands'.
//   * A split of the keys gives every CTA the same work: all row tiles side by
//     side, each as long as its keys, are cut into equal lengths, one per CTA, at
//     tile borders. A row tile that several CTAs share leaves its parts' sums in
//     scratch, and a second kernel joins them.
//   * Rows differ in the keys that they see only from the first new token on;
//     tiles past it are masked. What is not seen may be infinite or NaN: scores
//     are replaced, and values that some row must not see are set to zero in
//     shared memory (their NaN times weight 0 would be NaN) and, in rows that do
//     see them, added at the end.
#include "attn.h"
#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kSlotBytes = 128 * 128;       // 128 rows of 64 bf16
constexpr int kRawBytes = 128 * 64;         // 128 rows of 64 e4m3
constexpr int kSoftWarps = 8, kLoadWarp = 8, kMmaWarp = 9, kConvWarp = 10, kConvWarps = 4;
constexpr int kItemCost = 128;              // of a row tile beside its keys, in keys
constexpr uint32_t kTmemCols = 512, kColS = 256;
constexpr float kGrowth = 8.0f;             // log2 by which a maximum may be exceeded
constexpr int kMiscBytes = 4096;

template <int D, bool E>
struct Shape {
  static constexpr int NC = D / 64;
  static constexpr int kThreads = 32 * (E ? kConvWarp + kConvWarps : kConvWarp);
  // operand slots, and (8-bit) slots of codes, in what Q leaves of 227 KB
  static constexpr int kSlots = E ? (D == 256 ? 5 : 6) : (D == 256 ? 9 : 10);
  static constexpr int kRaw = E ? (D == 256 ? 8 : 10) : 0;
  static constexpr int kSmem = 1024 + kMiscBytes + (NC + kSlots) * kSlotBytes + kRaw * kRawBytes;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kSlots > NC, "a tile's values and a chunk beside them");
};

struct TaParams {
  CUtensorMap mq, mk, mv;
  AttnArgs a;
  AttnShared* shared;
  float2* ml;          // [cta][2][128] maximum (log2) and sum
  float* o;            // [cta][2][128][D]
  int G, R;            // query heads per key-value head, tokens per row tile
  DevErr err;
};

// ------------------------------------------------------------- tcgen05, TMA ---
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tma_load_4d(void* dst, const void* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// kind::f16 with bf16 operands, D fp32, A K-major; B K-major or (bit 16) not.
__host__ __device__ constexpr uint32_t idesc_bf16(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((128u >> 4) << 24);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void pair_sync(int quarter) {   // the two warps of a lane quarter
  __syncwarp();
  asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
}

// --------------------------------------------------------------- the walk ---
struct Req {
  int row, n, ctx, tiles;   // first row, new tokens, context (negative: not served), row tiles
};

__device__ __forceinline__ Req req_of(const TaParams& p, int lo, int hi, int len) {
  lo = min(max(lo, 0), p.a.T);
  hi = min(max(hi, 0), p.a.T);
  Req r;
  r.row = lo;
  r.n = max(hi - lo, 0);
  len = min(len, p.a.table_width << p.a.page_shift);
  r.ctx = len >= r.n ? len - r.n : -1;
  r.tiles = (r.n + p.R - 1) / p.R;
  return r;
}

__device__ __forceinline__ int keys_of(const TaParams& p, const Req& r, int t) {
  return r.ctx < 0 ? 0 : r.ctx + min(r.n, (t + 1) * p.R);
}
// cost of a request's first t row tiles under one head (all but the last are full)
__device__ __forceinline__ long long cost_before(const TaParams& p, const Req& r, int t) {
  long long c = (long long)t * (kItemCost + max(r.ctx, 0));
  if (r.ctx >= 0) c += (long long)p.R * t * (t + 1) / 2;
  return c;
}
__device__ __forceinline__ long long cost_of(const TaParams& p, const Req& r) {
  if (r.n == 0) return 0;
  return cost_before(p, r, r.tiles - 1) + kItemCost + keys_of(p, r, r.tiles - 1);
}

struct Start {
  long long at, share;   // cost before the CTA's first row tile; a CTA's cost
  int b, h, t;
};

// A CTA's part of a row tile: key tiles [k0, k1) of nk.
struct Seg {
  int b, h, row, tok0, tokens, ctx, keys, k0, k1, nk;
  long long at;    // the row tile's cost begins here
};

// All roles walk the same parts.
struct Walk {
  const TaParams& p;
  long long c0, c1, at;
  int b, h, t;
  Req r;
  int next_hi, next_len;

  __device__ __forceinline__ void load() {
    r = req_of(p, __ldg(p.a.offsets + b), __ldg(p.a.offsets + b + 1), __ldg(p.a.length + b));
  }
  __device__ __forceinline__ Walk(const TaParams& p_, const Start& s)
      : p(p_), c0((long long)blockIdx.x * s.share), c1(c0 + s.share), at(s.at), b(s.b), h(s.h), t(s.t) {
    if (b < p.a.requests) load();
  }
  // The next part of the CTA that has work (key tiles, or a row tile without
  // keys that begins here); false at the end.
  __device__ __forceinline__ bool next(Seg& s) {
    while (b < p.a.requests && at < c1) {
      const int keys = keys_of(p, r, t), nk = (keys + 127) >> 7;
      const long long cost = kItemCost + keys;
      s.b = b;
      s.h = h;
      s.row = r.row;
      s.tok0 = t * p.R;
      s.tokens = min(p.R, r.n - s.tok0);
      s.ctx = r.ctx;
      s.keys = keys;
      s.nk = nk;
      s.at = at;
      s.k0 = border(c0 - at, cost, nk);
      s.k1 = border(c1 - at, cost, nk);
      const bool begins = at >= c0;
      at += cost;
      if (++t == r.tiles) {
        t = 0;
        if (++h == p.a.kv_heads) {
          h = 0;
          do {
            if (++b >= p.a.requests) break;
            load();
          } while (r.n == 0);
        }
      }
      if (s.k0 < s.k1 || (nk == 0 && begins) || (begins && s.at + cost > c1)) return true;
    }
    return false;
  }
  // Key tile at which a cost x into a row tile falls.
  static __device__ __forceinline__ int border(long long x, long long cost, int nk) {
    if (x >= cost) return nk;
    const long long k = (x - kItemCost + 64) >> 7;
    return (int)(k < 0 ? 0 : k > nk ? nk : k);
  }
};

// Equal costs per CTA, at least what one key tile costs (a smaller part would
// have none), and where this CTA begins.
template <int kThreads>
__device__ __forceinline__ void find_start(const TaParams& p, Start* out, long long (&part)[kThreads / 32],
                                           bool flag_lengths) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.a.requests;
  const int per = (B + kThreads - 1) / kThreads, b0 = tid * per;
  long long mine = 0;
  for (int i = 0; i < per && b0 + i < B; ++i) {
    const int b = b0 + i, len = p.a.length[b];
    const Req r = req_of(p, p.a.offsets[b], p.a.offsets[b + 1], len);
    mine += p.a.kv_heads * cost_of(p, r);
    if (flag_lengths && r.n && len > (p.a.table_width << p.a.page_shift)) atomicOr(p.err.word, DEVERR_RANGE);
  }
  long long s = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  if (lane == 31) part[warp] = s;
  if (tid == 0) out->b = B;
  __syncthreads();
  long long before = s - mine, total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += part[i];
    total += part[i];
  }
  const long long share = max((total + gridDim.x - 1) / gridDim.x, (long long)(kItemCost + 128));
  const long long c0 = blockIdx.x * share;
  if (tid == 0) out->share = share;
  if (c0 >= before && c0 < before + mine) {
    for (int b = b0;; ++b) {
      const Req r = req_of(p, p.a.offsets[b], p.a.offsets[b + 1], p.a.length[b]);
      const long long head = cost_of(p, r);
      if (c0 < before + p.a.kv_heads * head) {
        const int h = (int)((c0 - before) / head);
        const long long x = c0 - before - h * head;
        int lo = 0, hi = r.tiles;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (cost_before(p, r, mid) <= x) lo = mid; else hi = mid;
        }
        out->at = before + h * head + cost_before(p, r, lo);
        out->b = b;
        out->h = h;
        out->t = lo;
        break;
      }
      before += p.a.kv_heads * head;
    }
  }
}

// Place in the operand ring, from a part's first chunk on, of the values of its
// key tile i of n. Scores run one tile ahead: K0 K1 V0 K2 V1 .. K(n-1) V(n-2) V(n-1).
__device__ __forceinline__ uint32_t value_chunk(int i, int n, int nc) {
  return nc * (i + 1 < n ? 2 * i + 2 : 2 * n - 1);
}

// Bits of the keys that a row sees among the 64 from node index `a` (key minus
// context) on; token i of its request, words of its mask or NULL.
__device__ __forceinline__ unsigned long long low_bits(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}
__device__ __forceinline__ unsigned long long seen_bits(int a, int i, const unsigned long long* words,
                                                        int nwords) {
  unsigned long long v = low_bits(i + 1 - a);
  if (words && a + 63 >= 0) {
    const int from = max(a, 0), w = from >> 6, sh = from & 63;
    unsigned long long m = w < nwords ? __ldg(words + w) >> sh : 0;
    if (sh && w + 1 < nwords) m |= __ldg(words + w + 1) << (64 - sh);
    v &= a < 0 ? (m << -a) | low_bits(-a) : m;
  }
  return v;
}

// Sets the elements of 8 bf16 that are no finite numbers to zero; true if any.
__device__ __forceinline__ bool clear_unbounded(uint4& x) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&x);
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool lo = (w[i] & 0x7f80u) == 0x7f80u, hi = (w[i] & 0x7f800000u) == 0x7f800000u;
    if (lo) w[i] &= 0xffff0000u;
    if (hi) w[i] &= 0x0000ffffu;
    any |= lo || hi;
  }
  return any;
}

template <bool E>
__device__ __forceinline__ float cache_value(const void* base, long long i) {
  if constexpr (E) {
    const uint16_t c = static_cast<const uint8_t*>(base)[i];
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return f16_lo(h);
  } else {
    return bf16_to_f32(static_cast<const uint16_t*>(base)[i]);
  }
}

// Two e4m3 (low half) as bf16x2, exactly; a NaN stays one.
__device__ __forceinline__ uint32_t e4m3x2_bf16x2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return pack_bf16x2(f16_lo(h), f16_hi(h));
}

// ----------------------------------------------------------------- kernel ---
template <int D, bool E>
__global__ void __launch_bounds__(Shape<D, E>::kThreads, 1) tree_attn_kernel(const __grid_constant__ TaParams p) {
  using Sh = Shape<D, E>;
  constexpr int NC = Sh::NC, kSlots = Sh::kSlots, kRaw = Sh::kRaw;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sq = smem;
  uint8_t* slots = sq + NC * kSlotBytes;
  uint8_t* raws = slots + kSlots * kSlotBytes;
  uint8_t* misc = raws + kRaw * kRawBytes;
  float* s_max = reinterpret_cast<float*>(misc);                   // [2][2][128]
  uint64_t* full = reinterpret_cast<uint64_t*>(misc + 2048);
  uint64_t* empty = full + kSlots;
  uint64_t* raw_full = empty + kSlots;
  uint64_t* raw_empty = raw_full + kRaw;
  uint64_t* q_full = raw_empty + kRaw;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;      // [2]
  uint64_t* p_full = s_full + 2;       // [2]
  uint64_t* pv_done = p_full + 2;
  uint64_t* o_full = pv_done + 1;
  uint64_t* o_free = o_full + 1;
  uint64_t* drain = o_free + 1;
  Start* start = reinterpret_cast<Start*>(drain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(start + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* s_unbounded = abort_flag + 1;
  long long(*part)[Sh::kThreads / 32] = reinterpret_cast<long long(*)[Sh::kThreads / 32]>(misc + 2048 + 1024);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], E ? kConvWarps : 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], kConvWarps);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kSoftWarps);
    }
    mbar_init(pv_done, 1);
    mbar_init(o_full, 1);
    mbar_init(o_free, kSoftWarps);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *s_unbounded = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.mq);
    tma_prefetch_desc(&p.mk);
    tma_prefetch_desc(&p.mv);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  pdl_begin();
  find_start<Sh::kThreads>(p, start, *part, blockIdx.x == 0);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // waits of a whole warp; after a wait that failed all others return at once
  auto wait = [&](uint64_t* bar, uint32_t parity, int site) {
    bool ok = mbar_try_wait(bar, parity) ||
              (!*abort_flag && mbar_wait(bar, parity, abort_flag, p.err.limit_ns));
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
      if (lane == 0 && !*abort_flag) report_timeout(p.err, site);
      *abort_flag = 1;
    }
    return ok;
  };

  Walk walk(p, *start);
  Seg s;
  if (warp == kLoadWarp) {
    // ---------------------------------------------------- loads, by TMA
    constexpr int kRing = E ? kRaw : kSlots, kBytes = E ? kRawBytes : kSlotBytes, kRow = E ? 64 : 128;
    uint8_t* ring = E ? raws : slots;
    uint64_t *rf = E ? raw_full : full, *re = E ? raw_empty : empty;
    const int page = 1 << p.a.page_shift, box = min(page, 128), nbox = 128 / box;
    uint32_t cnt = 0, segs = 0;
    bool ok = true, bad = false;
    while (ok && walk.next(s)) {
      if (s.k0 >= s.k1) continue;
      if (!(ok = wait(q_empty, (segs & 1) ^ 1, 1))) break;
      if (elect_one_sync()) {
        mbar_arrive_expect_tx(q_full, NC * 128 * p.G * p.R);
        for (int c = 0; c < NC; ++c)
          tma_load_3d(sq + c * kSlotBytes, &p.mq, 64 * c, s.h * p.G, s.row + s.tok0, q_full);
      }
      __syncwarp();
      ++segs;
      const int len_pages = (s.keys + page - 1) >> p.a.page_shift;
      const int32_t* table = p.a.table + (long long)s.b * p.a.table_width;
      // this lane's box of key tile k: its page, or one past the cache (zeros)
      auto page_of = [&](int k) {
        const int i = (128 * k + lane * box) >> p.a.page_shift;
        if (lane >= nbox || k >= s.k1 || i >= len_pages) return p.a.cache.pages;
        const int id = __ldg(table + i);
        if (id >= 0 && id < p.a.cache.pages) return id;
        bad = true;
        return p.a.cache.pages;
      };
      auto load = [&](const CUtensorMap* m, int k, int id) {
        for (int c = 0; c < NC && ok; ++c, ++cnt) {
          const int i = cnt % kRing;
          if (!(ok = wait(&re[i], ((cnt / kRing) & 1) ^ 1, 2))) break;
          if (lane == 0) mbar_arrive_expect_tx(&rf[i], kBytes);
          __syncwarp();
          if (lane < nbox)
            tma_load_4d(ring + i * kBytes + lane * box * kRow, m, 64 * c, (128 * k + lane * box) & (page - 1),
                        s.h, id, &rf[i]);
        }
      };
      int id = page_of(s.k0), ahead = page_of(s.k0 + 1);
      load(&p.mk, s.k0, id);
      for (int k = s.k0; k < s.k1 && ok; ++k) {
        const int later = page_of(k + 2);
        if (k + 1 < s.k1) load(&p.mk, k + 1, ahead);
        if (ok) load(&p.mv, k, id);
        id = ahead;
        ahead = later;
      }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.err.word, DEVERR_RANGE);
    if (!ok) {   // own copies land before shared memory is released
      for (int i = 0; i < kRing; ++i) {
        const uint32_t uses = (cnt + kRing - 1 - i) / kRing;
        if (uses) mbar_wait_drain(&rf[i], (uses - 1) & 1, p.err.limit_ns);
      }
      if (segs) mbar_wait_drain(q_full, (segs - 1) & 1, p.err.limit_ns);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------- products
    uint32_t cnt = 0, segs = 0, tiles = 0;
    bool ok = true;
    constexpr uint32_t kIdS = idesc_bf16(128, false), kIdO = idesc_bf16(64, true);
    const uint32_t q_addr = smem_u32(sq), slot_addr = smem_u32(slots);
    auto scores = [&](uint32_t n) {   // S[n & 1] = Q K^T
      for (int c = 0; c < NC && ok; ++c, ++cnt) {
        const int i = cnt % kSlots;
        if (!(ok = wait(&full[i], (cnt / kSlots) & 1, 3))) break;
        tc_fence_after();
        if (elect_one_sync()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16_ss(tmem + kColS + 128 * (n & 1), smem_desc_sw128(q_addr + c * kSlotBytes + 32 * kk),
                       smem_desc_sw128(slot_addr + i * kSlotBytes + 32 * kk), kIdS, (c | kk) != 0);
          mma_commit(&empty[i]);
          if (c == NC - 1) mma_commit(&s_full[n & 1]);
        }
        __syncwarp();
      }
    };
    while (ok && walk.next(s)) {
      const int n = s.k1 - s.k0;
      if (n <= 0) continue;
      if (!(ok = wait(q_full, segs & 1, 4))) break;
      tc_fence_after();
      scores(tiles);
      for (int t = 0; t < n && ok; ++t, ++tiles) {
        if (t + 1 < n) scores(tiles + 1);
        if (!ok) break;
        if (t == max(n - 2, 0)) {   // Q is free once the last scores' products are done
          if (elect_one_sync()) mma_commit(q_empty);
          __syncwarp();
        }
        if (!(ok = wait(&p_full[tiles & 1], (tiles >> 1) & 1, 5))) break;
        if (t == 0 && !(ok = wait(o_free, (segs & 1) ^ 1, 6))) break;
        tc_fence_after();
        const uint32_t pc = tmem + kColS + 128 * (tiles & 1);
        for (int c = 0; c < NC && ok; ++c, ++cnt) {
          const int i = cnt % kSlots;
          if (!(ok = wait(&full[i], (cnt / kSlots) & 1, 7))) break;
          tc_fence_after();
          if (elect_one_sync()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)   // 16 keys each; weights of keys 64.. lie 64 columns on
              mma_f16_ts(tmem + 64 * c, pc + 8 * (kk & 3) + 64 * (kk >> 2),
                         smem_desc_sw128(slot_addr + i * kSlotBytes + 2048 * kk), kIdO, (t | kk) != 0);
            mma_commit(&empty[i]);
            if (c == NC - 1) mma_commit(t + 1 < n ? pv_done : o_full);
          }
          __syncwarp();
        }
      }
      ++segs;
    }
    if (elect_one_sync()) mma_commit(drain);
    __syncwarp();
    mbar_wait_drain(drain, 0, p.err.limit_ns);
  } else if (E && warp >= kConvWarp) {
    // --------------------------------------------- e4m3 chunks to bf16
    const int w = warp - kConvWarp;
    uint32_t cnt = 0;
    bool ok = true;
    while (ok && walk.next(s)) {
      const int chunks = 2 * NC * max(s.k1 - s.k0, 0);
      for (int c = 0; c < chunks && ok; ++c, ++cnt) {
        const int ri = cnt % max(kRaw, 1), si = cnt % kSlots;
        if (!(ok = wait(&raw_full[ri], (cnt / max(kRaw, 1)) & 1, 8))) break;
        const uint8_t* src = raws + ri * kRawBytes;
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint4*>(src + 16 * (32 * (4 * w + i) + lane));
        if (!(ok = wait(&empty[si], ((cnt / kSlots) & 1) ^ 1, 9))) break;
        uint8_t* dst = slots + si * kSlotBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int id = 32 * (4 * w + i) + lane, row = id >> 2, piece = 2 * (id & 3);
          const uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o[2 * j] = e4m3x2_bf16x2((uint16_t)v[j]);
            o[2 * j + 1] = e4m3x2_bf16x2((uint16_t)(v[j] >> 16));
          }
          *reinterpret_cast<uint4*>(dst + 128 * row + 16 * (piece ^ (row & 7))) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(dst + 128 * row + 16 * ((piece + 1) ^ (row & 7))) =
              make_uint4(o[4], o[5], o[6], o[7]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[si]);
          mbar_arrive(&raw_empty[ri]);
        }
      }
    }
  } else {
    // ------------------------------------------------- softmax, output
    // After a failed wait these warps run through, so that the barriers they
    // share complete, and store nothing.
    const int half = warp >> 2, quarter = warp & 3, row = 32 * quarter + lane;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    // operand chunks, parts and key tiles before this part; products that pv_done counts
    uint32_t base = 0, segs = 0, tiles = 0, pvs = 0;
    AttnShared mine = {};
    while (walk.next(s)) {
      const int n = s.k1 - s.k0, rows = s.tokens * p.G;
      const bool live = row < rows, work = 32 * quarter < rows;
      const int tok = s.tok0 + row / p.G, head = s.h * p.G + row % p.G;
      uint16_t* out = p.a.out + (long long)(s.row + tok) * p.a.o_ld + (long long)head * D + half * (D / 2);
      const long long cost = kItemCost + s.keys, c0 = walk.c0, share = walk.c1 - walk.c0;
      if (s.at >= c0 && s.at + cost > c0 + share) {
        // this CTA begins a row tile that others go on with: which hold a part
        int first = blockIdx.x, last = (int)((s.at + cost - 1) / share);
        if (s.k1 == 0) ++first;
        if (Walk::border(last * share - s.at, cost, s.nk) == s.nk) --last;
        if (s.nk && last > first) {
          mine.row = s.row + s.tok0;
          mine.tokens = s.tokens;
          mine.head = s.h;
          mine.first = first;
          mine.count = last - first + 1;
        }
      }
      if (s.nk == 0) {   // no keys: zeros
        if (live && s.at >= c0 && !*abort_flag)
          for (int i = 0; i < D / 2; i += 8) *reinterpret_cast<uint4*>(out + i) = make_uint4(0, 0, 0, 0);
        continue;
      }
      if (n <= 0) continue;
      ++segs;
      const float ks = E ? p.a.cache.k_scale[s.h] : 1.0f;
      const float c2 = p.a.scale * ks * 1.4426950408889634f;   // scores in log2
      const unsigned long long* words = p.a.mask ? p.a.mask + (long long)(s.row + tok) * p.a.mask_words : nullptr;
      // keys before `seen` are seen by every row of the tile
      const int seen = p.a.mask ? s.ctx : s.ctx + s.tok0 + 1;
      float m = -INFINITY, l = 0.0f;
      for (int t = 0; t < n; ++t, ++tiles) {
        const int k = s.k0 + t, buf = tiles & 1;
        const bool masked = 128 * (k + 1) > seen;
        const uint32_t sc = tmem + lanes + kColS + 128 * buf + 64 * half;
        unsigned long long vis = ~0ull;
        if (masked) vis = live ? seen_bits(128 * k + 64 * half - s.ctx, tok, words, p.a.mask_words) : 0;
        wait(&s_full[buf], (tiles >> 1) & 1, 10);
        tc_fence_after();
        if (work) {
          uint32_t x[2][32];
          tmem_ld_32x32b_x32(sc, x[0]);
          tmem_ld_32x32b_x32(sc + 32, x[1]);
          tmem_wait_ld();
          if (masked) {
#pragma unroll
            for (int i = 0; i < 64; ++i) {
              const uint32_t w = (uint32_t)(vis >> (i & 32));
              if (!(w >> (i & 31) & 1)) x[i >> 5][i & 31] = 0xff800000u;
            }
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 64; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(x[i >> 5][i & 31]));
          float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          s_max[256 * buf + 128 * half + row] = top;
          pair_sync(quarter);
          top = fmaxf(top, s_max[256 * buf + 128 * (half ^ 1) + row]) * c2;
          // (NaN scores are left out of the maximum and make the sum NaN)
          const bool grow = top > m + kGrowth || m == -INFINITY;
          const float old = m;
          if (grow && top > m) m = top;
          if (t > 0 && __any_sync(0xffffffffu, grow && old != -INFINITY)) {
            // (the scores of this tile follow the product of the last but one: of pv_done's phases
            // only the last product's can be open)
            wait(pv_done, (pvs - 1) & 1, 11);
            tc_fence_after();
            const float f = grow && old != -INFINITY ? ex2(old - m) : 1.0f;
            l *= f;
#pragma unroll
            for (int i = 0; i < D / 2; i += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(tmem + lanes + half * (D / 2) + i, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st_32x32b_x32(tmem + lanes + half * (D / 2) + i, o);
            }
          }
          const float ref = m == -INFINITY ? 0.0f : m;
          float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float a = ex2(fmaf(__uint_as_float(x[i >> 4][2 * i & 31]), c2, -ref));
            const float b = ex2(fmaf(__uint_as_float(x[i >> 4][(2 * i & 31) + 1]), c2, -ref));
            sum[2 * i & 3] += a;
            sum[(2 * i & 3) + 1] += b;
            w[i] = pack_bf16x2(a, b);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_st_32x32b_x32(sc, w);
          tmem_wait_st();
        }
        if (masked) {
          // values that some row must not see: keys past the row tile's own are
          // nobody's, others only where they are no numbers
          const int key = threadIdx.x & 127, j = 128 * k + key;
          const uint32_t at = base + value_chunk(t, n, NC);
          bool any = false;
          for (int c = 0; c < NC; ++c) {
            const uint32_t i = (at + c) % kSlots;
            wait(&full[i], ((at + c) / kSlots) & 1, 12);
            if (j < seen) continue;
            uint4* v = reinterpret_cast<uint4*>(slots + i * kSlotBytes + 128 * key);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint4* piece = v + ((4 * half + q) ^ (key & 7));
              uint4 y = j < s.keys ? *piece : make_uint4(0, 0, 0, 0);
              const bool un = clear_unbounded(y);
              if (un || j >= s.keys) *piece = y;
              any |= un;
            }
          }
          if (any) *s_unbounded = (int)segs;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
        if (t + 1 < n) ++pvs;   // tile t's product
      }
      base += 2 * n * NC;
      // the part's sums
      wait(o_full, (segs - 1) & 1, 13);
      tc_fence_after();
      if (work) {
        s_max[128 * half + row] = l;
        pair_sync(quarter);
        l += s_max[128 * (half ^ 1) + row];
        pair_sync(quarter);   // read before the next part's maxima
        const bool whole = s.k0 == 0 && s.k1 == s.nk;
        const float inv = whole ? (l == 0.0f ? 0.0f : (E ? p.a.cache.v_scale[s.h] : 1.0f) / l) : 1.0f;
        const int place = 2 * blockIdx.x + (s.k0 == 0 && s.at >= c0 ? 1 : 0);
        const bool fix = *s_unbounded == (int)segs;
#pragma unroll 1
        for (int i = 0; i < D / 2; i += 32) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld_32x32b_x32(tmem + lanes + half * (D / 2) + i, o);
          tmem_wait_ld();
          if (!live || *abort_flag) continue;
          if (fix) {
            const int end = min(s.keys, 128 * s.k1);
            for (int j = max(seen, 128 * s.k0); j < end; ++j) {
              if (!(seen_bits(j - s.ctx, tok, words, p.a.mask_words) & 1)) continue;
              const int id = p.a.table[(long long)s.b * p.a.table_width + (j >> p.a.page_shift)];
              if (id < 0 || id >= p.a.cache.pages) continue;
              const long long e = ((((long long)id * p.a.kv_heads + s.h) << p.a.page_shift) +
                                   (j & ((1 << p.a.page_shift) - 1))) * D + half * (D / 2) + i;
#pragma unroll
              for (int q = 0; q < 32; ++q) {
                const float v = cache_value<E>(p.a.cache.v, e + q);
                if (!(fabsf(v) < INFINITY)) o[q] = __float_as_uint(__uint_as_float(o[q]) + v);
              }
            }
          }
          if (whole) {
#pragma unroll
            for (int q = 0; q < 32; q += 8) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = pack_bf16x2(__uint_as_float(o[q + 2 * j]) * inv, __uint_as_float(o[q + 2 * j + 1]) * inv);
              *reinterpret_cast<uint4*>(out + i + q) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            uint4* dst = reinterpret_cast<uint4*>(p.o + ((long long)place * 128 + row) * D + half * (D / 2) + i);
#pragma unroll
            for (int q = 0; q < 8; ++q) dst[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          }
        }
        if (!whole && half == 0 && live) p.ml[place * 128 + row] = make_float2(m == -INFINITY ? 0.0f : m, l);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
    }
    if (threadIdx.x == 0) {
      if (*abort_flag) mine.count = 0;
      p.shared[blockIdx.x] = mine;
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of the row tiles that CTAs share: block (c, i) takes the rows
// i, i + gridDim.y, .. of the tile that CTA c began. Its warps take alternate
// parts, then add up through shared memory.
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) tree_attn_join(const TaParams p) {
  pdl_begin();
  const AttnShared s = p.shared[blockIdx.x];
  constexpr int V = D / 32;
  __shared__ float s_o[kJoinWarps][D];
  __shared__ float2 s_ml[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (the CTA that began the tile holds its part in its second place)
  auto place = [&](int i) { return 2 * (s.first + i) + (s.first + i == (int)blockIdx.x ? 1 : 0); };
  for (int row = blockIdx.y; s.count && row < s.tokens * p.G; row += gridDim.y) {
    float o[V] = {}, m = -INFINITY, l = 0.0f;
    for (int i0 = warp; i0 < s.count; i0 += 4 * kJoinWarps) {
      float x[4][V];
      float2 ml[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * kJoinWarps;
        ml[u] = make_float2(0.0f, 0.0f);
        if (i < s.count) {
          const long long at = (long long)place(i) * 128 + row;
          ml[u] = p.ml[at];
#pragma unroll
          for (int v = 0; v < V; ++v) x[u][v] = p.o[at * D + lane + 32 * v];
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (ml[u].y == 0.0f) continue;
        const float mn = fmaxf(m, ml[u].x), f = ex2(m - mn), g = ex2(ml[u].x - mn);
        m = mn;
        l = l * f + ml[u].y * g;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = o[v] * f + x[u][v] * g;
      }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) s_o[warp][lane + 32 * v] = o[v];
    if (lane == 0) s_ml[warp] = make_float2(m, l);
    __syncthreads();
    float M = -INFINITY, L = 0.0f, f[kJoinWarps];
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, s_ml[w].x);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      f[w] = s_ml[w].y == 0.0f ? 0.0f : ex2(s_ml[w].x - M);
      L += s_ml[w].y * f[w];
    }
    const float scale = L == 0.0f ? 0.0f : (p.a.e4m3 ? p.a.cache.v_scale[s.head] : 1.0f) / L;
    for (int d = threadIdx.x; d < D; d += 32 * kJoinWarps) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) sum += s_ml[w].y == 0.0f ? 0.0f : s_o[w][d] * f[w];
      p.a.out[(long long)(s.row + row / p.G) * p.a.o_ld + (long long)(s.head * p.G + row % p.G) * D + d] =
          f32_to_bf16(sum * scale);
    }
  }
}

bool encode_maps(const AttnArgs& a, int G, int R, TaParams* p) {
  const uint64_t D = a.head_dim, P = 1ull << a.page_shift, e = a.e4m3 ? 1 : 2;
  const uint64_t qd[3] = {D, (uint64_t)a.heads, (uint64_t)a.T}, qs[2] = {2 * D, 2 * (uint64_t)a.q_ld};
  const uint32_t qb[3] = {64, (uint32_t)G, (uint32_t)R};
  const uint64_t cd[4] = {D, P, (uint64_t)a.kv_heads, (uint64_t)a.cache.pages};
  const uint64_t cs[3] = {D * e, D * e * P, D * e * P * a.kv_heads};
  const uint32_t cb[4] = {64, (uint32_t)(P < 128 ? P : 128), 1, 1};
  const auto dt = a.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return encode_nd(&p->mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.q, qd, qs, qb, true) &&
         encode_nd(&p->mk, dt, 4, a.cache.k, cd, cs, cb, !a.e4m3) &&
         encode_nd(&p->mv, dt, 4, a.cache.v, cd, cs, cb, !a.e4m3);
}

template <int D, bool E>
cudaError_t launch(const TaParams& p, int num_sms, cudaStream_t st) {
  using Sh = Shape<D, E>;
  auto kern = tree_attn_kernel<D, E>;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), Sh::kSmem);
  const int ctas = num_sms < kAttnMaxCtas ? num_sms : kAttnMaxCtas;
  if (e == cudaSuccess) e = launch_pdl(kern, dim3(ctas), dim3(Sh::kThreads), Sh::kSmem, st, p);
  if (e == cudaSuccess) e = launch_pdl(tree_attn_join<D>, dim3(ctas, 16), dim3(32 * kJoinWarps), 0, st, p);
  return e;
}

}  // namespace

cudaError_t launch_tree_attention(const AttnArgs& a, void* scratch, int num_sms, DevErr err,
                                  cudaStream_t st) {
  TaParams p;
  p.a = a;
  p.G = a.heads / a.kv_heads;
  p.R = 128 / p.G;
  p.err = err;
  p.shared = static_cast<AttnShared*>(scratch);
  p.o = reinterpret_cast<float*>(p.shared + kAttnMaxCtas);
  p.ml = reinterpret_cast<float2*>(p.o + (size_t)kAttnMaxCtas * 2 * 128 * a.head_dim);
  if (!encode_maps(a, p.G, p.R, &p)) return cudaErrorInvalidValue;
  switch (a.head_dim) {
    case 64: return a.e4m3 ? launch<64, true>(p, num_sms, st) : launch<64, false>(p, num_sms, st);
    case 128: return a.e4m3 ? launch<128, true>(p, num_sms, st) : launch<128, false>(p, num_sms, st);
    default: return a.e4m3 ? launch<256, true>(p, num_sms, st) : launch<256, false>(p, num_sms, st);
  }
}

}  // namespace moe
