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
//   * One persistent CTA per SM, its warps in roles: one plans the CTA's parts and
//     loads their queries, one loads keys and values by TMA (a box per page), one
//     issues S = Q K^T, one O += P V, and groups of 4 warps do the softmax, a row
//     per thread, the groups taking key tiles in turn. Scores lie in tensor memory,
//     2 or 3 tiles of them; a tile's weights go back into its scores' place, as the
//     product's A operand. The values are its B operand as stored (their keys are
//     the product's K: the other major order).
//   * The running maximum goes from group to group through shared memory. O in
//     tensor memory is scaled only when a row's maximum has grown by 2^8: weights
//     stay below 2^8, far from overflow, and the sums are as exact.
//   * An e4m3 cache: the codes of the keys are the product's operand as they lie in
//     the cache, times queries in two e4m3 terms. Four more warps make these, and
//     turn values to fp16 (exact; the weights are then fp16 as well). Converting
//     the keys too took 55 us where this took 45 (2 contexts of 131072 tokens, trees
//     of 8), and 157 where it took 117 (76 contexts of 16000, one token each).
//   * A split of the keys gives every CTA the same work: all row tiles side by
//     side, each as long as its keys and kItemCost, are cut into equal lengths, one
//     per CTA, at key tiles' borders. A row tile that several CTAs share leaves its
//     parts' sums in scratch, in FP32, and a second kernel joins them.
//   * Rows differ in the keys that they see only from the first new token on;
//     tiles past it are masked. What is not seen may be infinite or NaN: scores
//     are replaced, and values that some row must not see are set to zero in
//     shared memory (their NaN times weight 0 would be NaN) and, in rows that do
//     see them, added at the end.
//
// Measured (in a graph; 16 query heads, 2 key-value heads, pages of 64, one GB300):
// one token of each of 76 contexts of 16000, bf16: head_dim 64 98 us, 128 182, 256 348
// (6.3, 6.9, 7.2 TB/s: memory); e4m3 92, 110, 222 (3.4, 5.7, 5.6 TB/s: a tile's way
// through the roles, 1,400 cycles at 64 to 3,000 at 256, of which its bytes need 700 to
// 2,800). 76 are a row tile per SM, so that nothing is split; 60, 100 and 200 contexts at
// head_dim 128: bf16 153, 248, 476 us (6.4, 6.6, 6.9 TB/s), e4m3 102, 163, 317 (4.8, 5.0,
// 5.2). 2 prompts of 2000 tokens behind 4096 at head_dim 64, 128, 256: bf16 103, 129, 230
// us (0.81, 1.29, 1.45 PFLOP/s), e4m3 113, 141, 261 (every row tile turns its values to
// fp16 anew). There a key tile takes 1,500 cycles at head_dim 128 in bf16, its products
// 1,024: its chain of 4,400 (S 950, softmax 2,400, P V 1,050) runs in 3 tiles at a
// time, which is all that tensor memory has place for; and 5,000 more go where a
// row tile ends (masked tile, sums read and stored). One token of one context of
// 120, 2000 and 32000: 8.3, 10.9, 18.1 us: two launches, planning 2, a page's
// number and loads 1.5, the chain 2.5, sums out 1, join 2.
#include <limits.h>

#include "attn.h"
#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kSlotBytes = 128 * 128;       // 128 rows of 64 16-bit elements
// Warps: groups of 4 for the softmax; then one that plans, one for products with keys, one
// that loads, one for products with values; for e4m3 four that convert. One warp for both
// kinds of product would bound the kernel: its waits, issue and commits take longer than the
// products. The planner has little to do and shares its scheduler with the softmax of rows
// 0..31, often the only ones.
constexpr int kPlan = 0, kScore = 1, kLoad = 2, kSum = 3, kConv = 4, kConvWarps = 4;
// Cost of a row tile beside its keys, in keys, for equal shares. Measured with 192, 256, 320, 384
// and 512: 64 tokens behind 1 to 16384 (head_dim 128) 28.4, 28.3, 28.4, 28.3, 28.7 us, 300 behind 1
// to 1500 38.6, 37.3, 37.6, 38.7, 39.9, 32 trees of 16 behind 1 to 8192 (head_dim 256) 29.8, 28.6,
// 28.2, 27.9, 28.0, 7 trees of 61 (head_dim 64, e4m3) 17.3, 17.0, 16.2, 16.8, 16.5.
constexpr int kItemCost = 320;
constexpr uint32_t kTmemCols = 512;
constexpr float kGrowth = 8.0f;             // log2 by which a maximum may be exceeded
constexpr int kParts = 4;                    // parts told ahead

// E: an e4m3 cache. Keys and values of a key tile come in blocks of up to 128
// columns, each kind with its own ring of them.
template <int D, bool E>
struct Shape {
  static constexpr int NC = D / 64;                  // chunks of 64 columns
  static constexpr int GC = NC < 2 ? NC : 2;         // chunks of a block
  static constexpr int NG = NC / GC;                 // blocks of a tile
  static constexpr int KS = D == 64 ? 4 : E ? (D == 128 ? 4 : 3) : 2;   // blocks of keys held
  static constexpr int VS = D == 64 ? 4 : 2;         // and of values
  static constexpr int VR = E ? (D == 64 ? 4 : D == 128 ? 3 : 2) : 0;   // 8-bit blocks of values
  static constexpr int QB = E || D == 256 ? 1 : 2;   // parts whose queries are held
  static constexpr int SB = D == 256 ? 2 : 3;        // key tiles whose scores or weights are held
  static constexpr int OB = D == 64 ? 2 : 1;         // parts whose sums are held
  static constexpr int kColS = 512 - 128 * SB;       // tensor memory: sums, then scores
  // groups of softmax warps, which take key tiles in turn: as many as there are places for
  // scores, or as the registers of a CTA allow beside the warps that convert
  static constexpr int SG = E ? 2 : SB;
  static constexpr int kSoftWarps = 4 * SG, kThreads = 32 * (kSoftWarps + kConv + (E ? kConvWarps : 0));
  static constexpr int kKeyRow = E ? 64 * GC : 128;  // bytes of a block's row (bf16: of each chunk's)
  static constexpr int kVBlock = GC * kSlotBytes, kRawBlock = 128 * 64 * GC, kKBlock = E ? kRawBlock : kVBlock;
  static constexpr int kQBytes = NC * kSlotBytes;
  // 8-bit queries, two terms of kRawBlock per 128 columns, lie where the 16-bit ones
  // were, or behind them where rows of 64 columns would overlap
  static constexpr int kQ8 = E && D == 64 ? kSlotBytes : 0;
  static constexpr int kMisc = 2560 + 1024 * SG + 1024 * kParts * (SG - 1) + (E ? kParts * 512 : 0);
  static constexpr int kSmem = 1024 + kMisc + QB * kQBytes + kQ8 + KS * kKBlock + VS * kVBlock + VR * kRawBlock;
  static_assert(OB * D <= kColS, "tensor memory");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct TaParams {
  CUtensorMap mq, mk, mv;
  AttnArgs a;
  unsigned long long* shared;    // [cta] the tile that it begins and shares, packed
  float2* ml;          // [cta][2][128] maximum (log2) and sum
  float* o;            // [cta][2][D][128]: a warp stores a column of its 32 rows at a time
  unsigned long long inv_ctas;   // 2^64 / CTAs, rounded up
  int G, R;            // query heads per key-value head, tokens per row tile
  unsigned inv_r;      // 2^31 / R, rounded up
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

__device__ __forceinline__ void mma_f8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tma_load_q(uint32_t dst, const void* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_load_kv(uint32_t dst, const void* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// kind::f16, D fp32, A K-major; operands bf16 or fp16, B K-major or (mn) not.
__host__ __device__ constexpr uint32_t idesc_16(bool bf16, int n, bool mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((mn ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// kind::f8f6f4 with e4m3 operands, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
// An operand of 64-byte rows, 64-byte swizzle: 8 rows 512 bytes on.
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3fff) | 1ull << 16 | (uint64_t)(512 >> 4) << 32 | 1ull << 46 | 4ull << 61;
}

// Values as the product's B operand: 16 keys (rows of 128 bytes) of 64 columns
// per swizzle atom, 8 keys 1024 bytes on, the next 64 columns a slot on.
__device__ __forceinline__ uint64_t value_desc(uint32_t addr) {
  uint64_t d = smem_desc_sw128(addr) & ~(0x3fffull << 16);
  return d | (uint64_t)(kSlotBytes >> 4) << 16;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (a.x b + c, a.y b + c), two lanes of one instruction
__device__ __forceinline__ float2 fma2(float x, float y, float b, float c) {
  float2 r;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mov.b64 c, {%5, %5};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x), "f"(y), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}

// (with its wait)
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15}, [%16];\n tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Waits for the thread's loads from tensor memory, of which x is one: no use of
// x comes before it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&x)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]),
                 "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15]),
                 "+r"(x[16]), "+r"(x[17]), "+r"(x[18]), "+r"(x[19]), "+r"(x[20]), "+r"(x[21]), "+r"(x[22]),
                 "+r"(x[23]), "+r"(x[24]), "+r"(x[25]), "+r"(x[26]), "+r"(x[27]), "+r"(x[28]), "+r"(x[29]),
                 "+r"(x[30]), "+r"(x[31])
               :
               : "memory");
}

// --------------------------------------------------------------- the walk ---
struct Req {
  int row, n, ctx, tiles;   // first row, new tokens, context (negative: not served), row tiles
};

__device__ __forceinline__ Req req_of(const TaParams& p, int lo, int hi, int len) {
  lo = min(max(lo, 0), p.a.T);
  const int added = max(hi, lo) - lo;   // (rows past T are not here, but the length counts them)
  Req r;
  r.row = lo;
  r.n = min(added, p.a.T - lo);
  len = min(len, p.a.table_width << p.a.page_shift);
  r.ctx = len >= added ? len - added : -1;
  // (exact: the quotient's error is below (2^20 + 2^8) 2^8 / 2^31 of one)
  r.tiles = (int)((unsigned long long)(unsigned)(r.n + p.R - 1) * p.inv_r >> 31);
  return r;
}

__device__ __forceinline__ int keys_of(const TaParams& p, const Req& r, int t) {
  return r.ctx < 0 ? 0 : r.ctx + min(r.n, (t + 1) * p.R);
}
// cost of a request's first t row tiles under one head (all but the last are full), with
// `item` for each beside its keys. (Rows without keys are written by the one warp that plans.)
__device__ __forceinline__ long long cost_before(const TaParams& p, const Req& r, int t, int item) {
  if (r.ctx < 0) return (long long)t * kItemCost;
  return (long long)t * (item + r.ctx) + (long long)p.R * t * (t + 1) / 2;
}
__device__ __forceinline__ long long cost_of(const TaParams& p, const Req& r, int item) {
  if (r.ctx < 0) return (long long)r.tiles * kItemCost;
  return r.n ? cost_before(p, r, r.tiles - 1, item) + item + r.ctx + r.n : 0;
}
// By a whole warp: the largest i below n (n >= 1) with f(i) <= x, for f increasing and
// f(0) <= x; 32 places are tried at a time.
template <class F>
__device__ __forceinline__ int search(int n, long long x, F f) {
  int lo = 0;
#pragma unroll 1
  while (n > 1) {
    const int step = (n + 31) >> 5, i = (threadIdx.x & 31) * step;   // (lane 0: f(lo) <= x)
    const int k = __popc(__ballot_sync(0xffffffffu, i < n && f(lo + i) <= x)) - 1;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// A CTA's part of a row tile: key tiles [k0, k1) of nk.
struct Part {
  int b, h, row, tok0, tokens, ctx, keys, k0, k1, nk;
  int place;       // of the sums in scratch, if others hold parts of the tile
  int stop;        // the end of the CTA's parts
};

// A row tile that several CTAs share: its first token row, tokens and key-value head, and the
// CTAs that hold its parts (count 0: none). In 8 bytes, since every block of the join reads
// all of them.
struct Tile {
  int row, tokens, head, first, count;
};
__device__ __forceinline__ unsigned long long packed(const Tile& m) {
  static_assert(kAttnMaxCtas < 256, "fields of 8 bits");
  return (unsigned long long)(unsigned)m.row << 32 |
         (unsigned)(m.tokens << 24 | m.head << 16 | m.first << 8 | m.count);
}
__device__ __forceinline__ Tile unpacked(unsigned long long x) {
  const unsigned y = (unsigned)x;
  return {(int)(x >> 32), (int)(y >> 24), (int)(y >> 16 & 255), (int)(y >> 8 & 255), (int)(y & 255)};
}

// The CTA's parts, in order.
struct Walk {
  const TaParams& p;
  long long c0, c1, at, end;   // end: of the CTA's costs, or of all
  int b, h, t;
  Req r;
  int lo, hi, len;     // of request b + 1, read ahead
  int item;            // cost of a row tile beside its keys
  long long from;      // the row tile that this CTA begins and others go on with: its cost, -1 none
  Part* last;          // (in shared memory)

  __device__ __forceinline__ void ahead() {
    if (b + 1 < p.a.requests) {
      lo = __ldcg(p.a.offsets + b + 1);
      hi = __ldcg(p.a.offsets + b + 2);
      len = __ldcg(p.a.length + b + 1);
    }
  }
  __device__ __forceinline__ Req load(int i) const {
    return req_of(p, __ldcg(p.a.offsets + i), __ldcg(p.a.offsets + i + 1), __ldcg(p.a.length + i));
  }

  __device__ __forceinline__ explicit Walk(const TaParams& p_, Part* last_) : p(p_), last(last_) {}
  // By a whole warp. Equal costs per CTA, at least what one key tile costs (a
  // smaller part would have none): the costs of all requests are summed up, a
  // run of them per lane; the lane in whose run the CTA's cost begins finds the
  // request, and all lanes together the head and row tile.
  __device__ __forceinline__ void begin() {
    b = p.a.requests;
    from = -1;
    const int lane = threadIdx.x & 31, B = p.a.requests, per = (B + 31) >> 5;
    const int b0 = min(lane * per, B), b1 = min(b0 + per, B), cap = p.a.table_width << p.a.page_shift;
    long long mine = 0;
    int tiles = 0, longest = 0, first = b0;
    r = Req{};
#pragma unroll 1
    for (int i0 = b0; i0 < b1; i0 += 4) {
      // (four requests' loads at once)
      int from_row[4], to_row[4], lens[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = min(i0 + j, b1 - 1);
        from_row[j] = __ldcg(p.a.offsets + i);
        to_row[j] = __ldcg(p.a.offsets + i + 1);
        lens[j] = __ldcg(p.a.length + i);
      }
#pragma unroll 1
      for (int j = 0; j < min(b1 - i0, 4); ++j) {
        const Req q = req_of(p, from_row[0], to_row[0], lens[0]);
        if (r.n == 0 && q.n > 0) {   // the run's first that is not idle
          r = q;
          first = i0 + j;
        }
        mine += cost_of(p, q, 0);
        tiles += q.ctx < 0 ? 0 : q.tiles;
        longest = max(longest, q.n > 0 && q.ctx >= 0 ? q.ctx + q.n : 0);   // (of those with work)
        if (blockIdx.x == 0 && q.n && lens[0] > cap) atomicOr(p.err.word, DEVERR_RANGE);
#pragma unroll
        for (int x = 0; x < 3; ++x) {
          from_row[x] = from_row[x + 1];
          to_row[x] = to_row[x + 1];
          lens[x] = lens[x + 1];
        }
      }
    }
    mine *= p.a.kv_heads;
    tiles *= p.a.kv_heads;   // (below 2^29 where the requests' rows are apart)
    __syncwarp();
    long long before = mine;
    int tiles_before = tiles;
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, before, d);
      const int ot = __shfl_up_sync(0xffffffffu, tiles_before, d);
      if (lane >= d) {
        before += o;
        tiles_before += ot;
      }
    }
    long long total = __shfl_sync(0xffffffffu, before, 31);
    const int all_tiles = __shfl_sync(0xffffffffu, tiles_before, 31);
    // A share holds at least a row tile's cost and one key tile. Where that would leave SMs
    // idle the cost is taken lower: to nothing for few row tiles, whose key tiles then go
    // singly, else to a key tile, so that an SM does not begin many short ones; but the
    // longest row tile, if of up to 7,168 keys, is in 16 parts at most, which its warps join in
    // one round (a longer one bears the whole cost: 9,000 keys go in 21). Measured (head_dim
    // 128) so and with the whole cost: one token of 2000 11.1 and 11.5 us, 4 trees of 16 behind
    // 1000 13.0 and 14.2, 32 behind 1 to 2000 16.3 and 18.7; with no cost whatever the number,
    // the last 27.7; in more parts, one token of 8000 16.6 for 13.3.
    longest = __reduce_max_sync(0xffffffffu, longest);
    item = total + (long long)all_tiles * kItemCost >= (long long)gridDim.x * (kItemCost + 128)
               ? kItemCost : min(kItemCost, max(8 * all_tiles <= gridDim.x ? 1 : 128, longest / 16 - 128));
    total += (long long)all_tiles * item;
    mine += (long long)tiles * item;
    before += (long long)tiles_before * item - mine;
    // (a little more than the quotient: the shares cover the total)
    const long long share = max((long long)__umul64hi(total, p.inv_ctas) + 1, (long long)(item + 128));
    c0 = blockIdx.x * share;
    c1 = c0 + share;
    end = min(c1, total);
    const bool owner = c0 >= before && c0 < before + mine;
    const unsigned who = __ballot_sync(0xffffffffu, owner);
    if (!who) return;
    long long head = 0;
    if (owner) {
      head = cost_of(p, r, item);
      // (bounded: offsets that go back and forth can make the sums overflow)
      for (b = first; b + 1 < b1 && c0 >= before + p.a.kv_heads * head;) {
        before += p.a.kv_heads * head;
        r = load(++b);
        head = cost_of(p, r, item);
      }
    }
    __syncwarp();
    const int src = __ffs(who) - 1;
    auto all = [&](int v) { return __shfl_sync(0xffffffffu, v, src); };
    at = __shfl_sync(0xffffffffu, before, src);
    head = __shfl_sync(0xffffffffu, head, src);
    b = all(b);
    r = {all(r.row), all(r.n), all(r.ctx), all(r.tiles)};
    if (r.tiles == 0) b = p.a.requests;
    ahead();
    h = search(p.a.kv_heads, c0 - at, [&](int i) { return i * head; });
    at += h * head;
    t = search(r.tiles, c0 - at, [&](int i) { return cost_before(p, r, i, item); });
    at += cost_before(p, r, t, item);
  }
  // To the next request with new tokens, if the CTA's costs reach it; idle ones between are
  // passed over 32 at a time. (One at a time, and to the end of the batch: one token of 2000
  // before 255 idle requests took 55 us, before 4095 717; so 13 and 40, where it takes 11 alone.)
  __device__ __forceinline__ void following() {
    if (++b >= p.a.requests || at >= end) return;
    r = req_of(p, lo, hi, len);
    while (r.n == 0) {
      if (++b >= p.a.requests) return;
      const int i = min(b + (int)(threadIdx.x & 31), p.a.requests - 1);
      const Req q = load(i);
      const unsigned live = __ballot_sync(0xffffffffu, q.n > 0);
      const int src = live ? __ffs(live) - 1 : 31;
      b += src;
      r = {__shfl_sync(0xffffffffu, q.row, src), __shfl_sync(0xffffffffu, q.n, src),
           __shfl_sync(0xffffffffu, q.ctx, src), __shfl_sync(0xffffffffu, q.tiles, src)};
    }
    ahead();
  }
  // The next part that has work: key tiles, or a row tile without keys that
  // begins here.
  __device__ __forceinline__ bool next(Part& s) {
    while (b < p.a.requests && at < end) {
      const int keys = keys_of(p, r, t), nk = (keys + 127) >> 7;
      const long long cost = r.ctx < 0 ? kItemCost : item + keys;
      const bool begins = at >= c0;
      s.b = b;
      s.h = h;
      s.row = r.row;
      s.tok0 = t * p.R;
      s.tokens = min(p.R, r.n - s.tok0);
      s.ctx = r.ctx;
      s.keys = keys;
      s.nk = nk;
      s.k0 = border(c0 - at, cost, nk, item);
      s.k1 = border(c1 - at, cost, nk, item);
      s.place = 2 * blockIdx.x + (begins ? 1 : 0);
      s.stop = 0;
      if (begins && at + cost > c1) {
        from = at;
        if ((threadIdx.x & 31) == 0) *last = s;   // (for shared(), at the end)
      }
      at += cost;
      if (++t == r.tiles) {
        t = 0;
        if (++h == p.a.kv_heads) {
          h = 0;
          following();
        }
      }
      if (s.k0 < s.k1 || (nk == 0 && begins)) return true;
    }
    return false;
  }
  // The row tile that this CTA begins and others go on with: which hold a part.
  __device__ __forceinline__ Tile shared() const {
    Tile m = {};
    if (from < 0 || last->nk == 0) return m;
    const long long cost = item + last->keys, share = c1 - c0, x = from + cost - 1 - c0;
    const int n = search(kAttnMaxCtas, x, [&](int i) { return i * share; });   // CTAs on, where the tile ends
    int first = blockIdx.x, end = min(blockIdx.x + n, gridDim.x - 1);
    if (last->k1 == 0) ++first;
    if (border(end * share - from, cost, last->nk, item) == last->nk) --end;
    if (end > first) {
      m.row = last->row + last->tok0;
      m.tokens = last->tokens;
      m.head = last->h;
      m.first = first;
      m.count = end - first + 1;
    }
    return m;
  }
  // Key tile at which a cost x into a row tile falls.
  static __device__ __forceinline__ int border(long long x, long long cost, int nk, int item) {
    if (x >= cost) return nk;
    const long long k = (x - item + 64) >> 7;
    return (int)(k < 0 ? 0 : k > nk ? nk : k);
  }
};

// Page number of the lane-th box of a part's pages from key tile k on: -1 behind
// the keys, kBadPage for a number outside the cache.
constexpr int kBadPage = -2;
__device__ __forceinline__ int first_pages(const TaParams& p, const Part& s, int k, int lane) {
  const int key = 128 * k + lane * min(1 << p.a.page_shift, 128);
  if (key >= min(s.keys, 128 * s.k1)) return -1;
  const int id = __ldcg(p.a.table + (long long)s.b * p.a.table_width + (key >> p.a.page_shift));
  return id >= 0 && id < p.a.cache.pages ? id : kBadPage;
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

// Sets the elements of 8 bf16 that are no finite numbers to zero; true if there are any.
__device__ __forceinline__ bool clear_unbounded(uint4& x) {
  constexpr uint32_t kExp = 0x7f80u;
  uint32_t* w = reinterpret_cast<uint32_t*>(&x);
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool lo = (w[i] & kExp) == kExp, hi = (w[i] & kExp << 16) == kExp << 16;
    if (lo) w[i] &= 0xffff0000u;
    if (hi) w[i] &= 0x0000ffffu;
    any |= lo || hi;
  }
  return any;
}

// Sets those of 4 e4m3 codes that are NaNs (all ones but for the sign) to zero; true if there are any.
__device__ __forceinline__ bool clear_nan_codes(uint32_t& x) {
  const uint32_t nan = ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  x &= ~((nan >> 7) * 0xffu);
  return nan != 0;
}

// Two e4m3 as fp16, exactly; a NaN stays one.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return h;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {   // (a NaN stays one)
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool E>
__device__ __forceinline__ float cache_value(const void* base, long long i) {
  if constexpr (E)
    return f16_lo(e4m3x2_f16x2(static_cast<const uint8_t*>(base)[i]));
  else
    return bf16_to_f32(static_cast<const uint16_t*>(base)[i]);
}

// ----------------------------------------------------------------- kernel ---
// Barriers by their shared-memory addresses: a role's warp runs alone, so that every
// instruction of its loop costs it a latency, conversions of pointers among them.
using Bar = uint32_t;
__device__ __forceinline__ bool bar_try(Bar b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(b), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void bar_arrive(Bar b) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(b) : "memory");
}
__device__ __forceinline__ void bar_expect(Bar b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(b), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_commit(Bar b) {   // once the products issued so far are done
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(b) : "memory");
}
__device__ __forceinline__ bool bar_drain(Bar b, uint32_t parity, unsigned long long limit_ns) {
  const unsigned long long t0 = globaltimer_ns();
  while (!bar_try(b, parity))
    if (globaltimer_ns() - t0 > limit_ns) return false;
  return true;
}

// Waits by a whole warp: true once the phase is over, false (and the CTA's abort
// flag set) when the limit ran out or another role gave up. The part that has to
// wait is a function of its own, out of the way of the roles' code: that of all
// of them has to fit the instruction cache together. The limit runs from the
// CTA's last step, told behind the flag: the key tiles whose scores were issued, the
// row tiles without keys that were written, and, at head_dim 256, each 32 columns of
// values that are no numbers that a warp has added. A long part may thus take its time,
// while the planner waits for its end, or the others for a part.
constexpr int kProgress = 1 + kParts;
__device__ __forceinline__ int steps_of(volatile int* abort_flag) {
  return abort_flag[kProgress] + abort_flag[kProgress + 1] + abort_flag[kProgress + 2];
}
__device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, volatile int* abort_flag, const DevErr* err,
                                         int site) {
  unsigned long long t0 = globaltimer_ns();
  int seen = steps_of(abort_flag);
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kWaitSleepNs)
        : "memory");
    if (__all_sync(0xffffffffu, ok)) return true;
    const bool late = globaltimer_ns() - t0 > err->limit_ns, aborted = *abort_flag != 0;
    if (__any_sync(0xffffffffu, late || aborted)) {
      const int now = steps_of(abort_flag);
      if (!__any_sync(0xffffffffu, aborted) && __any_sync(0xffffffffu, now != seen)) {
        seen = now;
        t0 = globaltimer_ns();
        continue;
      }
      if ((threadIdx.x & 31) == 0 && !*abort_flag) report_timeout(*err, site);
      *abort_flag = 1;
      return false;
    }
  }
}

// A place in a ring of N and the parity of its phase.
template <int N>   // (0 where a kernel has none)
struct Ring {
  uint32_t i = 0, phase = 0;
  __device__ __forceinline__ void step() {
    if (++i == N) {
      i = 0;
      phase ^= 1;
    }
  }
};

// Waits for a ring's last loads to land; i, phase: the place and parity of the next one.
template <int kMost>
__device__ __noinline__ void drain_ring(Bar bars, uint32_t i, uint32_t phase, uint32_t loads, uint32_t places,
                                        unsigned long long limit_ns) {
  for (uint32_t j = 0; j < min(loads, places) && j < kMost; ++j) {
    if (i-- == 0) {
      i = places - 1;
      phase ^= 1;
    }
    bar_drain(bars + 8 * i, phase, limit_ns);
  }
}

// The barriers. Each role works out their addresses for itself, from a base that
// the compiler cannot see through: addresses shared by the roles would all be held
// in registers throughout, at the cost of the softmax, which has none to spare.
template <int D, bool E>
struct Bars {
  using Sh = Shape<D, E>;
  static constexpr int kCount = 3 * Sh::SB + Sh::OB + 2 * (Sh::KS + Sh::VS + Sh::VR) + 3 * Sh::QB + 8 * Sh::SG + 2 * kParts + 2;
  Bar s_full;      // [SB] scores
  Bar p_full;      // [SB] weights
  Bar pv_done;     // [SB] products with values
  Bar o_free;      // [OB] sums written
  Bar k_full, k_free;     // [KS]
  Bar v_full, v_free;     // [VS]
  Bar rv_full, rv_free;   // [VR]
  Bar q_raw;       // [QB] queries landed (e4m3)
  Bar q_full;      // [QB] queries ready
  Bar q_empty;
  Bar hand;        // [4 quarters][SG][2] maxima handed on
  Bar part_full, part_empty;   // [kParts]
  Bar drain;       // [2]
  __device__ __forceinline__ explicit Bars(uint32_t words) {
    asm volatile("mov.u32 %0, %1;" : "=r"(s_full) : "r"(words));
    p_full = s_full + 8 * Sh::SB;
    pv_done = p_full + 8 * Sh::SB;
    o_free = pv_done + 8 * Sh::SB;
    k_full = o_free + 8 * Sh::OB;
    k_free = k_full + 8 * Sh::KS;
    v_full = k_free + 8 * Sh::KS;
    v_free = v_full + 8 * Sh::VS;
    rv_full = v_free + 8 * Sh::VS;
    rv_free = rv_full + 8 * Sh::VR;
    q_raw = rv_free + 8 * Sh::VR;
    q_full = q_raw + 8 * Sh::QB;
    q_empty = q_full + 8 * Sh::QB;
    hand = q_empty + 8 * Sh::QB;
    part_full = hand + 8 * 8 * Sh::SG;
    part_empty = part_full + 8 * kParts;
    drain = part_empty + 8 * kParts;
  }
};

template <int D, bool E>
__global__ void __launch_bounds__(Shape<D, E>::kThreads, 1)
    tree_attn_kernel(const __grid_constant__ TaParams p) {
  using Sh = Shape<D, E>;
  constexpr int NC = Sh::NC, GC = Sh::GC, NG = Sh::NG, KS = Sh::KS, VS = Sh::VS, VR = Sh::VR,
                QB = Sh::QB, OB = Sh::OB, SB = Sh::SB, SG = Sh::SG;
  constexpr uint32_t kColS = Sh::kColS;
  constexpr int kBars = Bars<D, E>::kCount;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sq = smem;
  uint8_t* s_keys = sq + QB * Sh::kQBytes + Sh::kQ8;
  uint8_t* s_values = s_keys + KS * Sh::kKBlock;
  uint8_t* raw_values = s_values + VS * Sh::kVBlock;
  uint8_t* misc = raw_values + VR * Sh::kRawBlock;
  float* s_top = reinterpret_cast<float*>(misc);   // [SG][2][128] maxima handed on
  // [kParts][SG - 1][128] a part's sums of the other groups, and the maxima that they refer to
  float2* s_sum = reinterpret_cast<float2*>(s_top + 256 * SG);
  float* s_qs = reinterpret_cast<float*>(s_sum + 128 * kParts * (SG - 1));   // [kParts][128] factors of 8-bit queries
  uint64_t* bar_words = reinterpret_cast<uint64_t*>(s_qs + (E ? kParts * 128 : 0));
  Part* parts = reinterpret_cast<Part*>(bar_words + kBars);
  int* s_pages = reinterpret_cast<int*>(parts + kParts + 1);    // [kParts][32] a part's first pages
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_pages + 32 * kParts);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // [kParts] a part's number where values were cleared; behind them the CTA's steps
  volatile int* s_unbounded = abort_flag + 1;
  static_assert((256 * SG + 256 * kParts * (SG - 1) + (E ? kParts * 128 : 0)) * 4 + 8 * kBars + (kParts + 1) * sizeof(Part) +
                    128 * kParts + 64 <= Sh::kMisc, "room for barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, role = warp - Sh::kSoftWarps;
  if (threadIdx.x < kBars) {
    // arrivals that a phase takes: 1 but for these
    const Bars<D, E> bs(smem_u32(bar_words));
    const Bar b = bs.s_full + 8 * threadIdx.x;
    const bool group = (b >= bs.p_full && b < bs.pv_done) || (b >= bs.o_free && b < bs.k_full);
    const bool conv = E && ((b >= bs.v_full && b < bs.v_free) || (b >= bs.rv_free && b < bs.q_raw) ||
                            (b >= bs.q_full && b < bs.q_empty));
    mbar_init(bar_words + threadIdx.x, group ? 4 : b >= bs.part_empty && b < bs.drain ? Sh::kSoftWarps
                                       : conv ? kConvWarps : 1);
    fence_mbar_init();
  }
  if (threadIdx.x < kParts) s_unbounded[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    abort_flag[0] = abort_flag[kProgress] = abort_flag[kProgress + 1] = abort_flag[kProgress + 2] = 0;
    tma_prefetch_desc(&p.mq);
    tma_prefetch_desc(&p.mk);
    tma_prefetch_desc(&p.mv);
  }
  if (role == kScore) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](Bar bar, uint32_t parity, int site) {
    return __all_sync(0xffffffffu, bar_try(bar, parity)) ||
           wait_longer(bar, parity, abort_flag, &p.err, site);
  };
  pdl_begin();
  if (role == kPlan) {
    const Bars<D, E> bs(smem_u32(bar_words));
    // ------------------------------------- the CTA's parts, for all others
    Walk walk(p, parts + kParts);
    walk.begin();
    Ring<kParts> at;
    Ring<QB> qring;
    uint32_t loads = 0;
    Part s;
    bool more = true, ok = true;
    while (more && ok) {
      more = walk.next(s);
      s.stop = !more;
      if (more && s.nk == 0) {   // no keys: zeros
        const int per_row = D / 8, n = s.tokens * p.G * per_row;
#pragma unroll 1
        for (int i = lane; i < n; i += 32) {
          const int r = i / per_row, tok = s.row + s.tok0 + r / p.G, head = s.h * p.G + r % p.G;
          *reinterpret_cast<uint4*>(p.a.out + (long long)tok * p.a.o_ld + (long long)head * D + 8 * (i % per_row)) =
              make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
        if (lane == 0) abort_flag[kProgress + 1] = abort_flag[kProgress + 1] + 1;
        continue;
      }
      const int page = more ? first_pages(p, s, s.k0, lane) : 0;
      if (!(ok = wait(bs.part_empty + 8 * at.i, at.phase ^ 1, 1))) break;
      s_pages[32 * at.i + lane] = page;
      if (lane == 0) parts[at.i] = s;
      __syncwarp();
      if (lane == 0) bar_arrive(bs.part_full + 8 * at.i);
      at.step();
      if (!more || !(ok = wait(bs.q_empty + 8 * qring.i, qring.phase ^ 1, 2))) break;
      if (elect_one_sync()) {
        const Bar bar = (E ? bs.q_raw : bs.q_full) + 8 * qring.i;
        bar_expect(bar, NC * 128 * p.G * p.R);
#pragma unroll 1
        for (int c = 0; c < NC; ++c)
          tma_load_q(smem_u32(sq) + qring.i * Sh::kQBytes + c * kSlotBytes, &p.mq, 64 * c, s.h * p.G, s.row + s.tok0, bar);
      }
      __syncwarp();
      qring.step();
      ++loads;
    }
    // own copies land before shared memory is released
    if (!ok) drain_ring<QB>(E ? bs.q_raw : bs.q_full, qring.i, qring.phase, loads, QB, p.err.limit_ns);
    __syncwarp();
    Tile m = walk.shared();
    if (*abort_flag) m.count = 0;
    if (lane == 0) p.shared[blockIdx.x] = packed(m);
  } else if (role == kLoad) {
    const Bars<D, E> bs(smem_u32(bar_words));
    // ------------------------- loads by TMA: a tile's keys, then the last tile's values
    const int box_log = max(7 - p.a.page_shift, 0), nbox = 1 << box_log, box = 128 >> box_log;
    const int my_box = lane & (nbox - 1), my_chunk = lane >> box_log;   // (chunk of a block)
    const int y_mask = (1 << p.a.page_shift) - 1;
    const bool mine = my_chunk < (E ? 1 : GC);
    const uint32_t offset = my_chunk * kSlotBytes + my_box * box * Sh::kKeyRow;
    const uint32_t k_to = smem_u32(s_keys) + offset, v_to = smem_u32(E ? raw_values : s_values) + offset;
    constexpr int kVBytes = E ? Sh::kRawBlock : Sh::kVBlock, kValues = E ? VR : VS;
    const Bar vf = E ? bs.rv_full : bs.v_full, ve = E ? bs.rv_free : bs.v_free;
    Ring<KS> keys;
    Ring<kValues> vals;
    Ring<kParts> at;
    uint32_t nk = 0, nv = 0;   // blocks loaded
    int v_id = -1, v_y = 0, v_h = 0;   // of the last tile's values
    bool ok = true, bad = false, due = false;
    auto load = [&](Bar full, uint32_t bytes, uint32_t to, const CUtensorMap* map, int g, int y, int h, int id) {
      if (lane == 0) bar_expect(full, bytes);
      __syncwarp();
      if (mine) tma_load_kv(to, map, 64 * (g * GC + my_chunk), y, h, id, full);
    };
    auto values = [&] {
#pragma unroll 1
      for (int g = 0; g < NG; ++g, vals.step(), ++nv) {
        if (!(ok = wait(ve + 8 * vals.i, vals.phase ^ 1, 4))) break;
        load(vf + 8 * vals.i, kVBytes, v_to + vals.i * kVBytes, &p.mv, g, v_y, v_h, v_id);
      }
    };
    while (ok) {
      if (!(ok = wait(bs.part_full + 8 * at.i, at.phase, 3))) break;
      const Part s = parts[at.i];
      if (s.stop) break;
      // page numbers of 32 boxes, one per lane, and of the next 32, read ahead
      int now = s_pages[32 * at.i + lane], later = first_pages(p, s, s.k0 + (32 >> box_log), lane);
      int src = my_box;   // the lane that holds the number
      at.step();
#pragma unroll 1
      for (int k = s.k0; k < s.k1 && ok; ++k) {
        int id = __shfl_sync(0xffffffffu, now, src);
        src += nbox;
        if (src >= 32) {
          src -= 32;
          now = later;
          later = first_pages(p, s, k + 1 + (32 >> box_log), lane);
        }
        bad |= id == kBadPage;
        if (id < 0) id = p.a.cache.pages;   // reads as zeros
        const int y = (128 * k + my_box * box) & y_mask;
#pragma unroll 1
        for (int g = 0; g < NG; ++g, keys.step(), ++nk) {
          if (!(ok = wait(bs.k_free + 8 * keys.i, keys.phase ^ 1, 4))) break;
          load(bs.k_full + 8 * keys.i, Sh::kKBlock, k_to + keys.i * Sh::kKBlock, &p.mk, g, y, s.h, id);
        }
        if (due && ok) values();
        due = true;
        v_id = id;
        v_y = y;
        v_h = s.h;
      }
    }
    if (due && ok) values();
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.err.word, DEVERR_RANGE);
    if (!ok) {
      drain_ring<4>(bs.k_full, keys.i, keys.phase, nk, KS, p.err.limit_ns);
      drain_ring<4>(vf, vals.i, vals.phase, nv, kValues, p.err.limit_ns);
    }
  } else if (role == kScore) {
    const Bars<D, E> bs(smem_u32(bar_words));
    // ----------------------------------------------- S = Q K^T, by key tile
    // (a place of scores is free once the product with the weights that took it is done)
    // e4m3: the queries' two terms times the codes as they lie in the cache.
    constexpr uint32_t kId = E ? idesc_e4m3(128) : idesc_16(true, 128, false);
    const uint32_t q_addr = smem_u32(sq) + Sh::kQ8, k_addr = smem_u32(s_keys);
    const uint64_t qd0 = E && D == 64 ? smem_desc_sw64(q_addr) : smem_desc_sw128(q_addr);
    const uint64_t kd0 = E && D == 64 ? smem_desc_sw64(k_addr) : smem_desc_sw128(k_addr);
    Ring<KS> keys;
    Ring<SB> sring;
    Ring<QB> qring;
    Ring<kParts> at;
    int issued = 0;
    bool ok = true;
    while (ok) {
      if (!(ok = wait(bs.part_full + 8 * at.i, at.phase, 5))) break;
      if (parts[at.i].stop) break;
      int n = parts[at.i].k1 - parts[at.i].k0;
      at.step();
      if (!(ok = wait(bs.q_full + 8 * qring.i, qring.phase, 6))) break;
      const uint64_t qd = qd0 + qring.i * (Sh::kQBytes / 16);
#pragma unroll 1
      for (; n > 0 && ok; --n, sring.step()) {
        if (!(ok = wait(bs.pv_done + 8 * sring.i, sring.phase ^ 1, 8))) break;
#pragma unroll 1
        for (int g = 0; g < NG; ++g, keys.step()) {
          if (!(ok = wait(bs.k_full + 8 * keys.i, keys.phase, 7))) break;
          tc_fence_after();
          if (elect_one_sync()) {
            const uint64_t a = qd + g * (Sh::kKBlock / 16), b = kd0 + keys.i * (Sh::kKBlock / 16);
            const uint32_t d = tmem + kColS + 128 * sring.i;
#pragma unroll
            for (int c = 0; c < 2; ++c)   // e4m3: the two terms
#pragma unroll
              for (int kk = 0; kk < (E ? 2 * GC : 4); ++kk) {
                if constexpr (E) {
                  mma_f8_ss(d, a + (c * NG * Sh::kKBlock + 32 * kk) / 16, b + 2 * kk, kId, g != 0 || (c | kk) != 0);
                } else if (c < GC) {
                  mma_f16_ss(d, a + (c * kSlotBytes + 32 * kk) / 16, b + (c * kSlotBytes + 32 * kk) / 16, kId,
                             g != 0 || (c | kk) != 0);
                }
              }
            if (g == NG - 1) bar_commit(bs.s_full + 8 * sring.i);
            bar_commit(bs.k_free + 8 * keys.i);
            if (n == 1 && g == NG - 1) bar_commit(bs.q_empty + 8 * qring.i);
            abort_flag[kProgress] = ++issued;
          }
          __syncwarp();
        }
      }
      qring.step();
    }
    if (elect_one_sync()) bar_commit(bs.drain);
    __syncwarp();
    bar_drain(bs.drain, 0, p.err.limit_ns);
  } else if (role == kSum) {
    const Bars<D, E> bs(smem_u32(bar_words));
    // ---------------------------------------------------------- O += P V
    constexpr uint32_t kId = idesc_16(!E, 64 * GC, true);
    const uint64_t vd0 = value_desc(smem_u32(s_values));
    Ring<VS> vals;
    Ring<SB> sring;
    Ring<OB> oring;
    Ring<kParts> at;
    bool ok = true;
    while (ok) {
      if (!(ok = wait(bs.part_full + 8 * at.i, at.phase, 9))) break;
      if (parts[at.i].stop) break;
      const int n = parts[at.i].k1 - parts[at.i].k0;
      at.step();
#pragma unroll 1
      for (int t = 0; t < n && ok; ++t, sring.step()) {
        if (!(ok = wait(bs.p_full + 8 * sring.i, sring.phase, 10))) break;
        if (t == 0 && !(ok = wait(bs.o_free + 8 * oring.i, oring.phase ^ 1, 11))) break;
#pragma unroll 1
        for (int g = 0; g < NG; ++g, vals.step()) {
          if (!(ok = wait(bs.v_full + 8 * vals.i, vals.phase, 12))) break;
          tc_fence_after();
          if (elect_one_sync()) {
            const uint64_t b = vd0 + vals.i * (Sh::kVBlock / 16);
            const uint32_t pc = tmem + kColS + 128 * sring.i, o = tmem + D * oring.i + 64 * GC * g;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)   // 16 keys each
              mma_f16_ts(o, pc + 8 * kk, b + (2048 >> 4) * kk, kId, t != 0 || kk != 0);
            if (g == NG - 1) bar_commit(bs.pv_done + 8 * sring.i);
            bar_commit(bs.v_free + 8 * vals.i);
          }
          __syncwarp();
        }
      }
      oring.step();
    }
    if (elect_one_sync()) bar_commit(bs.drain + 8);
    __syncwarp();
    bar_drain(bs.drain + 8, 0, p.err.limit_ns);
  } else if (E && role >= kConv) {
    const Bars<D, E> bs(smem_u32(bar_words));
    // --------------------------- queries to two e4m3 terms, values to fp16
    // A row of queries is multiplied by the power of two that brings its largest
    // element to 2^7..2^8, and its scores by the inverse. The first term is the
    // nearest e4m3, the second the nearest to what is left: of a bf16's 8 bits 4
    // each, exactly down to 2^-9 of the row's largest element (the second term's steps
    // end at 2^-9, the last bit of an element of 2^-2), and smaller elements
    // to 2^-17 of it. The codes of values are fp16 values; a warp has 32 rows of a block.
    const int w = role - kConv;
    Ring<VR> rvals;
    Ring<VS> vals;
    Ring<kParts> at;
    uint32_t np = 0;
    bool ok = true;
    while (ok) {
      if (!(ok = wait(bs.part_full + 8 * at.i, at.phase, 11))) break;
      const Part s = parts[at.i];
      if (s.stop) break;
      if (!(ok = wait(bs.q_raw, np & 1, 12))) break;
      const int rows = s.tokens * p.G;   // 8 lanes to a row, each 8 elements of every chunk
#pragma unroll 1
      for (int r0 = 4 * w; r0 < rows; r0 += 4 * kConvWarps) {
        const int r = r0 + (lane >> 3), piece = lane & 7;
        const uint8_t* line = sq + 128 * r + 16 * (piece ^ (r & 7));
        uint4 x[NC];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          x[c] = *reinterpret_cast<const uint4*>(line + c * kSlotBytes);
          const uint32_t y[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) top = max(top, max(y[j] & 0x7fffu, y[j] >> 16 & 0x7fffu));
        }
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        // exponent of the largest element, within what keeps both factors normal
        const int e = top >= 0x7f80u ? 7 : max((int)(top >> 7) - 127, -100);
        const float f = __uint_as_float((uint32_t)(7 - e + 127) << 23);
        __syncwarp();   // the row is read: its terms take its place
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const uint32_t y[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // (times 0: an infinity becomes a NaN, as nearly all of its row's results are)
            const float a0 = bf16_lo(y[j]) * f, b0 = bf16_hi(y[j]) * f;
            const float a = a0 + 0.0f * a0, b = b0 + 0.0f * b0;
            hi[j] = e4m3x2(a, b);
            const uint32_t h2 = e4m3x2_f16x2(hi[j]);
            lo[j] = e4m3x2(a - f16_lo(h2), b - f16_hi(h2));
          }
          // columns 64 c + 8 piece on: 8 bytes of the row of block c / GC
          const int byte = 64 * (c % GC) + 8 * piece, row_bytes = 64 * GC;
          const int at16 = D == 64 ? (byte >> 4) ^ (r >> 1 & 3) : (byte >> 4) ^ (r & 7);
          uint8_t* dst = sq + Sh::kQ8 + c / GC * Sh::kKBlock + row_bytes * r + 16 * at16 + (byte & 8);
          *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
          *reinterpret_cast<uint2*>(dst + NG * Sh::kKBlock) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
        }
        if (piece == 0) s_qs[at.i * 128 + r] = __uint_as_float((uint32_t)(e - 7 + 127) << 23);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive(bs.q_full);
      at.step();
      const int seen = p.a.mask ? s.ctx : s.ctx + s.tok0 + 1;
      // a lane's piece of 16 columns of chunk c: row 8 i + lane / 4 of the warp's 32
      const int row = 32 * w + (lane >> 2), piece = lane & 3;
      const int p0 = 16 * ((2 * piece) ^ (row & 7)), p1 = 16 * ((2 * piece + 1) ^ (row & 7));
#pragma unroll 1
      for (int kb = NG * s.k0; kb < NG * s.k1; ++kb, rvals.step(), vals.step()) {
        if (!(ok = wait(bs.rv_full + 8 * rvals.i, rvals.phase, 13))) break;
        if (!(ok = wait(bs.v_free + 8 * vals.i, vals.phase ^ 1, 14))) break;
        uint8_t* dst = s_values + vals.i * Sh::kVBlock + 128 * row;
        const uint8_t* src = raw_values + rvals.i * Sh::kRawBlock + 64 * GC * row + 16 * piece;
        const int key0 = 128 * (kb / NG) + row;
        const bool masked = 128 * (kb / NG + 1) > seen;
        bool any = false;
#pragma unroll 1
        for (int c = 0; c < GC; ++c) {
          uint4 x[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const uint4*>(src + 64 * c + 512 * GC * j);
          if (masked) {
            // values of a tile that not every row sees whole: what some row must not see
            // is cleared, keys past the row tile's own, and what is no number
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (key0 + 8 * j < seen) continue;
              if (key0 + 8 * j >= s.keys) x[j] = make_uint4(0, 0, 0, 0);
              any |= clear_nan_codes(x[j].x) | clear_nan_codes(x[j].y) | clear_nan_codes(x[j].z) | clear_nan_codes(x[j].w);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 y = x[j];
            uint8_t* line = dst + c * kSlotBytes + 1024 * j;
            *reinterpret_cast<uint4*>(line + p0) = make_uint4(e4m3x2_f16x2(y.x), e4m3x2_f16x2(y.x >> 16),
                                                              e4m3x2_f16x2(y.y), e4m3x2_f16x2(y.y >> 16));
            *reinterpret_cast<uint4*>(line + p1) = make_uint4(e4m3x2_f16x2(y.z), e4m3x2_f16x2(y.z >> 16),
                                                              e4m3x2_f16x2(y.w), e4m3x2_f16x2(y.w >> 16));
          }
        }
        if (any) s_unbounded[np % kParts] = (int)np + 1;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          bar_arrive(bs.v_full + 8 * vals.i);
          bar_arrive(bs.rv_free + 8 * rvals.i);
        }
      }
      ++np;
    }
  } else if (role < 0) {
    const Bars<D, E> bs(smem_u32(bar_words));
    // ------------------------------------------------- softmax, output
    // Groups of 4 warps take key tiles in turn, a row per thread; a warp's lanes
    // are those of its quarter of tensor memory. The running maximum goes from one
    // group to the next, as soon as a tile's scores are read; each group keeps sums
    // of its own, and the group of a part's last tile writes the part.
    const int group = warp >> 2, quarter = warp & 3, row = 32 * quarter + lane;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const int from = group == 0 ? SG - 1 : group - 1;
    const Bar give = bs.hand + 8 * (2 * SG * quarter + 2 * group);
    const Bar take = bs.hand + 8 * (2 * SG * quarter + 2 * from);
    float* top_out = s_top + 256 * group + row;
    const float* top_in = s_top + 256 * from + row;
    Ring<kParts> at;
    Ring<SB> sring;          // of key tile u
    Ring<OB> oring;
    uint32_t np = 0, u = 0, given = 0, taken = 0;
    int turn = 0;            // the group that key tile u is for
    bool ok = true;
    while (ok) {
      if (!(ok = wait(bs.part_full + 8 * at.i, at.phase, 16))) break;
      // (what the loop does not need at every tile is read again where it is used:
      // registers are short)
      const Part& s = parts[at.i];
      if (s.stop) break;
      const int k0 = s.k0, n = s.k1 - k0;
      const bool work = 32 * quarter < s.tokens * p.G;
      // keys before `seen` are seen by every row
      const int seen = p.a.mask ? s.ctx : s.ctx + s.tok0 + 1;
      auto token = [&] { return s.tok0 + row / p.G; };
      auto mask_words = [&] {
        return p.a.mask ? p.a.mask + (long long)(s.row + token()) * p.a.mask_words : nullptr;
      };
      // scores in log2
      float c2 = p.a.scale * (E ? p.a.cache.k_scale[s.h] : 1.0f) * 1.4426950408889634f;
      float m = -INFINITY, l = 0.0f;   // the maximum referred to; sums of this group's tiles
      int t = 0;
      for (; t < n; ++t, ++u, sring.step()) {
        const bool mine = turn == group;
        turn = turn == SG - 1 ? 0 : turn + 1;
        if (!mine) continue;
        const bool masked = 128 * (k0 + t + 1) > seen, last = t + 1 == n;
        const uint32_t sc = tmem + lanes + kColS + 128 * sring.i;
        // the maximum that O refers to (as a rule there before the scores are)
        float old = -INFINITY;
        if (work && t > 0) {
          if (!(ok = wait(take + 8 * (taken & 1), (taken >> 1) & 1, 15))) break;
          old = top_in[128 * (taken & 1)];
        }
        if (!(ok = wait(bs.s_full + 8 * sring.i, sring.phase, 17))) break;
        tc_fence_after();
        if (E && t < SG) c2 = fmaxf(c2 * s_qs[at.i * 128 + row], 1e-37f);   // (this group's first tile)
        if (work) {
          // Chunks of 32 scores. Of the four, the first two stay in registers; the
          // others are read again for their weights. Hidden scores become -inf.
          uint32_t x[2][32];
          const unsigned long long* words = nullptr;
          int tok = 0, a = 0;
          if (masked) {
            tok = token();
            a = 128 * (k0 + t) - s.ctx;
            words = mask_words();
          }
          auto hide = [&](uint32_t (&y)[32], int i) {
            const uint32_t v = row < s.tokens * p.G ? (uint32_t)seen_bits(a + i, tok, words, p.a.mask_words) : 0;
            if (__all_sync(0xffffffffu, v == 0xffffffffu)) return;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(v >> j & 1)) y[j] = 0xff800000u;
            if (i >= 64) tmem_st_32x32b_x32(sc + i, y);
          };
          auto largest = [&](const uint32_t (&y)[32]) {
            float a = -INFINITY, b = -INFINITY;
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              a = fmaxf(a, fmaxf(__uint_as_float(y[j]), __uint_as_float(y[j + 1])));
              b = fmaxf(b, fmaxf(__uint_as_float(y[j + 2]), __uint_as_float(y[j + 3])));
            }
            return fmaxf(a, b);
          };
          float top = -INFINITY;
          // (a loop: with the chunks' loads all at once the compiler spills)
#pragma unroll 1
          for (int i = 64; i < 128; i += 32) {
            tmem_ld_32x32b_x32(sc + i, x[0]);
            tmem_wait_ld(x[0]);
            if (masked) hide(x[0], i);
            top = fmaxf(top, largest(x[0]));
          }
          tmem_ld_32x32b_x32(sc, x[0]);
          tmem_ld_32x32b_x32(sc + 32, x[1]);
          tmem_wait_ld(x[0]);
          tmem_wait_ld(x[1]);
          if (masked) {
            hide(x[0], 0);
            hide(x[1], 32);
            tmem_wait_st();
          }
          top = fmaxf(top, fmaxf(largest(x[0]), largest(x[1])));
          top *= c2;
          // (NaN scores are left out of the maximum and make the sum NaN)
          const bool grow = top > old + kGrowth || old == -INFINITY;
          const float now = grow && top > old ? top : old;
          if (!last) {
            top_out[128 * (given & 1)] = now;
            __syncwarp();
            if (lane == 0) bar_arrive(give + 8 * (given & 1));
          }
          if (__any_sync(0xffffffffu, grow && old != -INFINITY)) {
            // the last product has to be done
            const uint32_t i = sring.i == 0 ? SB - 1 : sring.i - 1;
            if (!(ok = wait(bs.pv_done + 8 * i, sring.i == 0 ? sring.phase ^ 1 : sring.phase, 18))) break;
            tc_fence_after();
            const float f = grow && old != -INFINITY ? ex2(old - now) : 1.0f;
            const uint32_t oc = tmem + lanes + D * oring.i;
#pragma unroll 1
            for (int i = 0; i < D; i += 16) {
              uint32_t o[16];
              tmem_ld_32x32b_x16(oc + i, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st_32x32b_x16(oc + i, o);
            }
          }
          // with fp16 weights the reference is 2^7 below the maximum, which keeps
          // small ones of long contexts above fp16's smallest
          const float ref = (E ? 7.0f : 0.0f) - (now == -INFINITY ? 0.0f : now);
          float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
          auto weights = [&](const uint32_t (&y)[32], int i) {
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float2 a = fma2(__uint_as_float(y[2 * j]), __uint_as_float(y[2 * j + 1]), c2, ref);
              a.x = ex2(a.x);
              a.y = ex2(a.y);
              sum[j & 1] = add2(sum[j & 1], a);
              if constexpr (E) {
                const __half2 hv = __floats2half2_rn(a.x, a.y);
                w[j] = *reinterpret_cast<const uint32_t*>(&hv);
              } else {
                w[j] = pack_bf16x2(a.x, a.y);
              }
            }
            tmem_st_32x32b_x16(sc + i / 2, w);   // (in the place of scores that are read)
          };
          weights(x[0], 0);
          tmem_ld_32x32b_x32(sc + 64, x[0]);
          weights(x[1], 32);
          tmem_ld_32x32b_x32(sc + 96, x[1]);
          tmem_wait_ld(x[0]);
          tmem_wait_ld(x[1]);
          weights(x[0], 64);
          weights(x[1], 96);
          if (m != now) {   // (this group's sums refer to an older one)
            l *= m == -INFINITY ? 0.0f : ex2(m - now);
            m = now;
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          // (another group writes the part; what orders this is its wait for the product)
          if (!last && t + SG >= n) s_sum[128 * ((SG - 1) * at.i + n - 2 - t) + row] = make_float2(m, l);
          taken += t > 0;
          given += !last;
          tmem_wait_st();
        }
        if (!E && masked) {
          // Values that some row must not see: keys past the row tile's own are
          // nobody's, others only where they are no numbers. The block that had the
          // place before has to be consumed, so that the wait for this one is for its
          // phase.
          if (u > 0) {
            const uint32_t i = sring.i == 0 ? SB - 1 : sring.i - 1;
            if (!(ok = wait(bs.pv_done + 8 * i, sring.i == 0 ? sring.phase ^ 1 : sring.phase, 19))) break;
          }
          const int key = threadIdx.x & 127, j = 128 * (k0 + t) + key, keys = s.keys;
          bool any = false;
#pragma unroll 1
          for (int g = 0; g < NG; ++g) {
            const uint32_t i = (u * NG + g) % VS;
            if (!(ok = wait(bs.v_full + 8 * i, ((u * NG + g) / VS) & 1, 20))) break;
            if (j < seen) continue;
            // piece q % 8 of chunk q / 8
            auto piece = [&](int q) {
              return reinterpret_cast<uint4*>(s_values + i * Sh::kVBlock + (q >> 3) * kSlotBytes + 128 * key) +
                     ((q & 7) ^ (key & 7));
            };
            if (j >= keys) {
#pragma unroll
              for (int q = 0; q < GC * 8; ++q) *piece(q) = make_uint4(0, 0, 0, 0);
              continue;
            }
            uint32_t un = 0;   // (an exponent of all ones carries into its half's top bit)
#pragma unroll
            for (int q = 0; q < GC * 8; ++q) {
              const uint4 y = *piece(q);
              un |= ((y.x & 0x7f807f80u) + 0x00800080u) | ((y.y & 0x7f807f80u) + 0x00800080u) |
                    ((y.z & 0x7f807f80u) + 0x00800080u) | ((y.w & 0x7f807f80u) + 0x00800080u);
            }
            if (!(un & 0x80008000u)) continue;
            any = true;
#pragma unroll 1
            for (int q = 0; q < GC * 8; ++q) {
              uint4 y = *piece(q);
              if (clear_unbounded(y)) *piece(q) = y;
            }
          }
          if (!ok) break;
          if (any) s_unbounded[np % kParts] = (int)np + 1;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(bs.p_full + 8 * sring.i);
        if (!last) continue;

        // ------------------------------------------------- the part's sums
        if (!(ok = wait(bs.pv_done + 8 * sring.i, sring.phase, 21))) break;
        tc_fence_after();
        bool freed = false;
        if (work) {
#pragma unroll
          for (int i = 0; i < SG - 1; ++i) {
            if (i + 1 >= n) break;
            const float2 x = s_sum[128 * ((SG - 1) * at.i + i) + row];
            l += x.x == m ? x.y : x.y * (x.x == -INFINITY ? 0.0f : ex2(x.x - m));   // (a NaN stays)
          }
          const bool whole = k0 == 0 && n == s.nk, live = row < s.tokens * p.G;
          const float inv = whole ? (l == 0.0f ? 0.0f : (E ? p.a.cache.v_scale[s.h] : 1.0f) / l) : 1.0f;
          const int tok = token();
          uint16_t* out = p.a.out + (long long)(s.row + tok) * p.a.o_ld + (long long)(s.h * p.G + row % p.G) * D;
          float* dst = p.o + (long long)s.place * D * 128 + row;
          const uint32_t oc = tmem + lanes + D * oring.i;
          const bool fix = s_unbounded[np % kParts] == (int)np + 1;
          if constexpr (D <= 128) {
            // a whole row tile's results fit in registers: the next part has the sums'
            // place before they are stored
            if (whole && !fix) {
              uint32_t w[D / 2];
#pragma unroll
              for (int i = 0; i < D; i += 32) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(oc + i, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  w[i / 2 + j] = pack_bf16x2(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
              }
              tc_fence_before();
              __syncwarp();
              if (lane == 0) bar_arrive(bs.o_free + 8 * oring.i);
              freed = true;
              if (live) {
#pragma unroll
                for (int i = 0; i < D / 2; i += 4)
                  *reinterpret_cast<uint4*>(out + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
              }
            }
          }
#pragma unroll 1
          for (int i = freed ? D : 0; i < D; i += 32) {
            uint32_t o[32];
            __syncwarp();
            tmem_ld_32x32b_x32(oc + i, o);
            tmem_wait_ld(o);
            if (!live) continue;
            if (fix) {
              const unsigned long long* words = mask_words();
              // (new tokens without a bit are seen by none)
              const int end = min(min(s.keys, 128 * s.k1), words ? s.ctx + 64 * p.a.mask_words : INT_MAX);
#pragma unroll 1
              for (int j = max(seen, 128 * k0); j < end; ++j) {
                if (!(seen_bits(j - s.ctx, tok, words, p.a.mask_words) & 1)) continue;
                const int id = p.a.table[(long long)s.b * p.a.table_width + (j >> p.a.page_shift)];
                if (id < 0 || id >= p.a.cache.pages) continue;
                const long long e = ((((long long)id * p.a.kv_heads + s.h) << p.a.page_shift) +
                                     (j & ((1 << p.a.page_shift) - 1))) * D + i;
#pragma unroll
                for (int q = 0; q < 32; ++q) {
                  const float v = cache_value<E>(p.a.cache.v, e + q);
                  if (!(fabsf(v) < INFINITY)) o[q] = __float_as_uint(__uint_as_float(o[q]) + v);
                }
              }
              // (a part's 256 keys at most take a row's warp 1 ms at head_dim 256, half of that below,
              // where one more address held in registers cost 2 contexts of 131072 in e4m3 2%)
              if constexpr (D == 256)
                if (lane == 0) atomicAdd(const_cast<int*>(abort_flag) + kProgress + 2, 1);
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
#pragma unroll
              for (int q = 0; q < 32; ++q) dst[(i + q) * 128] = __uint_as_float(o[q]);
            }
          }
          if (!whole && live) p.ml[s.place * 128 + row] = make_float2(m == -INFINITY ? 0.0f : m, l);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !freed) bar_arrive(bs.o_free + 8 * oring.i);
      }
      __syncwarp();
      if (lane == 0) bar_arrive(bs.part_empty + 8 * at.i);
      at.step();
      oring.step();
      ++np;
    }
  }
  __syncthreads();
  if (role == kScore) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of the row tiles that CTAs share. A unit is 8 columns of 32
// rows, a row per lane; it has as many warps as 2 parts each need, up to all 8 of
// a block, which take alternate parts and add up through shared memory. The units
// of all shared tiles, in groups that fill a block, are dealt over the grid. Bound
// by its launch and four round trips where rows are few, else by reading the parts.
// Blocks per SM 5 (48 registers each, which spill), 3 and 2: one token 12.5, 11.0,
// 10.8 us, 32 trees of 128 rows 28.9, 27.1, 27.9, 2 long contexts 42.4, 40.2, 39.3.
// (16 blocks for each CTA that may have begun a tile: 15 us for the trees alone.)
constexpr int kJoinWarps = 8, kJoinGrid = 2;
__device__ __forceinline__ int join_log_per(int count) {   // log2 of a unit's warps
  return count <= 2 ? 0 : count <= 4 ? 1 : count <= 8 ? 2 : 3;
}
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps, kJoinGrid) tree_attn_join(const TaParams p, int ctas) {
  pdl_begin();
  constexpr int V = 8, U = 3, kCols = D / V, kRuns = kAttnMaxCtas / 32;
  __shared__ float s_o[kJoinWarps][V][32];
  __shared__ float2 s_ml[kJoinWarps][32];
  __shared__ unsigned long long s_tiles[kAttnMaxCtas];
  __shared__ int s_groups[kAttnMaxCtas];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  static_assert(kAttnMaxCtas <= 32 * kJoinWarps, "a thread per CTA");
  if (threadIdx.x < kAttnMaxCtas) {
    const unsigned long long x = (int)threadIdx.x < ctas ? p.shared[threadIdx.x] : 0;
    const Tile s = unpacked(x);
    s_tiles[threadIdx.x] = x;
    const int units = (s.tokens * p.G + 31) / 32 * kCols, log_once = 3 - join_log_per(s.count);
    s_groups[threadIdx.x] = s.count ? (units + (1 << log_once) - 1) >> log_once : 0;
  }
  __syncthreads();
  // groups of the tiles that CTAs kRuns * lane on begin, and of all before
  int groups[kRuns], before = 0;
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    groups[i] = s_groups[kRuns * lane + i];
    before += groups[i];
  }
  int mine = before;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += o;
  }
  const int total = __shfl_sync(0xffffffffu, before, 31);
  before -= mine;
  for (int g = blockIdx.x; g < total; g += gridDim.x) {
    // the tile of group g
    const int owner = __ffs(__ballot_sync(0xffffffffu, g >= before && g < before + mine)) - 1;
    int c = 0, rest = g - before;
#pragma unroll
    for (int i = 0; i < kRuns - 1; ++i)
      if (c == i && rest >= groups[i]) {
        rest -= groups[i];
        ++c;
      }
    c = __shfl_sync(0xffffffffu, kRuns * lane + c, owner);
    rest = __shfl_sync(0xffffffffu, rest, owner);
    const Tile s = unpacked(s_tiles[c]);
    const int log_per = join_log_per(s.count), per = 1 << log_per, sub = warp & (per - 1);
    const int rows = s.tokens * p.G, unit = (rest << (3 - log_per)) + (warp >> log_per);
    const int col = unit % kCols * V, row = 32 * (unit / kCols) + lane;
    const bool on = row < rows;
    float o[V] = {}, m = -INFINITY, l = 0.0f;
    for (int i0 = sub; on && i0 < s.count; i0 += U * per) {
      float x[U][V];
      float2 ml[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * per, cta = s.first + i;
        ml[u] = make_float2(0.0f, 0.0f);
        if (i < s.count) {
          // (the CTA that began the tile holds its part in its second place)
          const long long place = 2ll * cta + (cta == c);
          ml[u] = p.ml[place * 128 + row];
#pragma unroll
          for (int v = 0; v < V; ++v) x[u][v] = p.o[(place * D + col + v) * 128 + row];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (ml[u].y == 0.0f) continue;
        const float mn = fmaxf(m, ml[u].x), f = ex2(m - mn), e = ex2(ml[u].x - mn);
        m = mn;
        l = l * f + ml[u].y * e;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = o[v] * f + x[u][v] * e;
      }
    }
    if (per > 1) {
      __syncthreads();   // the last group's sums are read
#pragma unroll
      for (int v = 0; v < V; ++v) s_o[warp][v][lane] = o[v];
      s_ml[warp][lane] = make_float2(m, l);
      __syncthreads();
      if (sub == 0) {
        float2 ml[kJoinWarps];
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
          ml[w] = w < per ? s_ml[warp + w][lane] : make_float2(0.0f, 0.0f);
          if (ml[w].y != 0.0f) m = fmaxf(m, ml[w].x);   // (warp w = 0: its own)
        }
        l = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = 0.0f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
          if (ml[w].y == 0.0f) continue;
          const float e = ex2(ml[w].x - m);
          l += ml[w].y * e;
#pragma unroll
          for (int v = 0; v < V; ++v) o[v] += s_o[warp + w][v][lane] * e;
        }
      }
    }
    if (on && sub == 0) {
      const float scale = l == 0.0f ? 0.0f : (p.a.e4m3 ? p.a.cache.v_scale[s.head] : 1.0f) / l;
      const int tok = s.row + row / p.G;
      *reinterpret_cast<uint4*>(p.a.out + tok * p.a.o_ld + (long long)(s.head * p.G + row % p.G) * D + col) =
          make_uint4(pack_bf16x2(o[0] * scale, o[1] * scale), pack_bf16x2(o[2] * scale, o[3] * scale),
                     pack_bf16x2(o[4] * scale, o[5] * scale), pack_bf16x2(o[6] * scale, o[7] * scale));
    }
  }
}

bool encode_maps(const AttnArgs& a, int G, int R, TaParams* p) {
  const uint64_t D = a.head_dim, P = 1ull << a.page_shift, e = a.e4m3 ? 1 : 2;
  const uint64_t qd[3] = {D, (uint64_t)a.heads, (uint64_t)a.T}, qs[2] = {2 * D, 2 * (uint64_t)a.q_ld};
  const uint32_t qb[3] = {64, (uint32_t)G, (uint32_t)R};
  const uint64_t cd[4] = {D, P, (uint64_t)a.kv_heads, (uint64_t)a.cache.pages};
  const uint64_t cs[3] = {D * e, D * e * P, D * e * P * a.kv_heads};
  const uint32_t rows = (uint32_t)(P < 128 ? P : 128), cb[4] = {a.e4m3 && D > 64 ? 128u : 64u, rows, 1, 1};
  const auto dt = a.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  // keys are operands as they land; 8-bit values go through the converting warps
  const auto key_rows = a.e4m3 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  return encode_nd(&p->mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.q, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B) &&
         encode_nd(&p->mk, dt, 4, a.cache.k, cd, cs, cb, key_rows) &&
         encode_nd(&p->mv, dt, 4, a.cache.v, cd, cs, cb,
                   a.e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, bool E>
cudaError_t launch(const TaParams& p, int ctas, cudaStream_t st) {
  using Sh = Shape<D, E>;
  auto kern = tree_attn_kernel<D, E>;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), Sh::kSmem);
  if (e == cudaSuccess) e = launch_pdl(kern, dim3(ctas), dim3(Sh::kThreads), Sh::kSmem, st, p);
  if (e == cudaSuccess)
    e = launch_pdl(tree_attn_join<D>, dim3(ctas * kJoinGrid), dim3(32 * kJoinWarps), 0, st, p, ctas);
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
  p.shared = static_cast<unsigned long long*>(scratch);
  p.o = reinterpret_cast<float*>(p.shared + kAttnMaxCtas);
  p.ml = reinterpret_cast<float2*>(p.o + (size_t)kAttnMaxCtas * 2 * 128 * a.head_dim);
  if (!encode_maps(a, p.G, p.R, &p)) return cudaErrorInvalidValue;
  const int ctas = num_sms < kAttnMaxCtas ? num_sms : kAttnMaxCtas;
  p.inv_ctas = ~0ull / ctas + 1;
  p.inv_r = ((1u << 31) + p.R - 1u) / p.R;
  if (a.head_dim == 64) return a.e4m3 ? launch<64, true>(p, ctas, st) : launch<64, false>(p, ctas, st);
  if (a.head_dim == 128) return a.e4m3 ? launch<128, true>(p, ctas, st) : launch<128, false>(p, ctas, st);
  return a.e4m3 ? launch<256, true>(p, ctas, st) : launch<256, false>(p, ctas, st);
}

}  // namespace moe
