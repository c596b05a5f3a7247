// route_scored.cu -- routing by scores (moe_route_scored): each token's choice
// (score_topk.cuh), then counts, offsets, tile offsets, the stable scatter and
// the block map, as moe_route makes them.
//
// CTA b takes tokens [b C, (b + 1) C), a warp a token at a time, and keeps, per
// expert, a bit for each of its tokens that chose it. Its counts go to a byte
// table [CTA][expert]; once all are there, every CTA reads the whole table, which
// gives it all totals and its own starting positions, and writes its slots:
// position = start + earlier tokens of the CTA that chose the expert (a popcount
// of the bits below). The block map is dealt over the CTAs by expert.
//
// Bound by the latency of one warp's choice for few tokens (one of 256 experts in
// 8 groups: 4.7 us in a graph) and by the choice's instructions for many, about
// 950 a token (4096 x 256 in 8 groups 12 us, 16384 x 512 32 us, of which the
// placing takes 4 to 5).
//
// Up to 32 tokens are one CTA's, in one launch. More are two launches, the
// choice and the placing. (With a grid barrier in one cooperative launch the GPU
// spent as long, 11.6 us at 4096 x 256 with 8 groups in a graph, but in a stream
// a cooperative launch waits 3 us longer for its turn.)
#include <type_traits>

#include "score_topk.cuh"

namespace moe {
namespace {

constexpr int kScThreads = 1024;
constexpr int kScMaxC = 224;          // tokens per CTA: counts fit a byte
constexpr int kScWords = kScMaxC / 32;

struct ScParams {
  ScoreDev s;
  const float* logits;
  int T, E, k, C;
  int32_t *idx;
  float* w;
  uint8_t* table;                     // [CTAs][E]
  int32_t *cnt, *off, *tile_off, *bmap, *num_tiles, *perm, *inv;
};

// kPart: kAll in one CTA, or kChoose and then kPlace.
enum { kAll, kChoose, kPlace };

template <int VPL, int kPart>
__global__ void __launch_bounds__(kScThreads) score_route_kernel(const ScParams p) {
  constexpr int kE = 32 * VPL;
  extern __shared__ float dyn[];           // a row per warp; kPlace: the partial sums
  __shared__ unsigned mask_s[kScWords * kE];   // [word][expert]
  __shared__ int start_s[kE];
  __shared__ int wrows_s[16], wtiles_s[16];
  __shared__ uint16_t idx_s[kScMaxC * 32];     // the CTA's choices, [token][k]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int E = p.E, k = p.k, b = blockIdx.x, G = gridDim.x;
  const int t0 = b * p.C, nt = min(p.C, p.T - t0);
  const int words = (p.C + 31) / 32;
  for (int i = tid; i < words * kE; i += kScThreads) mask_s[i] = 0u;
  __syncthreads();
  pdl_begin();

  if constexpr (kPart != kPlace) {
    for (int tl = warp; tl < nt; tl += kScThreads / 32) {
      const size_t t = t0 + tl;
      int idx;
      float w;
      score_select<VPL>(p.logits + t * E, E, k, p.s, dyn + warp * max(kE, 64), idx, w);
      if (lane < k) {
        p.idx[t * k + lane] = idx;
        p.w[t * k + lane] = w;
        if (kPart == kAll) idx_s[tl * k + lane] = (uint16_t)idx;
        atomicOr(&mask_s[(tl >> 5) * kE + idx], 1u << (tl & 31));
      }
      __syncwarp();
    }
  } else {
    for (int i = tid; i < nt * k; i += kScThreads) {
      const int tl = i / k, e = __ldcg(p.idx + (size_t)t0 * k + i);
      idx_s[i] = (uint16_t)e;
      atomicOr(&mask_s[(tl >> 5) * kE + e], 1u << (tl & 31));
    }
  }
  __syncthreads();
  int tot = 0, before = 0;                 // thread e < E: all CTAs', earlier CTAs'
  if (kPart != kPlace && tid < E)
    for (int i = 0; i < words; ++i) tot += __popc(mask_s[i * kE + tid]);
  if constexpr (kPart == kChoose) {
    if (tid < E) p.table[(size_t)b * E + tid] = (uint8_t)tot;
    return;
  }
  if constexpr (kPart == kPlace) {
    // the table, 4 experts per thread, the rows dealt over the rest of the
    // threads: totals in the low halves, earlier CTAs' in the high halves
    uint32_t* part = reinterpret_cast<uint32_t*>(dyn);   // [rows' share][E]
    const int e4 = E / 4, shares = min(kScThreads / e4, 32), q = tid / e4, c = tid % e4;
    if (q < shares) {
      uint32_t s0 = 0, s1 = 0, s2 = 0, s3 = 0;
      for (int r0 = q; r0 < G; r0 += 10 * shares) {   // 10 rows' loads at once
        uint32_t v[10];
#pragma unroll
        for (int i = 0; i < 10; ++i) {
          const int r = r0 + i * shares;
          v[i] = r < G ? __ldcg(reinterpret_cast<const uint32_t*>(p.table + (size_t)r * E) + c) : 0u;
        }
#pragma unroll
        for (int i = 0; i < 10; ++i) {
          const uint32_t f = r0 + i * shares < b ? 0x10001u : 1u;
          s0 += (v[i] & 0xFFu) * f;
          s1 += ((v[i] >> 8) & 0xFFu) * f;
          s2 += ((v[i] >> 16) & 0xFFu) * f;
          s3 += (v[i] >> 24) * f;
        }
      }
      uint32_t* o = part + q * E + 4 * c;
      o[0] = s0;
      o[1] = s1;
      o[2] = s2;
      o[3] = s3;
    }
    __syncthreads();
    if (tid < E) {
      tot = 0;
      for (int i = 0; i < shares; ++i) {
        const uint32_t v = part[i * E + tid];
        tot += v & 0xFFFFu;
        before += v >> 16;
      }
    }
  }
  // exclusive scans over the experts: rows and tiles
  const int tiles = (tot + kBM - 1) / kBM;
  int ri = tot, ti = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int rn = __shfl_up_sync(0xffffffffu, ri, o), tn = __shfl_up_sync(0xffffffffu, ti, o);
    if (lane >= o) {
      ri += rn;
      ti += tn;
    }
  }
  if (lane == 31 && warp < 16) {
    wrows_s[warp] = ri;
    wtiles_s[warp] = ti;
  }
  __syncthreads();
  if (tid < E) {
    int ro = ri - tot, to = ti - tiles;
#pragma unroll
    for (int w2 = 0; w2 < 16; ++w2)
      if (w2 < warp) {
        ro += wrows_s[w2];
        to += wtiles_s[w2];
      }
    start_s[tid] = ro + before;
    if (tid % G == b) {
      p.cnt[tid] = tot;
      p.off[tid] = ro;
      p.tile_off[tid] = to;
      for (int i = 0; i < tiles; ++i) {
        int32_t* m = p.bmap + 3 * (size_t)(to + i);
        m[0] = tid;
        m[1] = ro + kBM * i;
        m[2] = min(kBM, tot - kBM * i);
      }
    }
    if (b == 0 && tid == E - 1) {
      p.off[E] = ro + tot;
      p.tile_off[E] = to + tiles;
      p.num_tiles[0] = to + tiles;
    }
  }
  __syncthreads();
  // the CTA's slots, in token order within each expert
  for (int i = tid; i < nt * k; i += kScThreads) {
    const int tl = i / k, slot = t0 * k + i;
    const int e = idx_s[i];
    int pos = start_s[e] + __popc(mask_s[(tl >> 5) * kE + e] & ((1u << (tl & 31)) - 1u));
    for (int wd = 0; wd < (tl >> 5); ++wd) pos += __popc(mask_s[wd * kE + e]);
    p.perm[pos] = slot;
    p.inv[slot] = pos;
  }
}

// The choice alone, 32 tokens per CTA, with the block's counts as
// launch_route_scan takes them (batches beyond score_route_kernel's).
template <int VPL>
__global__ void __launch_bounds__(kScThreads) score_topk_kernel(const ScoreDev s, const float* logits,
                                                                int T, int E, int k, int32_t* topk_idx,
                                                                float* topk_w, int32_t* blk_cnt) {
  constexpr int kE = 32 * VPL;
  extern __shared__ float dyn[];
  __shared__ int cnt_s[kE];
  pdl_begin();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = blockIdx.x * kRouterTB + warp;
  for (int i = tid; i < E; i += kScThreads) cnt_s[i] = 0;
  __syncthreads();
  if (t < T) {
    int idx;
    float w;
    score_select<VPL>(logits + (size_t)t * E, E, k, s, dyn + warp * max(kE, 64), idx, w);
    if (lane < k) {
      topk_idx[(size_t)t * k + lane] = idx;
      topk_w[(size_t)t * k + lane] = w;
      atomicAdd(&cnt_s[idx], 1);
    }
  }
  __syncthreads();
  for (int e = tid; e < E; e += kScThreads) blk_cnt[(size_t)blockIdx.x * E + e] = cnt_s[e];
}

// Experts per lane.
int vpl_of(int E) { return E <= 64 ? 2 : E <= 128 ? 4 : E <= 256 ? 8 : 16; }

ScoreDev dev_of(const ScoreArgs& a, int E) {
  ScoreDev s{a.sigmoid, a.groups, a.topk_groups, a.renorm, a.scale, a.bias, E / a.groups, 0, 0, 0};
  s.gdiv = ((1 << 20) + s.gsz - 1) / s.gsz;
  const int vpl = vpl_of(E), per = s.gsz / vpl;
  s.whole = s.gsz % vpl == 0 && (per & (per - 1)) == 0;
  int lanes = per;
  if (!s.whole)
    for (lanes = 32; lanes * a.groups > 32; lanes >>= 1) {
    }
  while ((1 << s.span_log2) < lanes) ++s.span_log2;
  return s;
}

// dynamic shared memory: a row per warp, or the partial sums (1024 threads' four)
constexpr int kPartBytes = kScThreads * 16;
constexpr int dyn_bytes(int vpl) { return 32 * 32 * (vpl < 4 ? 4 : vpl) * 4; }

}  // namespace

// Tokens per CTA and CTAs: one CTA up to 32 tokens (a token per warp); then 16
// tokens a CTA until every SM has one.
static void score_grid(int T, int num_sms, int* C, int* G) {
  int g = T <= 32 ? 1 : (T + 15) / 16;
  if (g > num_sms) g = num_sms;
  *C = (T + g - 1) / g;
  *G = (T + *C - 1) / *C;
}

bool score_route_fits(int T, int num_sms) {
  int C, G;
  score_grid(T, num_sms, &C, &G);
  return C <= kScMaxC;
}

cudaError_t launch_score_route(const ScoreArgs& a, const float* logits, int T, int E, int k,
                               int32_t* topk_idx, float* topk_w, uint8_t* table, int32_t* cnt,
                               int32_t* off, int32_t* tile_off, int32_t* bmap, int32_t* num_tiles,
                               int32_t* perm, int32_t* inv, int num_sms, cudaStream_t st) {
  ScParams p;
  int G;
  score_grid(T, num_sms, &p.C, &G);
  if (p.C > kScMaxC || E > 512 || k > 32) return cudaErrorInvalidValue;
  p.s = dev_of(a, E);
  p.logits = logits;
  p.T = T;
  p.E = E;
  p.k = k;
  p.idx = topk_idx;
  p.w = topk_w;
  p.table = table;
  p.cnt = cnt;
  p.off = off;
  p.tile_off = tile_off;
  p.bmap = bmap;
  p.num_tiles = num_tiles;
  p.perm = perm;
  p.inv = inv;
  auto go = [&](auto kern, int smem) -> cudaError_t {
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
    return e != cudaSuccess ? e : launch_pdl(kern, dim3(G), dim3(kScThreads), smem, st, p);
  };
  auto all = [&](auto vpl) -> cudaError_t {
    constexpr int V = decltype(vpl)::value;
    if (G == 1) return go(score_route_kernel<V, kAll>, dyn_bytes(V));
    const cudaError_t e = go(score_route_kernel<V, kChoose>, dyn_bytes(V));
    return e != cudaSuccess ? e : go(score_route_kernel<V, kPlace>, kPartBytes);
  };
  switch (vpl_of(E)) {
    case 2: return all(std::integral_constant<int, 2>{});
    case 4: return all(std::integral_constant<int, 4>{});
    case 8: return all(std::integral_constant<int, 8>{});
    default: return all(std::integral_constant<int, 16>{});
  }
}

cudaError_t launch_score_topk(const ScoreArgs& a, const float* logits, int T, int E, int k,
                              int32_t* topk_idx, float* topk_w, int32_t* blk_cnt, cudaStream_t st) {
  const int nblk = (T + kRouterTB - 1) / kRouterTB;
  auto go = [&](auto kern, int smem) -> cudaError_t {
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(nblk), dim3(kScThreads), smem, st, dev_of(a, E), logits, T, E, k,
                      topk_idx, topk_w, blk_cnt);
  };
  switch (vpl_of(E)) {
    case 2: return go(score_topk_kernel<2>, dyn_bytes(2));
    case 4: return go(score_topk_kernel<4>, dyn_bytes(4));
    case 8: return go(score_topk_kernel<8>, dyn_bytes(8));
    default: return go(score_topk_kernel<16>, dyn_bytes(16));
  }
}

}  // namespace moe
