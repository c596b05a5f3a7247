// tree_attn.cu -- attention of new tokens, chains or drafted trees, over a paged
// cache (moe_tree_attention).
//
//   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  s_j = scale q . k_j
//
// in one pass over the keys with a running maximum m. One CTA per query row; its
// warps take alternate keys and their sums are joined at the end.
#include "attn.h"
#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kSimpleWarps = 8;

template <bool kE4m3>
__device__ __forceinline__ float cache_value(const void* base, long long i) {
  if constexpr (kE4m3) {
    const uint16_t c = static_cast<const uint8_t*>(base)[i];
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return f16_lo(h);
  } else {
    return bf16_to_f32(static_cast<const uint16_t*>(base)[i]);
  }
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(32 * kSimpleWarps) tree_attn_simple(const AttnArgs p, DevErr err) {
  pdl_begin();
  constexpr int N = D / 32;
  __shared__ float s_m[kSimpleWarps], s_l[kSimpleWarps], s_o[kSimpleWarps][D];
  __shared__ int s_bad;
  const int t = blockIdx.x, h = blockIdx.y, kh = h / (p.heads / p.kv_heads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int b = -1, i = 0, n = 0;
  for (int r = 0; r < p.requests; ++r) {
    const int lo = max(p.offsets[r], 0), hi = min(p.offsets[r + 1], p.T);
    if (t >= lo && t < hi) {
      b = r;
      i = t - lo;
      n = hi - lo;
      break;
    }
  }
  if (b < 0) return;
  int len = p.length[b];
  if (len > (p.table_width << p.page_shift)) {
    len = p.table_width << p.page_shift;
    if (threadIdx.x == 0) atomicOr(err.word, DEVERR_RANGE);
  }
  if (len < n) len = 0;
  const int ctx = len - n;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  float q[N], o[N], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int x = 0; x < N; ++x) {
    q[x] = bf16_to_f32(p.q[t * p.q_ld + (long long)h * D + lane + 32 * x]);
    o[x] = 0.0f;
  }
  const float ks = kE4m3 ? p.cache.k_scale[kh] : 1.0f, vs = kE4m3 ? p.cache.v_scale[kh] : 1.0f;
  const int last = min(len, ctx + i + 1);
  for (int j = warp; j < last; j += kSimpleWarps) {
    const int node = j - ctx;
    if (node >= 0 && p.mask &&
        (node >= 64 * p.mask_words ||
         !(p.mask[(long long)t * p.mask_words + (node >> 6)] >> (node & 63) & 1)))
      continue;
    const int page = p.table[(long long)b * p.table_width + (j >> p.page_shift)];
    const bool there = page >= 0 && page < p.cache.pages;
    if (!there) s_bad = 1;
    const long long row = ((((long long)page * p.kv_heads + kh) << p.page_shift) +
                           (j & ((1 << p.page_shift) - 1))) * D + lane;
    float s = 0.0f;
#pragma unroll
    for (int x = 0; x < N; ++x)
      if (there) s += q[x] * cache_value<kE4m3>(p.cache.k, row + 32 * x);
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= p.scale * ks;
    const float mn = s > m || s != s ? s : m;
    const float f = m == mn ? 1.0f : expf(m - mn), w = expf(s - mn);
    m = mn;
    l = l * f + w;
#pragma unroll
    for (int x = 0; x < N; ++x) {
      o[x] *= f;
      if (there) o[x] += w * cache_value<kE4m3>(p.cache.v, row + 32 * x);
    }
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int x = 0; x < N; ++x) s_o[warp][lane + 32 * x] = o[x];
  __syncthreads();
  if (threadIdx.x == 0 && s_bad) atomicOr(err.word, DEVERR_RANGE);
  float M = -INFINITY;
  for (int w = 0; w < kSimpleWarps; ++w) M = s_m[w] > M || s_m[w] != s_m[w] ? s_m[w] : M;
  for (int d = threadIdx.x; d < D; d += 32 * kSimpleWarps) {
    float sum = 0.0f, tot = 0.0f;
    for (int w = 0; w < kSimpleWarps; ++w) {
      if (s_l[w] == 0.0f) continue;
      const float f = s_m[w] == M ? 1.0f : expf(s_m[w] - M);
      sum += f * s_l[w];
      tot += f * s_o[w][d];
    }
    p.out[t * p.o_ld + (long long)h * D + d] = f32_to_bf16(sum == 0.0f ? 0.0f : tot / sum * vs);
  }
}

}  // namespace

cudaError_t launch_tree_attention(const AttnArgs& a, DevErr err, cudaStream_t st) {
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3(a.T, a.heads), dim3(32 * kSimpleWarps), 0, st, a, err);
  };
  if (a.head_dim == 64) return a.e4m3 ? go(tree_attn_simple<64, true>) : go(tree_attn_simple<64, false>);
  if (a.head_dim == 128) return a.e4m3 ? go(tree_attn_simple<128, true>) : go(tree_attn_simple<128, false>);
  return a.e4m3 ? go(tree_attn_simple<256, true>) : go(tree_attn_simple<256, false>);
}

}  // namespace moe
