// w4_linear.cu -- 4-bit projection with the low-rank adapters of many requests
// at once (moe_linear_forward):
//   y[t] = x_scale[t] (x[t] W^T + scale[a] (x[t] A[a]^T) B[a]^T),  a = adapter[t]
// W is 4-bit affine in groups of 64 along K (moe_w4).
//
// A decode batch is a matter of latency and of the packed weights' bytes: one
// launch takes h = scale x A^T, and the next, which starts while that runs,
// multiplies straight from the packed weights on mma.sync and adds h B^T at
// its end. More tokens are tensor-core work (linear_tc.cu); the launch here
// that goes before it writes x and W as fp16 and h.
#include <cuda_fp8.h>

#include <type_traits>

#include "moe_common.cuh"

namespace moe {
namespace {

// D += A B, m16n8k16, bf16 operands, fp32 accumulation
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// two e4m3 codes -> f16x2 (exact)
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
  return r;
}

// 8 values of a row, as stored
struct Raw8 {
  uint4 v;   // bf16, or e4m3 codes in x and y
};

__device__ __forceinline__ Raw8 load8(const LinearArgs& a, int t, int k) {
  Raw8 r;
  if (a.e4m3) {
    const uint2 c = __ldcg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.x) + t * a.x_ld + k));
    r.v = make_uint4(c.x, c.y, 0u, 0u);
  } else {
    r.v = __ldcg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + t * a.x_ld + k));
  }
  return r;
}

// The 8 values as fp16 in their order; sets `over` where a bf16 value is
// beyond fp16's range (it saturates).
__device__ __forceinline__ uint4 to_f16(const LinearArgs& a, const Raw8& r, uint32_t& over) {
  if (a.e4m3)
    return make_uint4(e4m3x2_to_f16x2(r.v.x), e4m3x2_to_f16x2(r.v.x >> 16),
                      e4m3x2_to_f16x2(r.v.y), e4m3x2_to_f16x2(r.v.y >> 16));
  over |= bf16x2_f16_overflow(r.v.x) | bf16x2_f16_overflow(r.v.y) | bf16x2_f16_overflow(r.v.z) |
          bf16x2_f16_overflow(r.v.w);
  return make_uint4(bf16x2_to_f16x2_sat(r.v.x), bf16x2_to_f16x2_sat(r.v.y),
                    bf16x2_to_f16x2_sat(r.v.z), bf16x2_to_f16x2_sat(r.v.w));
}

// The 8 values as bf16 (exact for e4m3: 4 significant bits).
__device__ __forceinline__ uint4 to_bf16(const LinearArgs& a, const Raw8& r) {
  if (!a.e4m3) return r.v;
  uint32_t over = 0u;
  const uint4 f = to_f16(a, r, over);
  return make_uint4(pack_bf16x2(f16_lo(f.x), f16_hi(f.x)), pack_bf16x2(f16_lo(f.y), f16_hi(f.y)),
                    pack_bf16x2(f16_lo(f.z), f16_hi(f.z)), pack_bf16x2(f16_lo(f.w), f16_hi(f.w)));
}

// The adapter of token t, or -1.
__device__ __forceinline__ int adapter_of(const LinearArgs& a, int t) {
  if (!a.la || t >= a.T) return -1;
  const int id = __ldcg(a.adapter + t);
  return (unsigned)id < (unsigned)a.n_adapters ? id : -1;
}

// Whether a bf16 scale or bias is outside the fp16 operand contract: a scale
// is 0 or in [2^-14, 2^12), a bias below 2^11.
__device__ __forceinline__ bool sb_out_of_range(uint32_t s, uint32_t b) {
  const uint32_t ms = s & 0x7FFFu, mb = b & 0x7FFFu;
  return (ms != 0u && (ms < 0x3880u || ms >= 0x4580u)) || mb >= 0x4500u;
}

// ---------------------------------------------------------------------------
// Decode batches, first launch: h[t][r] = scale[a] sum_k x[t][k] A[a][r][k],
// one warp per (t, r).
// ---------------------------------------------------------------------------
template <bool kE4m3>
__global__ void __launch_bounds__(1024) lora_shrink_kernel(const LinearArgs args) {
  LinearArgs a = args;
  a.e4m3 = kE4m3;
  pdl_begin();
  const int lane = threadIdx.x & 31;
  const int w = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (w >= a.T * a.rank) return;
  const int t = w / a.rank, r = w - t * a.rank;
  const int id = adapter_of(a, t);
  float s = 0.f;
  if (id >= 0) {
    const uint16_t* ar = a.la + ((size_t)id * a.rank + r) * a.K;
#pragma unroll 8
    for (int k = 8 * lane; k < a.K; k += 256) {
      const Raw8 r = load8(a, t, k);
      const uint4 av = __ldg(reinterpret_cast<const uint4*>(ar + k));
      const uint32_t aw[4] = {av.x, av.y, av.z, av.w}, xw[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float x0, x1;
        if (a.e4m3) {
          const uint32_t f = e4m3x2_to_f16x2(xw[j >> 1] >> (16 * (j & 1)));
          x0 = f16_lo(f);
          x1 = f16_hi(f);
        } else {
          x0 = bf16_lo(xw[j]);
          x1 = bf16_hi(xw[j]);
        }
        s = fmaf(x0, bf16_lo(aw[j]), fmaf(x1, bf16_hi(aw[j]), s));
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) a.h[w] = id >= 0 ? s * (a.lscale ? __ldg(a.lscale + id) : 1.f) : 0.f;
}

// ---------------------------------------------------------------------------
// Decode batches, the product: a CTA takes 16 weight rows and up to 32 tokens, its
// 16 warps every 16th group of 64 K each. The packed words are the MMA's A
// rows: lane (g, q) rebuilds the 16 weights of words 2q and 2q + 1 of rows g
// and g + 8, in the order in which the nibbles come out (perm8), and takes the
// same K positions of token g's row as B. The warps' sums are added in a fixed
// order through shared memory. All loads of two groups are in flight before the
// first is used (24 tokens of 2048 x 2048, without adapters: 4.7 us, 6.1 with x
// loaded where it is used), which takes 128 registers above 8 tokens: then a CTA
// has its SM for itself. Weights are loaded before the wait for the launch
// before. With adapters that launch is lora_shrink_kernel, and x and the adapters'
// ids are older than it: all that does not need h runs beside it. Bound by
// latency: one token of 2048 x 2048 2.9 us, with an adapter 4.3; 16 tokens 3.6
// and 5.2.
// (h taken in this launch instead, once per cluster of 8 CTAs and shared over
// distributed shared memory, was slower when it was tried: 6.6 against 4.7 us at
// one token of 2048 x 2048 and rank 16, 12.4 against 6.6 us at 16. Against 8 warps
// of twice the groups, 16 warps: 3.2 against 4.6 us at one token without
// adapters.)
// ---------------------------------------------------------------------------
constexpr int kSmRows = 16;
constexpr int kSmWarps = 16;

template <int NT, bool kE4m3>   // tiles of 8 tokens; the rows' type
__global__ void __launch_bounds__(32 * kSmWarps) __maxnreg__(NT == 1 ? 64 : 128)
    linear_small_kernel(const LinearArgs args, const DevErr err) {
  LinearArgs a = args;
  a.e4m3 = kE4m3;
  __shared__ float red[kSmWarps][kSmRows][8 * NT + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int n0 = blockIdx.x * kSmRows, kg = a.K / 64;
  const int r0 = min(n0 + g, a.N - 1), r1 = min(n0 + g + 8, a.N - 1);   // rows past N: not stored
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  uint32_t over = 0u;
  bool bad = false, waited = a.la != nullptr;
  // This thread's output: row tid % 16 of the CTA's token tid / 16. What its adapter adds
  // is loaded ahead, up to 16 ranks, so that only h is left to come when the
  // sums are done.
  const int t0 = 8 * NT * blockIdx.y, tl = tid / kSmRows;
  const int to = tl < 8 * NT ? t0 + tl : a.T, no = n0 + tid % kSmRows;
  int id = -1;
  uint4 b0v = make_uint4(0u, 0u, 0u, 0u), b1v = b0v;
  float xsc = 1.f;
  auto ahead = [&] {
    if (to >= a.T) return;
    id = adapter_of(a, to);
    if (a.x_scale) xsc = __ldcg(a.x_scale + to);
    if (id >= 0 && no < a.N) {
      const uint4* br = reinterpret_cast<const uint4*>(a.lb + ((size_t)id * a.N + no) * a.rank);
      b0v = __ldg(br);
      if (a.rank > 8) b1v = __ldg(br + 1);
    }
  };
  if (waited) ahead();
  constexpr int kAhead = 2;
  for (int gb = warp; gb < kg || !waited; gb += kSmWarps * kAhead) {
    uint2 w0[kAhead], w1[kAhead];
    uint32_t s0[kAhead], s1[kAhead], b0[kAhead], b1[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int gr = gb + kSmWarps * i;
      w0[i] = w1[i] = make_uint2(0u, 0u);
      s0[i] = s1[i] = b0[i] = b1[i] = 0u;
      if (gr < kg) {
        w0[i] = __ldg(reinterpret_cast<const uint2*>(a.w.q + (size_t)r0 * (a.K / 8) + 8 * gr + 2 * q));
        w1[i] = __ldg(reinterpret_cast<const uint2*>(a.w.q + (size_t)r1 * (a.K / 8) + 8 * gr + 2 * q));
        s0[i] = __ldg(a.w.s + (size_t)r0 * kg + gr);
        s1[i] = __ldg(a.w.s + (size_t)r1 * kg + gr);
        b0[i] = __ldg(a.w.b + (size_t)r0 * kg + gr);
        b1[i] = __ldg(a.w.b + (size_t)r1 * kg + gr);
      }
    }
    if (!waited) {
      pdl_begin();
      waited = true;
      ahead();
    }
    Raw8 xr[kAhead][NT][2];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int wd = 0; wd < 2; ++wd) {
          const int gr = gb + kSmWarps * i, t = t0 + 8 * nt + g;
          xr[i][nt][wd].v = make_uint4(0u, 0u, 0u, 0u);
          if (gr < kg && t < a.T) xr[i][nt][wd] = load8(a, t, 64 * gr + 8 * (2 * q + wd));
        }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int gr = gb + kSmWarps * i;
      if (gr >= kg) break;
      bad |= sb_out_of_range(s0[i], b0[i]) || sb_out_of_range(s1[i], b1[i]);
      const __half2 sa = __half2half2(__float2half_rn(bf16_to_f32((uint16_t)s0[i])));
      const __half2 ba = __half2half2(__float2half_rn(bf16_to_f32((uint16_t)b0[i])));
      const __half2 sb = __half2half2(__float2half_rn(bf16_to_f32((uint16_t)s1[i])));
      const __half2 bb = __half2half2(__float2half_rn(bf16_to_f32((uint16_t)b1[i])));
#pragma unroll
      for (int wd = 0; wd < 2; ++wd) {
        uint32_t oa[4], ob[4];
        dequant_word_f16_perm8(wd ? w0[i].y : w0[i].x, sa, ba, oa);
        dequant_word_f16_perm8(wd ? w1[i].y : w1[i].x, sb, bb, ob);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint4 xv = f16x8_to_perm8(to_f16(a, xr[i][nt][wd], over));
          mma_m16n8k16_f16(acc[nt], oa[0], ob[0], oa[1], ob[1], xv.x, xv.y);
          mma_m16n8k16_f16(acc[nt], oa[2], ob[2], oa[3], ob[3], xv.z, xv.w);
        }
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 4; ++j) red[warp][g + 8 * (j >> 1)][8 * nt + 2 * q + (j & 1)] = acc[nt][j];
  if (__any_sync(0xffffffffu, over != 0u || bad) && lane == 0) atomicOr(err.word, DEVERR_RANGE);
  __syncthreads();
  float v = 0.f;
  if (tl < 8 * NT) {
#pragma unroll
    for (int w = 0; w < kSmWarps; ++w) v += red[w][tid % kSmRows][tl];
  }
  if (a.la) pdl_begin();   // h
  if (to >= a.T || no >= a.N) return;
  if (id >= 0) {
    const uint4* br = reinterpret_cast<const uint4*>(a.lb + ((size_t)id * a.N + no) * a.rank);
    const float4* hr = reinterpret_cast<const float4*>(a.h + (size_t)to * a.rank);
    float e = 0.f;
    auto eight = [&](int c, const uint4& b) {
      const float4 h0 = __ldcg(hr + 2 * c), h1 = __ldcg(hr + 2 * c + 1);
      e = fmaf(h0.x, bf16_lo(b.x), fmaf(h0.y, bf16_hi(b.x), e));
      e = fmaf(h0.z, bf16_lo(b.y), fmaf(h0.w, bf16_hi(b.y), e));
      e = fmaf(h1.x, bf16_lo(b.z), fmaf(h1.y, bf16_hi(b.z), e));
      e = fmaf(h1.z, bf16_lo(b.w), fmaf(h1.w, bf16_hi(b.w), e));
    };
    eight(0, b0v);
    if (a.rank > 8) eight(1, b1v);
#pragma unroll 2
    for (int c = 2; c < a.rank / 8; ++c) eight(c, __ldg(br + c));
    v += e;
  }
  a.y[to * a.y_ld + no] = f32_to_bf16(v * xsc);
}

// ---------------------------------------------------------------------------
// Larger batches, first launch, in clusters of 4 CTAs, or 8 where the tokens'
// tile of a quarter of K is beyond shared memory. The first nx CTAs are
// token CTAs (they take longer): a cluster takes 32 tokens, each of its CTAs an
// equal part of K. A CTA writes its part of x as fp16 rows in perm8 order and
// keeps it in shared memory as bf16; then its 8 warps take jobs of (adapter
// among the 32 tokens, 8 ranks) on mma.sync, each over the CTA's whole part of
// K, and put the rows of the adapter's own tokens into shared memory. The
// cluster adds its CTAs' sums in order, over distributed shared memory, into h.
// (One CTA per 16 tokens that went through the adapters one by one, its warps
// splitting K, took 20 us for 4096 tokens of 2048 and 80 us for 128 tokens of
// 16 adapters: one chain of L2 round trips per adapter.)
// The other CTAs rebuild 8192 packed weights each as fp16 in perm8 order.
// Weights are loaded before the wait for the launch before; x and the adapters'
// ids, which that launch may write, after it. Bound by latency and L2: about 8 us
// of the 53.2 at 4096 x 2048 x 4096. (Eight parts of K: 4096 tokens of 14,336 x
// 4096 with 8 adapters of rank 16 463 us, four parts at K = 13,056, the largest
// that fits at every rank, 408.)
// ---------------------------------------------------------------------------
constexpr int kPrepTok = 32;
constexpr int kPrepWords = 1024;   // packed words per weight CTA

// K columns of a token CTA (a multiple of 32), and bytes of a row of its tile
// (64 more: 8 lanes of one 16-byte load then touch all banks)
__host__ __device__ constexpr int prep_cols(int K, int split) { return (K / 32 + split - 1) / split * 32; }
__host__ __device__ constexpr int prep_row_bytes(int K, int split) { return prep_cols(K, split) * 2 + 64; }
// shared memory of a token CTA beside its static 4.5 KB: the tile and the sums
constexpr int prep_smem(int K, int rank, int split) { return kPrepTok * (prep_row_bytes(K, split) + rank * 4); }
constexpr int kPrepSmemMax = 227 * 1024 - 5 * 1024;

__device__ __forceinline__ void prep_weights(const LinearArgs& a, uint16_t* __restrict__ w16, int cta,
                                             const DevErr& err) {
  const long long words = (long long)a.N * (a.K / 8);
  // loaded before the wait for the launch before, whose last CTAs this runs beside
  constexpr int kN = kPrepWords / 256;
  uint32_t q[kN], s[kN], b[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const long long wi = (long long)cta * kPrepWords + 256 * i + threadIdx.x;
    q[i] = s[i] = b[i] = 0u;
    if (wi < words) {
      q[i] = __ldg(a.w.q + wi);
      s[i] = __ldg(a.w.s + (wi >> 3));
      b[i] = __ldg(a.w.b + (wi >> 3));
    }
  }
  pdl_begin();
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const long long wi = (long long)cta * kPrepWords + 256 * i + threadIdx.x;
    if (wi < words) {
      bad |= sb_out_of_range(s[i], b[i]);
      uint32_t o[4];
      dequant_word_f16_perm8(q[i], __half2half2(__float2half_rn(bf16_to_f32((uint16_t)s[i]))),
                             __half2half2(__float2half_rn(bf16_to_f32((uint16_t)b[i]))), o);
      reinterpret_cast<uint4*>(w16)[wi] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  report_range_warp(err, bad);
}

// Orders the block of n tokens from blk0 by adapter modulo 256 (none: as 255), a
// warp's tokens one after the other, and keeps the 32 tokens (and their adapters)
// that get the cluster's places, from t0. bins: 8 x 256, tokens by warp and bin.
// Every CTA does it by itself. (Out of line: most calls skip it.)
__device__ __noinline__ void order_block(const int32_t* adapter, int n_adapters, int blk0, int n, int t0,
                                         uint16_t* bins, int* s_sum, int* s_tok, int* s_id) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int steps = (n + 255) / 256, w0 = 32 * steps * warp;
  constexpr int kSteps = kOrderBlock / 256;
  int id[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int j = w0 + 32 * i + lane;
    id[i] = i < steps && j < n ? __ldcg(adapter + blk0 + j) : -1;
    if ((unsigned)id[i] >= (unsigned)n_adapters) id[i] = -1;
  }
  reinterpret_cast<uint4*>(bins)[tid] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  // a token's number among its warp's of its bin, the bins' counts
  int nth[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    if (i < steps) {
      const int bin = w0 + 32 * i + lane < n ? id[i] & 255 : 256;
      const unsigned same = __match_any_sync(0xffffffffu, bin);
      const int before = bin < 256 ? bins[256 * warp + bin] : 0;
      nth[i] = before + __popc(same & ((1u << lane) - 1u));
      __syncwarp();
      if (bin < 256 && (same >> lane) == 1u) bins[256 * warp + bin] = (uint16_t)(nth[i] + 1);
      __syncwarp();
    }
  }
  __syncthreads();
  // thread b: where bin b starts, and each warp's part of it
  int count = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const int c = bins[256 * w + tid];
    bins[256 * w + tid] = (uint16_t)count;
    count += c;
  }
  int start = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, start, o);
    if (lane >= o) start += v;
  }
  if (lane == 31) s_sum[warp] = start;
  __syncthreads();
  start -= count;
#pragma unroll
  for (int w = 0; w < 8; ++w) start += w < warp ? s_sum[w] : 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) bins[256 * w + tid] += (uint16_t)start;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSteps; ++i)
    if (i < steps && w0 + 32 * i + lane < n) {
      const int place = bins[256 * warp + (id[i] & 255)] + nth[i] - (t0 - blk0);
      if (place >= 0 && place < kPrepTok) {
        s_tok[place] = blk0 + w0 + 32 * i + lane;
        s_id[place] = id[i];
      }
    }
  __syncthreads();
}

// kDeep: twice the loads in flight per thread, for half the CTAs per SM: faster
// where the launch has at most four CTAs per SM, the shorter weight CTAs counted
// half (128, 1024, 2048 tokens of 2048 x 2048: 13.6, 17.3, 23.9 us for the call
// against 14.6, 19.2, 25.9), slower beyond (4096 tokens: 37.1 against 34.8).
template <int kSplit, bool kDeep, bool kE4m3>   // kSplit: parts of K, CTAs per cluster
__global__ void __cluster_dims__(kSplit, 1, 1) __launch_bounds__(256, kDeep ? 2 : 4)
    linear_prep_kernel(const LinearArgs args, uint16_t* __restrict__ x16, uint16_t* __restrict__ w16, int nx,
                       const DevErr err) {
  LinearArgs a = args;
  a.e4m3 = kE4m3;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int s_id[kPrepTok], s_list[kPrepTok], s_tok[kPrepTok], s_sum[8];
  __shared__ __align__(16) uint16_t s_bin[8][256];   // tokens by warp and bin of adapters
  if ((int)blockIdx.x >= nx) {
    prep_weights(a, w16, (int)blockIdx.x - nx, err);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part_k = (int)blockIdx.x % kSplit, t0 = (int)blockIdx.x / kSplit * kPrepTok;
  const int cols = prep_cols(a.K, kSplit), k0 = part_k * cols, kn = max(0, min(cols, a.K - k0));
  const int row_bytes = prep_row_bytes(a.K, kSplit);
  float* part = reinterpret_cast<float*>(smem + kPrepTok * row_bytes);   // [token][rank]
  // x, 8 columns at a time: a warp takes every 8th row, kCols vectors of each of
  // its 4 rows in flight per lane
  constexpr int kCols = kDeep ? 2 : 1, kABatch = kDeep ? 16 : 8;
  const int vec = kn / 8;
  uint32_t over = 0u;
  Raw8 xv[4][kCols];
  auto get_x = [&](int c0, auto&& token) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        const int c = c0 + 32 * j + lane, t = token(warp + 8 * r);
        xv[r][j].v = make_uint4(0u, 0u, 0u, 0u);
        if (c < vec && t < a.T) xv[r][j] = load8(a, t, k0 + 8 * c);
      }
  };
  auto put_x = [&](int c0) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        const int c = c0 + 32 * j + lane, tl = warp + 8 * r, t = t0 + tl;
        if (c >= vec) continue;
        if (t < a.T)
          *reinterpret_cast<uint4*>(x16 + (size_t)t * a.K + k0 + 8 * c) = f16x8_to_perm8(to_f16(a, xv[r][j], over));
        if (a.la) *reinterpret_cast<uint4*>(smem + tl * row_bytes + 16 * c) = to_bf16(a, xv[r][j]);
      }
  };
  pdl_begin();   // (x and the ids may be the launch before's output)
  const int blk0 = t0 / kOrderBlock * kOrderBlock, n = min(kOrderBlock, a.T - blk0);
  int id0 = -1, id1 = -1, own_id = -1;
  if (a.la) {
    const int at = order_sample(tid, n);
    if (tid < kOrderSamples && at < n) {
      id0 = adapter_of(a, blk0 + at - 1);
      id1 = adapter_of(a, blk0 + at);
    }
    if (tid < kPrepTok) own_id = adapter_of(a, t0 + tid);
  }
  get_x(0, [&](int tl) { return t0 + tl; });
  if (a.la) {
    // are the block's tokens to be ordered by adapter?
    const bool change = id0 != id1;
    if (tid < kPrepTok) {
      s_tok[tid] = t0 + tid;
      s_id[tid] = own_id;
    }
    const bool ordered = order_rule(__syncthreads_count(change), n);
    // (x's loads stay where they are, under the ids')
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < kCols; ++j)
        asm volatile("" : "+r"(xv[r][j].v.x), "+r"(xv[r][j].v.y), "+r"(xv[r][j].v.z), "+r"(xv[r][j].v.w));
    if (ordered) {
      order_block(a.adapter, a.n_adapters, blk0, n, t0, &s_bin[0][0], s_sum, s_tok, s_id);
      get_x(0, [&](int tl) { return s_tok[tl]; });
    }
    if (part_k == 0 && tid < kPrepTok && t0 + tid < a.T) a.order[t0 + tid] = s_tok[tid];
  }
  put_x(0);
  for (int c0 = 32 * kCols; c0 < vec; c0 += 32 * kCols) {
    get_x(c0, [&](int tl) { return a.la ? s_tok[tl] : t0 + tl; });
    put_x(c0);
  }
  report_range_warp(err, over != 0u);
  if (!a.la) return;
  // the 32 tokens' distinct adapters, in order (every warp alike)
  const int tiles = a.rank / 8;
  int jobs;
  {
    const int id = s_id[lane];
    bool first = id >= 0;
#pragma unroll
    for (int j = 0; j < 31; ++j) {
      const int o = __shfl_sync(0xffffffffu, id, j);
      if (j < lane && o == id) first = false;
    }
    const unsigned firsts = __ballot_sync(0xffffffffu, first);
    if (warp == 0) {
      if (first) s_list[__popc(firsts & ((1u << lane) - 1u))] = id;
    }
    jobs = __popc(firsts) * tiles;
  }
  __syncthreads();
  const int g = lane >> 2, q = lane & 3;
  for (int job = warp; job < jobs; job += 8) {
    const int ad = s_list[job / tiles], r0 = 8 * (job % tiles);
    const uint16_t* ar = a.la + ((size_t)ad * a.rank + r0 + g) * a.K + k0 + 8 * q;
    const uint8_t* xr = smem + g * row_bytes + 16 * q;
    float acc[2][4] = {};
    for (int kb0 = 0; kb0 < kn; kb0 += 32 * kABatch) {
      uint4 w[kABatch];
#pragma unroll
      for (int j = 0; j < kABatch; ++j)
        w[j] = kb0 + 32 * j < kn ? __ldg(reinterpret_cast<const uint4*>(ar + kb0 + 32 * j))
                                 : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int j = 0; j < kABatch; ++j) {
        const int kb = kb0 + 32 * j;
        if (kb < kn) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            const uint4 xa = *reinterpret_cast<const uint4*>(xr + (16 * mt) * row_bytes + 2 * kb);
            const uint4 xb = *reinterpret_cast<const uint4*>(xr + (16 * mt + 8) * row_bytes + 2 * kb);
            mma_bf16(acc[mt], xa.x, xb.x, xa.y, xb.y, w[j].x, w[j].y);
            mma_bf16(acc[mt], xa.z, xb.z, xa.w, xb.w, w[j].z, w[j].w);
          }
        }
      }
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tl = 16 * mt + 8 * h + g;
        if (s_id[tl] == ad)
          *reinterpret_cast<float2*>(part + tl * a.rank + r0 + 2 * q) =
              make_float2(acc[mt][2 * h], acc[mt][2 * h + 1]);
      }
  }
  // the cluster's sums, each CTA an equal part of the entries
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  const int sums = kPrepTok * a.rank;
  for (int i = part_k * 256 + tid; i < sums; i += 256 * kSplit) {
    const int tl = i / a.rank, ad = s_id[tl];
    if (ad < 0) continue;
    float v = 0.f;
#pragma unroll
    for (int c = 0; c < kSplit; ++c) {
      uint32_t addr;
      float o;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(part + i)), "r"(c));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o) : "r"(addr) : "memory");
      v += o;
    }
    a.h[(size_t)(t0 + tl) * a.rank + i % a.rank] = v * (a.lscale ? __ldg(a.lscale + ad) : 1.f);
  }
  // no CTA leaves while another still reads its sums
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Tiles of 8 tokens per CTA, and microseconds that the product of a decode batch
// takes: rounds of CTAs over the SMs, each of them by K and tiles. Measured
// without adapters, one round of 2, 3, 4 tiles of bf16 at K = 1024 2.5, 3.0, 4.1,
// at 2048 3.7, 4.7, 6.6, at 4096 5.7, 7.6, 11.1 us, two rounds of 4 tiles 8.1,
// 12.7, 22.0; of e4m3 2.0, 2.3, 2.9, 3.2, 3.6, 4.5, 4.0, 4.8, 6.1, and 6.0, 7.7,
// 12.4. (Two CTAs of one tile are not better than one of two: 16 tokens of 4096 x
// 1024 6.0 and 5.7, with adapters 10.0 and 7.4.)
double small_cost(const LinearArgs& a, int num_sms, int* nt_out) {
  const double k = a.K / 1024.0;
  const int ctas = (a.N + kSmRows - 1) / kSmRows;
  double best = 1e30;
  for (int nt = a.T > 8 ? 2 : 1; nt <= 4; ++nt) {
    const long long all = (long long)ctas * ((a.T + 8 * nt - 1) / (8 * nt));
    const double c = 1.0 + (double)((all + num_sms - 1) / num_sms) * (a.e4m3 ? 1.0 + 0.3 * nt * k : 0.9 + 0.6 * nt * k);
    if (c < best) {
      best = c;
      *nt_out = nt;
    }
  }
  return best;
}

}  // namespace

// Beyond 32 tokens small sizes stay with the decode batches' kernels while
// conversion and tcgen05 product are estimated to take longer: these measured, at
// 48 and 64 tokens without adapters, 7.4 us at K x N = 1024 x 1024, 10.2 at 2048 x
// 2048, 13.2 at 4096 x 1024, 12.8 at 2048 x 4096, 17.2 at 4096 x 4096 (the estimate
// is 0.4 less to 1.2 more), and 6 to 11 us more with adapters. (48 bf16 tokens of
// rank 16, both ways: 1024 x 1024 4.8 and 15.5 us, 2048 x 2048 10.7 and 17.1, 4096 x
// 1024 9.6 and 24.1, 2048 x 4096 19.1 and 18.7, 4096 x 4096 31.9 and 28.2; without
// adapters 3.0 and 7.4, 8.9 and 10.1, 8.1 and 13.2, 16.5 and 12.8, 28.6 and 17.1.)
bool linear_is_small(const LinearArgs& a, int num_sms) {
  if (a.T <= kLinearSmallT) return true;
  const double k = a.K / 1024.0;
  int nt;
  double small = small_cost(a, num_sms, &nt), large = 6.5 + 1.65 * k + 0.33 * k * (a.N / 1024.0);
  if (a.la) {
    small += 1.5 + 1.1 * k * ((double)a.T * a.rank / 1024.0);
    large += 3.0 + 1.6 * k;
  }
  return small < large;
}

cudaError_t launch_linear_small(const LinearArgs& a, DevErr err, int num_sms, cudaStream_t st) {
  int nt;
  small_cost(a, num_sms, &nt);
  const int ny = (a.T + 8 * nt - 1) / (8 * nt), rows = (a.N + kSmRows - 1) / kSmRows, ctas = rows * ny;
  if (a.la) {
    // Of more than one tile the product's CTAs find no room beside this launch's,
    // which are then made fewer: so that each has an SM, if that can be had (2048 x
    // 2048, rank 16, CTAs of 8, 16, 32 warps: 16 tokens 6.4, 5.2, 5.3 us, 32
    // tokens 10.0, 9.9, 8.6; of 64 registers at 4 tokens 4.4, 4.8, 5.2).
    auto shrink_ctas = [&](int warps) { return (a.T * a.rank + warps - 1) / warps; };
    int warps = nt == 1 ? 8 : 16;
    if (nt > 1 && shrink_ctas(16) + ctas > num_sms && shrink_ctas(32) + ctas <= num_sms) warps = 32;
    const cudaError_t e = launch_pdl(a.e4m3 ? lora_shrink_kernel<true> : lora_shrink_kernel<false>,
                                     dim3(shrink_ctas(warps)), dim3(32 * warps), 0, st, a);
    if (e != cudaSuccess) return e;
  }
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3(rows, ny), dim3(32 * kSmWarps), 0, st, a, err);
  };
  auto pick = [&](auto e4m3) {
    constexpr bool k = decltype(e4m3)::value;
    return nt == 1   ? go(linear_small_kernel<1, k>)
           : nt == 2 ? go(linear_small_kernel<2, k>)
           : nt == 3 ? go(linear_small_kernel<3, k>)
                     : go(linear_small_kernel<4, k>);
  };
  return a.e4m3 ? pick(std::true_type{}) : pick(std::false_type{});
}

cudaError_t launch_linear_prep(const LinearArgs& a, uint16_t* x16, uint16_t* w16, DevErr err,
                               int num_sms, cudaStream_t st) {
  const long long words = (long long)a.N * (a.K / 8);
  // (beyond K = 13,056 to 13,952, by rank; the largest sizes fit eight parts)
  static_assert(prep_smem(16384, 128, 8) <= kPrepSmemMax, "K and rank at most");
  const bool eight = a.la && prep_smem(a.K, a.rank, 4) > kPrepSmemMax;
  const int split = eight ? 8 : 4, smem = a.la ? prep_smem(a.K, a.rank, split) : 0;
  int nw = (int)((words + kPrepWords - 1) / kPrepWords);
  nw = (nw + split - 1) / split * split;   // whole clusters
  const int nx = (a.T + kPrepTok - 1) / kPrepTok * split;
  auto go = [&](auto kern) {
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
    return e != cudaSuccess
               ? e
               : launch_pdl(kern, dim3(nx + nw), dim3(256), (size_t)smem, st, a, x16, w16, nx, err);
  };
  auto pick = [&](auto e4m3) {
    constexpr bool k = decltype(e4m3)::value;
    // (a tile of more than 100 KB leaves an SM no more CTAs than the deep kernel's)
    if (eight) return go(linear_prep_kernel<8, true, k>);
    return nx + nw / 2 <= 4 * num_sms ? go(linear_prep_kernel<4, true, k>) : go(linear_prep_kernel<4, false, k>);
  };
  return a.e4m3 ? pick(std::true_type{}) : pick(std::false_type{});
}

}  // namespace moe
