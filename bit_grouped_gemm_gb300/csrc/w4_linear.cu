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
__global__ void __launch_bounds__(256) lora_shrink_kernel(const LinearArgs a) {
  pdl_begin();
  const int lane = threadIdx.x & 31;
  const int w = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= a.T * a.rank) return;
  const int t = w / a.rank, r = w - t * a.rank;
  const int id = adapter_of(a, t);
  float s = 0.f;
  if (id >= 0) {
    const uint16_t* ar = a.la + ((size_t)id * a.rank + r) * a.K;
#pragma unroll 4
    for (int k = 8 * lane; k < a.K; k += 256) {
      const uint4 xv = to_bf16(a, load8(a, t, k));
      const uint4 av = __ldg(reinterpret_cast<const uint4*>(ar + k));
      const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w}, aw[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s = fmaf(bf16_lo(xw[j]), bf16_lo(aw[j]), fmaf(bf16_hi(xw[j]), bf16_hi(aw[j]), s));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) a.h[w] = id >= 0 ? s * (a.lscale ? __ldg(a.lscale + id) : 1.f) : 0.f;
}

// ---------------------------------------------------------------------------
// Decode batches, the product: a CTA takes 16 weight rows and all tokens, its
// 8 warps every 8th group of 64 K each. The packed words are the MMA's A rows:
// lane (g, q) rebuilds the 16 weights of words 2q and 2q + 1 of rows g and
// g + 8, in the order in which the nibbles come out (perm8), and takes the
// same K positions of token g's row as B. Weights are loaded before the wait
// for the launch before; x too when that launch is this call's own (it is then
// older). The warps' sums are added in a fixed order through shared memory.
// ---------------------------------------------------------------------------
constexpr int kSmRows = 16;

template <int NT>   // tiles of 8 tokens
__global__ void __launch_bounds__(256) linear_small_kernel(const LinearArgs a, const DevErr err) {
  __shared__ float red[8][kSmRows][8 * NT + 1];
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
  constexpr int kAhead = 4;
  for (int gb = warp; gb < kg; gb += 8 * kAhead) {
    uint2 w0[kAhead], w1[kAhead];
    uint32_t s0[kAhead], s1[kAhead], b0[kAhead], b1[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int gr = gb + 8 * i;
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
      pdl_wait();
      waited = true;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int gr = gb + 8 * i;
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
        const int k = 64 * gr + 8 * (2 * q + wd);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int t = 8 * nt + g;
          uint4 xv = make_uint4(0u, 0u, 0u, 0u);
          if (t < a.T) xv = f16x8_to_perm8(to_f16(a, load8(a, t, k), over));
          mma_m16n8k16_f16(acc[nt], oa[0], ob[0], oa[1], ob[1], xv.x, xv.y);
          mma_m16n8k16_f16(acc[nt], oa[2], ob[2], oa[3], ob[3], xv.z, xv.w);
        }
      }
    }
  }
  if (!waited || a.la) pdl_wait();   // h; and every thread waits before it stores
  pdl_trigger();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 4; ++j) red[warp][g + 8 * (j >> 1)][8 * nt + 2 * q + (j & 1)] = acc[nt][j];
  if (__any_sync(0xffffffffu, over != 0u || bad) && lane == 0) atomicOr(err.word, DEVERR_RANGE);
  __syncthreads();
  for (int o = tid; o < kSmRows * a.T; o += 256) {
    const int t = o / kSmRows, r = o % kSmRows, n = n0 + r;
    if (n >= a.N) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += red[w][r][t];
    const int id = adapter_of(a, t);
    if (id >= 0) {
      const uint4* br = reinterpret_cast<const uint4*>(a.lb + ((size_t)id * a.N + n) * a.rank);
      const float4* hr = reinterpret_cast<const float4*>(a.h + (size_t)t * a.rank);
      float e = 0.f;
      for (int i = 0; i < a.rank / 8; ++i) {
        const uint4 b = __ldg(br + i);
        const float4 h0 = __ldcg(hr + 2 * i), h1 = __ldcg(hr + 2 * i + 1);
        e = fmaf(h0.x, bf16_lo(b.x), fmaf(h0.y, bf16_hi(b.x), e));
        e = fmaf(h0.z, bf16_lo(b.y), fmaf(h0.w, bf16_hi(b.y), e));
        e = fmaf(h1.x, bf16_lo(b.z), fmaf(h1.y, bf16_hi(b.z), e));
        e = fmaf(h1.z, bf16_lo(b.w), fmaf(h1.w, bf16_hi(b.w), e));
      }
      v += e;
    }
    if (a.x_scale) v *= __ldcg(a.x_scale + t);
    a.y[t * a.y_ld + n] = f32_to_bf16(v);
  }
}

// ---------------------------------------------------------------------------
// Larger batches, first launch. CTAs [0, nw): 8192 packed weights each, as
// fp16 in perm8 order. The others: 16 tokens each, x as fp16 rows in perm8
// order and, for every adapter among the 16 tokens, h on mma.sync (bf16, the
// 8 warps every 8th block of 32 K, their sums added in a fixed order). A
// lane's 16 bytes of x are at once what it converts and its fragment: the K
// order inside a block of 32 is the same for x and A, so it need not be the
// MMA's.
// ---------------------------------------------------------------------------
constexpr int kPrepWords = 1024;   // packed words per weight CTA

__global__ void __launch_bounds__(256) linear_prep_kernel(const LinearArgs a, uint16_t* __restrict__ x16,
                                                          uint16_t* __restrict__ w16, int nw,
                                                          const DevErr err) {
  __shared__ float red[8][16][33];
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if ((int)blockIdx.x < nw) {
    const long long words = (long long)a.N * (a.K / 8);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPrepWords / 256; ++i) {
      const long long wi = (long long)blockIdx.x * kPrepWords + 256 * i + tid;
      if (wi < words) {
        const uint32_t s = __ldg(a.w.s + (wi >> 3)), b = __ldg(a.w.b + (wi >> 3));
        bad |= sb_out_of_range(s, b);
        uint32_t o[4];
        dequant_word_f16_perm8(__ldg(a.w.q + wi), __half2half2(__float2half_rn(bf16_to_f32((uint16_t)s))),
                               __half2half2(__float2half_rn(bf16_to_f32((uint16_t)b))), o);
        reinterpret_cast<uint4*>(w16)[wi] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    report_range_warp(err, bad);
    return;
  }
  const int t0 = ((int)blockIdx.x - nw) * 16;
  uint32_t over = 0u;
  const int my_id = adapter_of(a, t0 + (lane & 15));
  unsigned todo = __ballot_sync(0xffffffffu, lane < 16 && my_id >= 0);
  const int g = lane >> 2, q = lane & 3;
  const int ta = t0 + g, tb = t0 + g + 8;
  bool convert = true;
  do {
    const int cur = todo ? __shfl_sync(0xffffffffu, my_id, __ffs(todo) - 1) : -1;
    const unsigned mine = __ballot_sync(0xffffffffu, lane < 16 && my_id == cur);
    todo &= ~mine;
    for (int rc = 0; rc == 0 || (cur >= 0 && rc < a.rank); rc += 32) {
      float acc[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 2
      for (int kb = 32 * warp; kb < a.K; kb += 256) {
        const int k = kb + 8 * q;
        Raw8 va{make_uint4(0u, 0u, 0u, 0u)}, vb{make_uint4(0u, 0u, 0u, 0u)};
        if (ta < a.T) va = load8(a, ta, k);
        if (tb < a.T) vb = load8(a, tb, k);
        if (convert) {
          if (ta < a.T)
            *reinterpret_cast<uint4*>(x16 + (size_t)ta * a.K + k) = f16x8_to_perm8(to_f16(a, va, over));
          if (tb < a.T)
            *reinterpret_cast<uint4*>(x16 + (size_t)tb * a.K + k) = f16x8_to_perm8(to_f16(a, vb, over));
        }
        if (cur >= 0) {
          const uint4 xa = to_bf16(a, va), xb = to_bf16(a, vb);
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            const int r = rc + 8 * nt;
            if (r < a.rank) {
              const uint4 w = __ldg(reinterpret_cast<const uint4*>(
                  a.la + ((size_t)cur * a.rank + r + g) * a.K + k));
              mma_bf16(acc[nt], xa.x, xb.x, xa.y, xb.y, w.x, w.y);
              mma_bf16(acc[nt], xa.z, xb.z, xa.w, xb.w, w.z, w.w);
            }
          }
        }
      }
      convert = false;
      if (cur < 0) break;
      __syncthreads();   // the last block's sums have been read
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) red[warp][g + 8 * (j >> 1)][8 * nt + 2 * q + (j & 1)] = acc[nt][j];
      __syncthreads();
      const float sc = a.lscale ? __ldg(a.lscale + cur) : 1.f;
      for (int o = tid; o < 16 * 32; o += 256) {
        const int t = o >> 5, r = o & 31;
        if (((mine >> t) & 1u) && rc + r < a.rank) {
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < 8; ++w) v += red[w][t][r];
          a.h[(size_t)(t0 + t) * a.rank + rc + r] = v * sc;
        }
      }
    }
  } while (todo);
  report_range_warp(err, over != 0u);
}

}  // namespace

cudaError_t launch_lora_shrink(const LinearArgs& a, cudaStream_t st) {
  return launch_pdl(lora_shrink_kernel, dim3((a.T * a.rank + 7) / 8), dim3(256), 0, st, a);
}

cudaError_t launch_linear_small(const LinearArgs& a, DevErr err, cudaStream_t st) {
  const int nt = (a.T + 7) / 8;
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3((a.N + kSmRows - 1) / kSmRows), dim3(256), 0, st, a, err);
  };
  return nt <= 1 ? go(linear_small_kernel<1>)
         : nt <= 2 ? go(linear_small_kernel<2>)
         : nt <= 4 ? go(linear_small_kernel<4>)
                   : go(linear_small_kernel<8>);
}

cudaError_t launch_linear_prep(const LinearArgs& a, uint16_t* x16, uint16_t* w16, DevErr err,
                               cudaStream_t st) {
  const long long words = (long long)a.N * (a.K / 8);
  const int nw = (int)((words + kPrepWords - 1) / kPrepWords);
  return launch_pdl(linear_prep_kernel, dim3(nw + (a.T + 15) / 16), dim3(256), 0, st, a, x16, w16, nw, err);
}

}  // namespace moe
