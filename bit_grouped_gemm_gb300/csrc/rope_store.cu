// rope_store.cu -- rotary positions of queries and keys, and the store of keys
// and values into a paged cache in bf16 or e4m3 (moe_rope_store).
//
//   (a, b) -> gain (a cos x - b sin x, b cos x + a sin x),  x = 2 pi pos f_i
//
// The angle is kept in turns as a 64-bit fixed-point fraction: pos times the
// frequency's fraction, modulo 2^64, is the fraction of a turn for every int32
// position; its top 32 bits go to sincospi. The fractions come from doubles, right to
// 2^-55 turns per position: 2^-35 at position 10^6, 2^-24 at the ends of int32; the
// argument's rounding to FP32 is up to 2^-26. A float product pos * f would lose the
// angle of far positions (0.06 rad at position 10^6).
//
// Bound by memory: every row is read once and written once. A thread takes 16
// elements of a head (8 pairs where they turn) and up to 4 heads of the same
// token, so one set of 8 sines and cosines serves 4 heads and 8 loads are in
// flight. Measured (in a graph; 16,384 tokens, 16 + 2 heads of 128): bf16 29.0 us (5.8
// TB/s), e4m3 32.5 (4.9); 4096 tokens of 8 + 8 heads 9.9 and 13.5: an e4m3 element is
// divided by its scale, rounded as the definition's, where memory leaves little time.
#include "attn.h"
#include "moe_common.cuh"

namespace moe {
namespace {

constexpr int kRopeThreads = 128, kRopeHeads = 4;

__device__ __forceinline__ void unpack8(const uint4& a, float (&v)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = bf16_lo(w[j]);
    v[2 * j + 1] = bf16_hi(w[j]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// Saturates, keeps a NaN. The quotient is rounded as the definition's.
__device__ __forceinline__ uint32_t e4m3x2_over(float lo, float hi, float s) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(__fdiv_rn(hi, s)), "f"(__fdiv_rn(lo, s)));
  return r;
}

__device__ __forceinline__ uint2 quant8(const float (&v)[8], float s) {
  return make_uint2(e4m3x2_over(v[0], v[1], s) | e4m3x2_over(v[2], v[3], s) << 16,
                    e4m3x2_over(v[4], v[5], s) | e4m3x2_over(v[6], v[7], s) << 16);
}

template <bool kInter, bool kE4m3>
__global__ void __launch_bounds__(kRopeThreads) rope_store_kernel(const RopeArgs p, int dim_shift,
                                                                  int groups) {
  pdl_begin();
  // 16-element units of a head, then groups of heads, then tokens
  const long long id = (long long)blockIdx.x * kRopeThreads + threadIdx.x;
  const int u = (int)id & ((1 << dim_shift) - 1);
  const long long rest = id >> dim_shift;
  const int t = (int)(rest / groups), g = (int)(rest - (long long)t * groups);
  if (t >= p.T) return;
  const int D = p.head_dim, half = p.rotary_dim / 2, Hr = p.heads + p.kv_heads;
  const bool turns = 8 * u < half;
  // offsets of the unit's two vectors of 8 in a head
  const int c0 = !kInter && turns ? 8 * u : 16 * u, c1 = !kInter && turns ? c0 + half : c0 + 8;
  uint4 x[kRopeHeads][2];
#pragma unroll
  for (int i = 0; i < kRopeHeads; ++i) {
    const int h = g + groups * i;
    if (h >= Hr + p.kv_heads) continue;
    const uint16_t* src = h < p.heads ? p.q + t * p.q_ld + (long long)h * D
                          : h < Hr    ? p.k + t * p.k_ld + (long long)(h - p.heads) * D
                                      : p.v + t * p.v_ld + (long long)(h - Hr) * D;
    x[i][0] = *reinterpret_cast<const uint4*>(src + c0);
    x[i][1] = *reinterpret_cast<const uint4*>(src + c1);
  }
  const int slot = p.slot[t];
  float cs[8], sn[8];
  if (turns && g < Hr) {
    const unsigned long long pos = (unsigned long long)(long long)p.position[t];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int part = (int)((pos * __ldg(p.turns + 8 * u + j)) >> 32);   // of 2^32 a turn
      sincospif((float)part * 0x1p-31f, &sn[j], &cs[j]);
      sn[j] *= p.gain;
      cs[j] *= p.gain;
    }
  }
  const bool stored = slot >= 0 && (slot >> p.page_shift) < p.cache.pages;
#pragma unroll
  for (int i = 0; i < kRopeHeads; ++i) {
    const int h = g + groups * i;
    if (h >= Hr + p.kv_heads || (h >= p.heads && !stored)) continue;
    float a[8], b[8];
    unpack8(x[i][0], a);
    unpack8(x[i][1], b);
    if (turns && h < Hr) {
      if constexpr (kInter) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a0 = a[2 * j], a1 = a[2 * j + 1], b0 = b[2 * j], b1 = b[2 * j + 1];
          a[2 * j] = a0 * cs[j] - a1 * sn[j];
          a[2 * j + 1] = a1 * cs[j] + a0 * sn[j];
          b[2 * j] = b0 * cs[4 + j] - b1 * sn[4 + j];
          b[2 * j + 1] = b1 * cs[4 + j] + b0 * sn[4 + j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float a0 = a[j], b0 = b[j];
          a[j] = a0 * cs[j] - b0 * sn[j];
          b[j] = b0 * cs[j] + a0 * sn[j];
        }
      }
    }
    if (h < p.heads) {
      uint16_t* dst = p.q_out + t * p.o_ld + (long long)h * D;
      *reinterpret_cast<uint4*>(dst + c0) = pack8(a);
      *reinterpret_cast<uint4*>(dst + c1) = pack8(b);
      continue;
    }
    const bool key = h < Hr;
    const int kh = key ? h - p.heads : h - Hr;
    const long long row = ((((long long)(slot >> p.page_shift) * p.kv_heads + kh) << p.page_shift) +
                           (slot & ((1 << p.page_shift) - 1))) * D;
    if constexpr (kE4m3) {
      const float s = (key ? p.cache.k_scale : p.cache.v_scale)[kh];
      uint8_t* dst = static_cast<uint8_t*>(key ? p.cache.k : p.cache.v) + row;
      *reinterpret_cast<uint2*>(dst + c0) = quant8(a, s);
      *reinterpret_cast<uint2*>(dst + c1) = quant8(b, s);
    } else {
      uint16_t* dst = static_cast<uint16_t*>(key ? p.cache.k : p.cache.v) + row;
      *reinterpret_cast<uint4*>(dst + c0) = pack8(a);
      *reinterpret_cast<uint4*>(dst + c1) = pack8(b);
    }
  }
}

}  // namespace

cudaError_t launch_rope_store(const RopeArgs& a, cudaStream_t st) {
  int shift = 0;   // units of a head: 4, 8 or 16
  while ((16 << shift) < a.head_dim) ++shift;
  const int groups = (a.heads + 2 * a.kv_heads + kRopeHeads - 1) / kRopeHeads;
  const long long n = ((long long)a.T * groups) << shift;
  const dim3 grid((unsigned)((n + kRopeThreads - 1) / kRopeThreads));
  auto go = [&](auto kern) { return launch_pdl(kern, grid, dim3(kRopeThreads), 0, st, a, shift, groups); };
  if (a.interleaved) return a.e4m3 ? go(rope_store_kernel<true, true>) : go(rope_store_kernel<true, false>);
  return a.e4m3 ? go(rope_store_kernel<false, true>) : go(rope_store_kernel<false, false>);
}

}  // namespace moe
