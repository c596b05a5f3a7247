// norm_quant.cu -- residual addition, RMS norm and 8-bit output in one pass
// over a row (moe_norm_quant).
//
//   x' = bf16(x + alpha d);  v = x' w / sqrt(mean x'^2 + eps)
//   xn = bf16(v);  q = e4m3(v 448 / max|v|), scale = max|v| / 448
//
// Bound by memory: every input is read once and every output written once, a
// row staying in the registers of its threads in between. Both row statistics
// come from one reduction: the mean of squares needs x', and max|v| is
// max|x' w| times the row's factor (rounding is monotone, so this is the largest
// |v| to the bit). CTAs walk the rows and load the next one before they reduce
// and store the last. 16384 rows of 4096 with a bf16 delta and group scales, 606
// MB: 105 us a call (5.8 TB/s); 4096 rows of 2048 with an fp32 delta, 92 MB: 16.0;
// one row 1.7 us in a graph.
#include "moe_common.cuh"

namespace moe {
namespace {

struct NqParams {
  const uint16_t* x;
  const void* d;
  const uint16_t* w;
  uint16_t* xo;
  uint16_t* xn;
  uint8_t* q;
  float* qs;
  long long x_ld, d_ld, o_ld;
  unsigned T;               // (a step past the last row then does not wrap)
  int H, group;             // group: 0 the row, 128
  float eps, alpha;
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void unpack8(const uint4& a, float (&v)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = bf16_lo(w[j]);
    v[2 * j + 1] = bf16_hi(w[j]);
  }
}

// NaN-keeping maximum of magnitudes
__device__ __forceinline__ float nan_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// TPR threads per row (a power of two from 16), each with NV vectors of 8
// columns, vector c = lane-in-row + TPR i; kD: delta 0 none, 1 bf16, 2 f32.
// Several rows share a CTA of 256 threads where TPR is less.
constexpr int cta_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

template <int TPR, int NV, int kD>
__global__ void __launch_bounds__(cta_threads(TPR)) norm_quant_kernel(const NqParams p) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR, kRows = kThreads / TPR, kWarps = TPR / 32;
  pdl_begin();
  __shared__ float2 s_red[2][kThreads / 32];
  const int sub = threadIdx.x / TPR, tid = threadIdx.x % TPR, lane = threadIdx.x & 31;
  const int nvec = p.H / 8;
  const int ngroups = p.group ? (p.H + p.group - 1) / p.group : 1;
  uint4 xr[NV], dr[NV * (kD == 2 ? 2 : 1)];
  auto load = [&](unsigned t) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + TPR * i;
      if (t < p.T && c < nvec) {
        xr[i] = *reinterpret_cast<const uint4*>(p.x + t * p.x_ld + 8 * c);
        if constexpr (kD == 1)
          dr[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.d) + t * p.d_ld + 8 * c);
        if constexpr (kD == 2) {
          const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p.d) + t * p.d_ld + 8 * c);
          dr[2 * i] = q[0];
          dr[2 * i + 1] = q[1];
        }
      }
    }
  };
  unsigned t = blockIdx.x * kRows + sub;
  load(t);
  // (the trip count is the CTA's, not the row's: every thread meets the barrier)
  int buf = 0;
  for (unsigned t0 = blockIdx.x * kRows; t0 < p.T; t0 += gridDim.x * kRows, t += gridDim.x * kRows, buf ^= 1) {
    const bool row = t < p.T;
    float v[NV][8];
    float ss = 0.f, mx = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + TPR * i;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
      if (!row || c >= nvec) continue;
      unpack8(xr[i], v[i]);
      if constexpr (kD != 0) {
        float d[8];
        if constexpr (kD == 1) {
          unpack8(dr[i], d);
        } else {
          const uint4 q0 = dr[2 * i], q1 = dr[2 * i + 1];
          const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] = __uint_as_float(w[j]);
        }
        uint4 o;
        uint32_t* ow = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          ow[j] = pack_bf16x2(fmaf(p.alpha, d[2 * j], v[i][2 * j]), fmaf(p.alpha, d[2 * j + 1], v[i][2 * j + 1]));
        unpack8(o, v[i]);
        if (p.xo) *reinterpret_cast<uint4*>(p.xo + t * p.x_ld + 8 * c) = o;
      } else if (p.xo && p.xo != p.x) {
        *reinterpret_cast<uint4*>(p.xo + t * p.x_ld + 8 * c) = xr[i];
      }
      float w[8];
      if (p.w) unpack8(__ldg(reinterpret_cast<const uint4*>(p.w + 8 * c)), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(v[i][j], v[i][j], ss);
        if (p.w) v[i][j] *= w[j];
        mx = nan_max(mx, fabsf(v[i][j]));
      }
    }
    load(t + gridDim.x * kRows);
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      mx = nan_max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    if constexpr (TPR > 32) {
      if (lane == 0) s_red[buf][threadIdx.x >> 5] = make_float2(ss, mx);
      __syncthreads();   // (the other buffer is free again after the next one)
      ss = mx = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float2 r = s_red[buf][sub * kWarps + i];
        ss += r.x;
        mx = nan_max(mx, r.y);
      }
    }
    const float inv = 1.0f / sqrtf(ss / (float)p.H + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + TPR * i;
      const bool on = row && c < nvec;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= inv;
      if (p.xn && on) {
        uint4 o;
        o.x = pack_bf16x2(v[i][0], v[i][1]);
        o.y = pack_bf16x2(v[i][2], v[i][3]);
        o.z = pack_bf16x2(v[i][4], v[i][5]);
        o.w = pack_bf16x2(v[i][6], v[i][7]);
        *reinterpret_cast<uint4*>(p.xn + t * p.o_ld + 8 * c) = o;
      }
      if (!p.q) continue;
      float am = mx * inv;
      if (p.group) {   // 128 columns: 16 neighbouring lanes
        am = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) am = nan_max(am, fabsf(v[i][j]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) am = nan_max(am, __shfl_xor_sync(0xffffffffu, am, o));
      }
      const bool none = am < 0x1p-100f;
      const float qk = none ? 0.f : 448.0f / am;
      if (on) {
        uint2 o;
        o.x = e4m3x2(v[i][0] * qk, v[i][1] * qk) | (e4m3x2(v[i][2] * qk, v[i][3] * qk) << 16);
        o.y = e4m3x2(v[i][4] * qk, v[i][5] * qk) | (e4m3x2(v[i][6] * qk, v[i][7] * qk) << 16);
        *reinterpret_cast<uint2*>(p.q + t * p.o_ld + 8 * c) = o;
        if (p.group ? (c & 15) == 0 : c == 0)
          p.qs[(size_t)t * ngroups + (p.group ? c / 16 : 0)] = none ? 0.f : am / 448.0f;
      }
    }
  }
}

template <int TPR, int NV, int kD>
cudaError_t launch_nq(const NqParams& p, cudaStream_t st) {
  constexpr int kRows = cta_threads(TPR) / TPR;
  const int ctas = (int)((p.T + kRows - 1) / kRows);
  static int resident[64] = {};   // CTAs the device holds at once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int cap = dev < 64 ? resident[dev] : 0;
  if (!cap) {
    int sms = 0, per = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, norm_quant_kernel<TPR, NV, kD>, cta_threads(TPR), 0);
    if (e != cudaSuccess) return e;
    cap = sms * per;
    if (dev < 64) resident[dev] = cap;
  }
  return launch_pdl(norm_quant_kernel<TPR, NV, kD>, dim3(ctas < cap ? ctas : cap), dim3(cta_threads(TPR)), 0, st, p);
}

// Threads per row by its width, so that a thread holds one vector, two from
// 2,056 columns on.
template <int kD>
cudaError_t launch_width(const NqParams& p, cudaStream_t st) {
  const int nvec = p.H / 8;
  return nvec <= 16     ? launch_nq<16, 1, kD>(p, st)
         : nvec <= 32   ? launch_nq<32, 1, kD>(p, st)
         : nvec <= 64   ? launch_nq<64, 1, kD>(p, st)
         : nvec <= 128  ? launch_nq<128, 1, kD>(p, st)
         : nvec <= 256  ? launch_nq<256, 1, kD>(p, st)
         : nvec <= 512  ? launch_nq<256, 2, kD>(p, st)
         : nvec <= 1024 ? launch_nq<512, 2, kD>(p, st)
                        : launch_nq<1024, 2, kD>(p, st);
}

bool al16(const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; }

struct Span {   // bytes [lo, hi) that T rows of a tensor touch
  uintptr_t lo, hi;
};
Span span_of(const void* p, int T, long long ld, int H, int elem) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (!p) return {0, 0};
  return {a, a + ((size_t)(T - 1) * ld + H) * elem};
}
bool overlap(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

}  // namespace
}  // namespace moe

extern "C" moe_status moe_norm_quant(const moe_norm_desc* d, const uint16_t* x, const void* delta,
                                     const uint16_t* weight, int T, uint16_t* x_out,
                                     uint16_t* xn_out, uint8_t* q_out, float* q_scale,
                                     moe_stream_t stream) {
  using namespace moe;
  if (!d || !x || T < 1) return MOE_ERR_INVALID_ARG;
  const int H = d->hidden;
  if (H < 8 || H % 8) return MOE_ERR_INVALID_ARG;
  if (H > 16384) return MOE_ERR_UNSUPPORTED;
  if (!(d->eps >= 0.f) || d->eps > 3e38f || !(d->alpha > -3e38f && d->alpha < 3e38f))
    return MOE_ERR_INVALID_ARG;
  if ((d->delta_f32 != 0 && d->delta_f32 != 1) || (d->quant_group != 0 && d->quant_group != 128))
    return MOE_ERR_INVALID_ARG;
  NqParams p;
  p.x_ld = d->x_stride ? d->x_stride : H;
  p.d_ld = d->delta_stride ? d->delta_stride : H;
  p.o_ld = d->out_stride ? d->out_stride : H;
  for (long long ld : {p.x_ld, p.d_ld, p.o_ld})
    if (ld < H || ld % 8) return MOE_ERR_INVALID_ARG;
  if (!x_out && !xn_out && !q_out) return MOE_ERR_INVALID_ARG;
  if ((q_out == nullptr) != (q_scale == nullptr)) return MOE_ERR_INVALID_ARG;
  for (const void* q : {(const void*)x, delta, (const void*)weight, (const void*)x_out,
                        (const void*)xn_out, (const void*)q_out, (const void*)q_scale})
    if (!al16(q)) return MOE_ERR_INVALID_ARG;
  const int ng = d->quant_group ? (H + 127) / 128 : 1;
  const Span in[3] = {span_of(x, T, p.x_ld, H, 2), span_of(delta, T, p.d_ld, H, d->delta_f32 ? 4 : 2),
                      span_of(weight, 1, H, H, 2)};
  const Span out[4] = {span_of(x_out, T, p.x_ld, H, 2), span_of(xn_out, T, p.o_ld, H, 2),
                       span_of(q_out, T, p.o_ld, H, 1), span_of(q_scale, T, ng, ng, 4)};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 3; ++j)
      if (overlap(out[i], in[j]) && !(i == 0 && j == 0 && x_out == x)) return MOE_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return MOE_ERR_INVALID_ARG;
  }
  p.x = x;
  p.d = delta;
  p.w = weight;
  p.xo = x_out;
  p.xn = xn_out;
  p.q = q_out;
  p.qs = q_scale;
  p.T = (unsigned)T;
  p.H = H;
  p.group = d->quant_group;
  p.eps = d->eps;
  p.alpha = d->alpha;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = !delta ? launch_width<0>(p, st)
                        : d->delta_f32 ? launch_width<2>(p, st)
                                       : launch_width<1>(p, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
