// w4_linear.cu -- 4-bit projection with the low-rank adapters of many requests
// at once (moe_linear_forward):
//   y[t] = x_scale[t] (x[t] W^T + scale[a] (x[t] A[a]^T) B[a]^T),  a = adapter[t]
// W is 4-bit affine in groups of 64 along K (moe_w4).
#include <cuda_fp8.h>

#include "moe_common.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float x_at(const LinearArgs& a, int t, int k) {
  if (a.e4m3) {
    __nv_fp8_e4m3 v;
    v.__x = static_cast<const uint8_t*>(a.x)[t * a.x_ld + k];
    return float(v);
  }
  return bf16_to_f32(static_cast<const uint16_t*>(a.x)[t * a.x_ld + k]);
}

// The adapter of token t, or -1.
__device__ __forceinline__ int adapter_of(const LinearArgs& a, int t) {
  if (!a.la) return -1;
  const int id = a.adapter[t];
  return (unsigned)id < (unsigned)a.n_adapters ? id : -1;
}

// h[t][r] = scale[a] * sum_k x[t][k] A[a][r][k]: one warp per (t, r).
__global__ void __launch_bounds__(256) lora_shrink_kernel(const LinearArgs a) {
  pdl_begin();
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w >= (long long)a.T * a.rank) return;
  const int t = (int)(w / a.rank), r = (int)(w % a.rank);
  const int id = adapter_of(a, t);
  float s = 0.f;
  if (id >= 0) {
    const uint16_t* ar = a.la + ((size_t)id * a.rank + r) * a.K;
    for (int k = lane; k < a.K; k += 32) s = fmaf(x_at(a, t, k), bf16_to_f32(ar[k]), s);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) a.h[w] = id >= 0 ? s * (a.lscale ? a.lscale[id] : 1.f) : 0.f;
}

// 16 tokens x 64 weight rows per CTA, K in groups of 64, FP32 throughout.
__global__ void __launch_bounds__(256) linear_simple_kernel(const LinearArgs a) {
  pdl_begin();
  __shared__ float ws[64][65], xs[16][65];
  const int tid = threadIdx.x, n0 = blockIdx.x * 64, t0 = blockIdx.y * 16;
  const int n = tid & 63, tq = tid >> 6;
  const int kg = a.K / 64;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int g = 0; g < kg; ++g) {
    for (int i = tid; i < 64 * 8; i += 256) {
      const int r = i >> 3, wd = i & 7;
      uint32_t q = 0u;
      float s = 0.f, b = 0.f;
      if (n0 + r < a.N) {
        q = a.w.q[(size_t)(n0 + r) * (a.K / 8) + 8 * g + wd];
        s = bf16_to_f32(a.w.s[(size_t)(n0 + r) * kg + g]);
        b = bf16_to_f32(a.w.b[(size_t)(n0 + r) * kg + g]);
      }
      for (int j = 0; j < 8; ++j) ws[r][8 * wd + j] = fmaf((float)((q >> (4 * j)) & 15u), s, b);
    }
    for (int i = tid; i < 16 * 64; i += 256) {
      const int t = t0 + (i >> 6);
      xs[i >> 6][i & 63] = t < a.T ? x_at(a, t, 64 * g + (i & 63)) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < 64; ++k) {
      const float w = ws[n][k];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(xs[tq + 4 * i][k], w, acc[i]);
    }
    __syncthreads();
  }
  if (n0 + n >= a.N) return;
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + tq + 4 * i;
    if (t >= a.T) continue;
    const int id = adapter_of(a, t);
    float v = acc[i];
    if (id >= 0) {
      const uint16_t* br = a.lb + ((size_t)id * a.N + n0 + n) * a.rank;
      for (int r = 0; r < a.rank; ++r) v = fmaf(a.h[(size_t)t * a.rank + r], bf16_to_f32(br[r]), v);
    }
    if (a.x_scale) v *= a.x_scale[t];
    a.y[t * a.y_ld + n0 + n] = f32_to_bf16(v);
  }
}

}  // namespace

cudaError_t launch_lora_shrink(const LinearArgs& a, cudaStream_t st) {
  const long long warps = (long long)a.T * a.rank;
  return launch_pdl(lora_shrink_kernel, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, st, a);
}

cudaError_t launch_linear_simple(const LinearArgs& a, cudaStream_t st) {
  return launch_pdl(linear_simple_kernel, dim3((a.N + 63) / 64, (a.T + 15) / 16), dim3(256), 0, st, a);
}

}  // namespace moe
