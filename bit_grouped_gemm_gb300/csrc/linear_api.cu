// linear_api.cu -- the C ABI of the 4-bit projection with adapters
// (moe_linear_*): handle and scratch, host-side argument checks, launches.
#include <new>

#include "moe_internal.h"

using namespace moe;

namespace {

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

struct Layout {
  size_t err, h, x16, w16, order, total;
};

constexpr int kWidths = 8;   // tile widths of the large product: 32, 64, .. 256

Layout make_layout(const moe_linear_desc& d) {
  Layout L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t r = o;
    o = align256(o + bytes);
    return r;
  };
  L.err = take(16);
  L.h = take((size_t)d.max_tokens * d.max_rank * 4);
  if (d.max_tokens > kLinearSmallT) {
    L.x16 = take((size_t)d.max_tokens * d.in_features * 2);
    L.w16 = take((size_t)d.out_features * d.in_features * 2);
    L.order = take((size_t)d.max_tokens * 4);
  } else {
    L.x16 = L.w16 = L.order = 0;
  }
  L.total = o;
  return L;
}

moe_status check_desc(const moe_linear_desc* d) {
  if (!d) return MOE_ERR_INVALID_ARG;
  if (d->in_features <= 0 || d->out_features <= 0 || d->max_tokens <= 0 || d->max_rank < 0 ||
      d->wait_limit_ms < 0)
    return MOE_ERR_INVALID_ARG;
  if (d->in_features % kGroup || d->max_rank % 8) return MOE_ERR_INVALID_ARG;
  if (d->in_features > 16384 || d->out_features > (1 << 20) || d->max_rank > 128 ||
      d->max_tokens > (1 << 20))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uint8_t *x = static_cast<const uint8_t*>(a), *y = static_cast<const uint8_t*>(b);
  return a && b && x < y + bn && y < x + an;
}

}  // namespace

struct moe_linear {
  moe_linear_desc d;
  int device = 0;
  int num_sms = 0;
  Layout L;
  uint8_t* scratch = nullptr;
  CUtensorMap mx, mw[kWidths];   // x16, and w16 by tile width

  DevErr err() const {
    DevErr e;
    e.word = reinterpret_cast<int*>(scratch + L.err);
    e.where = e.word + 1;
    e.limit_ns = (unsigned long long)(d.wait_limit_ms > 0 ? d.wait_limit_ms : 1000) * 1000000ull;
    return e;
  }
  template <class T>
  T* at(size_t off) const {
    return reinterpret_cast<T*>(scratch + off);
  }
  bool encode() {
    if (d.max_tokens <= kLinearSmallT) return true;
    bool ok = encode_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, at<uint16_t>(L.x16), d.max_tokens,
                        d.in_features, 64, 128);
    for (int i = 0; i < kWidths && ok; ++i)
      ok = encode_2d(&mw[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, at<uint16_t>(L.w16),
                     d.out_features, d.in_features, 64, 16 * (i + 1));
    return ok;
  }
};

extern "C" {

moe_status moe_linear_scratch_bytes(const moe_linear_desc* desc, size_t* bytes) {
  const moe_status s = check_desc(desc);
  if (s != MOE_OK) return s;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = make_layout(*desc).total;
  return MOE_OK;
}

moe_status moe_linear_create(const moe_linear_desc* desc, int device, moe_linear_t* out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  const moe_status s = check_desc(desc);
  if (s != MOE_OK) return s;
  if (device < 0) return MOE_ERR_INVALID_ARG;
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess || device >= ndev) return MOE_ERR_CUDA;
  int prev = 0;
  cudaGetDevice(&prev);
  if (cudaSetDevice(device) != cudaSuccess) return MOE_ERR_CUDA;
  moe_status res = MOE_OK;
  moe_linear* p = nullptr;
  cudaDeviceProp prop;
  if (cudaGetDeviceProperties(&prop, device) != cudaSuccess) {
    res = MOE_ERR_CUDA;
  } else if (prop.major != 10 || prop.minor != 3) {   // kernels are built for sm_103a only
    res = MOE_ERR_UNSUPPORTED;
  } else if (!(p = new (std::nothrow) moe_linear())) {
    res = MOE_ERR_CUDA;
  } else {
    p->d = *desc;
    p->device = device;
    p->num_sms = prop.multiProcessorCount;
    p->L = make_layout(*desc);
    if (cudaMalloc(&p->scratch, p->L.total) != cudaSuccess) {
      res = MOE_ERR_CUDA;
    } else if (!p->encode() || cudaMemset(p->scratch + p->L.err, 0, 16) != cudaSuccess ||
               cudaDeviceSynchronize() != cudaSuccess) {
      cudaFree(p->scratch);
      res = MOE_ERR_CUDA;
    }
    if (res != MOE_OK) {
      delete p;
      p = nullptr;
    }
  }
  cudaSetDevice(prev);
  *out = p;
  return res;
}

moe_status moe_linear_destroy(moe_linear_t p) {
  if (!p) return MOE_ERR_INVALID_ARG;
  int prev = 0;
  cudaGetDevice(&prev);
  cudaSetDevice(p->device);
  cudaDeviceSynchronize();
  cudaFree(p->scratch);
  cudaSetDevice(prev);
  delete p;
  return MOE_OK;
}

moe_status moe_linear_forward(moe_linear_t p, const void* x, int x_type, long long x_stride,
                              const float* x_scale, int T, const moe_w4* w, const moe_lora* lora,
                              const int32_t* adapter, uint16_t* y, long long y_stride,
                              moe_stream_t stream) {
  if (!p || !x || !w || !y || T < 1) return MOE_ERR_INVALID_ARG;
  const int K = p->d.in_features, N = p->d.out_features;
  if (T > p->d.max_tokens) return MOE_ERR_CAPACITY;
  if (x_type != MOE_X_BF16 && x_type != MOE_X_E4M3) return MOE_ERR_INVALID_ARG;
  if (x_type == MOE_X_BF16 && x_scale) return MOE_ERR_INVALID_ARG;
  if ((lora == nullptr) != (adapter == nullptr)) return MOE_ERR_INVALID_ARG;
  const long long x_ld = x_stride ? x_stride : K, y_ld = y_stride ? y_stride : N;
  if (x_ld < K || x_ld % 16 || y_ld < N) return MOE_ERR_INVALID_ARG;
  if (!w->qweight || !w->scales || !w->biases) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(x_scale, 16) || !aligned(w->qweight, 16) ||
      !aligned(w->scales, 16) || !aligned(w->biases, 16) || !aligned(y, 4) || !aligned(adapter, 4))
    return MOE_ERR_INVALID_ARG;
  const size_t kg = K / kGroup, xe = x_type == MOE_X_E4M3 ? 1 : 2;
  const size_t yb = ((size_t)(T - 1) * y_ld + N) * 2;
  if (overlap(y, yb, x, ((size_t)(T - 1) * x_ld + K) * xe) || overlap(y, yb, x_scale, (size_t)T * 4) ||
      overlap(y, yb, w->qweight, (size_t)N * K / 2) || overlap(y, yb, w->scales, N * kg * 2) ||
      overlap(y, yb, w->biases, N * kg * 2) || overlap(y, yb, adapter, (size_t)T * 4))
    return MOE_ERR_INVALID_ARG;
  if (lora) {
    if (!lora->a || !lora->b || lora->n < 1 || lora->rank < 8 || lora->rank % 8)
      return MOE_ERR_INVALID_ARG;
    if (!aligned(lora->a, 16) || !aligned(lora->b, 16) || !aligned(lora->scale, 4))
      return MOE_ERR_INVALID_ARG;
    if (lora->rank > p->d.max_rank) return MOE_ERR_CAPACITY;
    if (lora->n > 65536) return MOE_ERR_UNSUPPORTED;
    if (overlap(y, yb, lora->a, (size_t)lora->n * lora->rank * K * 2) ||
        overlap(y, yb, lora->b, (size_t)lora->n * lora->rank * N * 2) ||
        overlap(y, yb, lora->scale, (size_t)lora->n * 4))
      return MOE_ERR_INVALID_ARG;
  }
  LinearArgs a{};
  a.T = T;
  a.K = K;
  a.N = N;
  a.x = x;
  a.e4m3 = x_type == MOE_X_E4M3;
  a.x_ld = x_ld;
  a.x_scale = x_scale;
  a.w = W4Dev{w->qweight, w->scales, w->biases};
  a.y = y;
  a.y_ld = y_ld;
  if (lora) {
    a.la = lora->a;
    a.lb = lora->b;
    a.lscale = lora->scale;
    a.n_adapters = lora->n;
    a.rank = lora->rank;
    a.adapter = adapter;
    a.h = p->at<float>(p->L.h);
    a.order = p->at<int>(p->L.order);
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (linear_is_small(a, p->num_sms)) {
    e = launch_linear_small(a, p->err(), p->num_sms, st);
  } else {
    e = launch_linear_prep(a, p->at<uint16_t>(p->L.x16), p->at<uint16_t>(p->L.w16), p->err(),
                           p->num_sms, st);
    if (e == cudaSuccess) e = launch_linear_tc(a, p->mx, p->mw, p->err(), p->num_sms, st);
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_linear_get_error(moe_linear_t p) {
  if (!p) return MOE_ERR_INVALID_ARG;
  int h[2] = {0, 0};
  int* word = reinterpret_cast<int*>(p->scratch + p->L.err);
  int prev = 0;
  cudaGetDevice(&prev);
  cudaSetDevice(p->device);
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(h, word, sizeof h, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(word, 0, sizeof h);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  cudaSetDevice(prev);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  if (h[0] & DEVERR_TIMEOUT_BIT) return MOE_ERR_DEVICE_TIMEOUT;
  if (h[0] & DEVERR_RANGE_BIT) return MOE_ERR_OPERAND_RANGE;
  return MOE_OK;
}

}  // extern "C"
