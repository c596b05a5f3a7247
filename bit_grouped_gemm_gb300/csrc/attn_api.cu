// attn_api.cu -- the C ABI of attention over a paged cache (moe_attn_*,
// moe_rope_store, moe_tree_attention): handle, argument checks, launches.
#include <math.h>

#include <new>

#include "attn.h"
#include "spans.h"

using namespace moe;

namespace {

constexpr int kMaxHalf = 128;                       // frequencies of the widest head
constexpr size_t kErrBytes = 256, kTurnsBytes = kMaxHalf * 8;

int page_shift(int size) {
  for (int s = 4; s <= 8; ++s)
    if ((1 << s) == size) return s;
  return -1;
}

moe_status check_desc(const moe_attn_desc* d) {
  if (!d) return MOE_ERR_INVALID_ARG;
  if (d->heads < 1 || d->kv_heads < 1 || d->heads % d->kv_heads || d->head_dim < 1 ||
      d->page_size < 1 || d->max_tokens < 1 || d->max_requests < 1 || d->wait_limit_ms < 0)
    return MOE_ERR_INVALID_ARG;
  if (d->cache_type != MOE_CACHE_BF16 && d->cache_type != MOE_CACHE_E4M3) return MOE_ERR_INVALID_ARG;
  if (!(d->softmax_scale >= 0.0f) || !(d->softmax_scale < 1e30f)) return MOE_ERR_INVALID_ARG;
  if (d->rotary_dim < 0 || d->rotary_dim > d->head_dim || d->rotary_dim % 2) return MOE_ERR_INVALID_ARG;
  if (d->rope_layout != MOE_ROPE_HALF && d->rope_layout != MOE_ROPE_INTERLEAVED) return MOE_ERR_INVALID_ARG;
  if (d->rope_scaling < MOE_ROPE_PLAIN || d->rope_scaling > MOE_ROPE_BY_PARTS) return MOE_ERR_INVALID_ARG;
  if (!(fabsf(d->rope_gain) < 1e30f)) return MOE_ERR_INVALID_ARG;
  if (d->rotary_dim) {
    if (!(d->rope_theta >= 1.0) || !(d->rope_theta < 1e30)) return MOE_ERR_INVALID_ARG;
    if (d->rope_scaling != MOE_ROPE_PLAIN && (!(d->rope_factor >= 1.0) || !(d->rope_factor < 1e30)))
      return MOE_ERR_INVALID_ARG;
    if (d->rope_scaling == MOE_ROPE_BY_PARTS &&
        (!(d->rope_low < d->rope_high) || !(d->rope_low > -1e30) || !(d->rope_high < 1e30) ||
         d->rope_original < 1))
      return MOE_ERR_INVALID_ARG;
  }
  if ((d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) || page_shift(d->page_size) < 0 ||
      d->rotary_dim % 16 || d->kv_heads > 256 || d->heads / d->kv_heads > 128 ||
      d->max_tokens > (1 << 20) || d->max_requests > 4096)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t scratch_of(const moe_attn_desc& d) {
  return kErrBytes + kTurnsBytes + attn_scratch_bytes(d.head_dim);
}

// Turns per position of pair i, as a fraction of 2^64.
unsigned long long turns_of(const moe_attn_desc& d, int i) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  double f = pow(d.rope_theta, -2.0 * i / d.rotary_dim);
  if (d.rope_scaling == MOE_ROPE_LINEAR) f /= d.rope_factor;
  if (d.rope_scaling == MOE_ROPE_BY_PARTS) {
    const double r = d.rope_original * f / kTwoPi;
    const double g = fmin(fmax((r - d.rope_low) / (d.rope_high - d.rope_low), 0.0), 1.0);
    f *= g + (1.0 - g) / d.rope_factor;
  }
  return (unsigned long long)ldexp(f / kTwoPi, 64);   // f <= 1: below a turn
}

// The handle's device for the length of a call.
class OnDevice {
 public:
  explicit OnDevice(int dev) {
    ok_ = cudaGetDevice(&prev_) == cudaSuccess && (prev_ == dev || cudaSetDevice(dev) == cudaSuccess);
    moved_ = ok_ && prev_ != dev;
  }
  ~OnDevice() {
    if (moved_) cudaSetDevice(prev_);
  }
  bool ok() const { return ok_; }

 private:
  int prev_ = 0;
  bool ok_ = false, moved_ = false;
};

}  // namespace

struct moe_attn {
  moe_attn_desc d;
  int device = 0, num_sms = 0;
  uint8_t* scratch = nullptr;

  DevErr err() const {
    DevErr e;
    e.word = reinterpret_cast<int*>(scratch);
    e.where = e.word + 1;
    e.limit_ns = (unsigned long long)(d.wait_limit_ms > 0 ? d.wait_limit_ms : 1000) * 1000000ull;
    return e;
  }
  const unsigned long long* turns() const {
    return reinterpret_cast<const unsigned long long*>(scratch + kErrBytes);
  }
};

namespace {

// The cache's own fields, and its ranges (k, v, their scales).
moe_status check_cache(const moe_attn& p, const moe_kv_cache* c, Span (&s)[4]) {
  if (!c || !c->k || !c->v || c->pages < 1) return MOE_ERR_INVALID_ARG;
  const bool e4m3 = p.d.cache_type == MOE_CACHE_E4M3;
  if (e4m3 != (c->k_scale != nullptr) || e4m3 != (c->v_scale != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!is_aligned(c->k, 16) || !is_aligned(c->v, 16) || !is_aligned(c->k_scale, 4) ||
      !is_aligned(c->v_scale, 4))
    return MOE_ERR_INVALID_ARG;
  // slots are int32
  if (c->pages > 0x7fffffff / p.d.page_size) return MOE_ERR_UNSUPPORTED;
  const size_t bytes = (size_t)c->pages * p.d.kv_heads * p.d.page_size * p.d.head_dim * (e4m3 ? 1 : 2);
  const size_t scales = 4 * (size_t)p.d.kv_heads;
  s[0] = {c->k, bytes};
  s[1] = {c->v, bytes};
  s[2] = {c->k_scale, scales};
  s[3] = {c->v_scale, scales};
  return MOE_OK;
}

CacheDev dev_of(const moe_kv_cache& c) { return {c.k, c.v, c.k_scale, c.v_scale, c.pages}; }

// Row stride in elements: 0 dense, else at least `cols` and a multiple of 8.
bool stride_of(long long given, long long cols, long long* ld) {
  *ld = given ? given : cols;
  return *ld >= cols && *ld % 8 == 0 && *ld < (1ll << 31);
}

size_t rows_bytes(int T, long long ld, long long cols) { return ((size_t)(T - 1) * ld + cols) * 2; }

}  // namespace

extern "C" {

moe_status moe_attn_scratch_bytes(const moe_attn_desc* desc, size_t* bytes) {
  const moe_status s = check_desc(desc);
  if (s != MOE_OK) return s;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = scratch_of(*desc);
  return MOE_OK;
}

moe_status moe_attn_create(const moe_attn_desc* desc, int device, moe_attn_t* out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  const moe_status s = check_desc(desc);
  if (s != MOE_OK) return s;
  if (device < 0) return MOE_ERR_INVALID_ARG;
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess || device >= ndev) return MOE_ERR_CUDA;
  const OnDevice on(device);
  if (!on.ok()) return MOE_ERR_CUDA;
  cudaDeviceProp prop;
  if (cudaGetDeviceProperties(&prop, device) != cudaSuccess) return MOE_ERR_CUDA;
  if (prop.major != 10 || prop.minor != 3) return MOE_ERR_UNSUPPORTED;   // built for sm_103a only
  moe_attn* p = new (std::nothrow) moe_attn();
  if (!p) return MOE_ERR_CUDA;
  p->d = *desc;
  p->device = device;
  p->num_sms = prop.multiProcessorCount;
  unsigned long long turns[kMaxHalf] = {};
  for (int i = 0; i < desc->rotary_dim / 2; ++i) turns[i] = turns_of(*desc, i);
  const size_t bytes = scratch_of(*desc);
  if (cudaMalloc(&p->scratch, bytes) != cudaSuccess) {
    delete p;
    return MOE_ERR_CUDA;
  }
  if (cudaMemset(p->scratch, 0, bytes) != cudaSuccess ||
      cudaMemcpy(p->scratch + kErrBytes, turns, sizeof turns, cudaMemcpyHostToDevice) != cudaSuccess ||
      cudaDeviceSynchronize() != cudaSuccess) {
    cudaFree(p->scratch);
    delete p;
    return MOE_ERR_CUDA;
  }
  *out = p;
  return MOE_OK;
}

moe_status moe_attn_destroy(moe_attn_t p) {
  if (!p) return MOE_ERR_INVALID_ARG;
  const OnDevice on(p->device);
  cudaDeviceSynchronize();
  cudaFree(p->scratch);
  delete p;
  return MOE_OK;
}

moe_status moe_attn_get_error(moe_attn_t p) {
  if (!p) return MOE_ERR_INVALID_ARG;
  const OnDevice on(p->device);
  if (!on.ok()) return MOE_ERR_CUDA;
  int h[2] = {0, 0};
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(h, p->scratch, sizeof h, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(p->scratch, 0, sizeof h);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  if (h[0] & DEVERR_TIMEOUT_BIT) return MOE_ERR_DEVICE_TIMEOUT;
  if (h[0] & DEVERR_RANGE_BIT) return MOE_ERR_OPERAND_RANGE;
  return MOE_OK;
}

moe_status moe_rope_store(moe_attn_t p, const uint16_t* q, long long q_stride, const uint16_t* k,
                          long long k_stride, const uint16_t* v, long long v_stride, int T,
                          const int32_t* position, const int32_t* slot, uint16_t* q_out,
                          long long out_stride, const moe_kv_cache* cache, moe_stream_t stream) {
  if (!p || !q || !k || !v || !position || !slot || !q_out || T < 1) return MOE_ERR_INVALID_ARG;
  if (T > p->d.max_tokens) return MOE_ERR_CAPACITY;
  const long long qc = (long long)p->d.heads * p->d.head_dim, kc = (long long)p->d.kv_heads * p->d.head_dim;
  RopeArgs a{};
  if (!stride_of(q_stride, qc, &a.q_ld) || !stride_of(k_stride, kc, &a.k_ld) ||
      !stride_of(v_stride, kc, &a.v_ld) || !stride_of(out_stride, qc, &a.o_ld))
    return MOE_ERR_INVALID_ARG;
  if (!is_aligned(q, 16) || !is_aligned(k, 16) || !is_aligned(v, 16) || !is_aligned(q_out, 16) ||
      !is_aligned(position, 4) || !is_aligned(slot, 4))
    return MOE_ERR_INVALID_ARG;
  Span c[4];
  const moe_status s = check_cache(*p, cache, c);
  if (s != MOE_OK) return s;
  const Span in[] = {{q, rows_bytes(T, a.q_ld, qc)}, {k, rows_bytes(T, a.k_ld, kc)},
                     {v, rows_bytes(T, a.v_ld, kc)}, {position, 4 * (size_t)T},
                     {slot, 4 * (size_t)T},          c[2], c[3]};
  const Span out{q_out, rows_bytes(T, a.o_ld, qc)};
  const bool in_place = q_out == q && a.o_ld == a.q_ld;
  for (int i = 0; i < 7; ++i) {
    const Span& x = in[i];
    // in place, q's rows may lie between those of k and v: the parts of one
    // projection's rows, which the rows' own columns keep apart
    const bool fused = in_place && ((i == 1 && a.k_ld == a.q_ld) || (i == 2 && a.v_ld == a.q_ld));
    if (!(in_place && i == 0) && !fused && clash(out, x)) return MOE_ERR_INVALID_ARG;
    if (fused) {
      const long long d = (const uint16_t*)x.p - q, r = ((d % a.q_ld) + a.q_ld) % a.q_ld;
      if (clash(out, x) && !(r >= qc && r + kc <= a.q_ld)) return MOE_ERR_INVALID_ARG;
    }
    if (clash(c[0], x) || clash(c[1], x)) return MOE_ERR_INVALID_ARG;
  }
  if (clash(out, c[0]) || clash(out, c[1]) || clash(c[0], c[1])) return MOE_ERR_INVALID_ARG;
  const OnDevice on(p->device);
  if (!on.ok()) return MOE_ERR_CUDA;
  a.T = T;
  a.heads = p->d.heads;
  a.kv_heads = p->d.kv_heads;
  a.head_dim = p->d.head_dim;
  a.rotary_dim = p->d.rotary_dim;
  a.interleaved = p->d.rope_layout == MOE_ROPE_INTERLEAVED;
  a.e4m3 = p->d.cache_type == MOE_CACHE_E4M3;
  a.page_shift = page_shift(p->d.page_size);
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.position = position;
  a.slot = slot;
  a.turns = p->turns();
  a.gain = p->d.rope_gain != 0.0f ? p->d.rope_gain : 1.0f;
  a.cache = dev_of(*cache);
  return launch_rope_store(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_tree_attention(moe_attn_t p, const uint16_t* q, long long q_stride, int T,
                              const moe_kv_cache* cache, const int32_t* table, int table_width,
                              int requests, const int32_t* offsets, const int32_t* length,
                              const uint64_t* mask, int mask_words, uint16_t* out,
                              long long out_stride, moe_stream_t stream) {
  if (!p || !q || !table || !offsets || !length || !out || T < 1 || table_width < 1 || requests < 1)
    return MOE_ERR_INVALID_ARG;
  if (T > p->d.max_tokens || requests > p->d.max_requests) return MOE_ERR_CAPACITY;
  if (mask ? mask_words < 1 || mask_words > 4 : mask_words != 0) return MOE_ERR_INVALID_ARG;
  if (table_width > (1 << 18)) return MOE_ERR_UNSUPPORTED;
  const long long cols = (long long)p->d.heads * p->d.head_dim;
  AttnArgs a{};
  if (!stride_of(q_stride, cols, &a.q_ld) || !stride_of(out_stride, cols, &a.o_ld))
    return MOE_ERR_INVALID_ARG;
  if (!is_aligned(q, 16) || !is_aligned(out, 16) || !is_aligned(table, 4) || !is_aligned(offsets, 4) ||
      !is_aligned(length, 4) || !is_aligned(mask, 8))
    return MOE_ERR_INVALID_ARG;
  Span c[4];
  const moe_status s = check_cache(*p, cache, c);
  if (s != MOE_OK) return s;
  const Span o{out, rows_bytes(T, a.o_ld, cols)};
  const Span in[] = {{q, rows_bytes(T, a.q_ld, cols)}, {table, 4 * (size_t)requests * table_width},
                     {offsets, 4 * ((size_t)requests + 1)}, {length, 4 * (size_t)requests},
                     {mask, 8 * (size_t)T * mask_words}, c[0], c[1], c[2], c[3]};
  for (const Span& x : in)
    if (clash(o, x)) return MOE_ERR_INVALID_ARG;
  const OnDevice on(p->device);
  if (!on.ok()) return MOE_ERR_CUDA;
  a.T = T;
  a.heads = p->d.heads;
  a.kv_heads = p->d.kv_heads;
  a.head_dim = p->d.head_dim;
  a.page_shift = page_shift(p->d.page_size);
  a.e4m3 = p->d.cache_type == MOE_CACHE_E4M3;
  a.q = q;
  a.out = out;
  a.table = table;
  a.offsets = offsets;
  a.length = length;
  a.table_width = table_width;
  a.requests = requests;
  a.mask = reinterpret_cast<const unsigned long long*>(mask);
  a.mask_words = mask_words;
  a.scale = p->d.softmax_scale > 0.0f ? p->d.softmax_scale : 1.0f / sqrtf((float)p->d.head_dim);
  a.cache = dev_of(*cache);
  return launch_tree_attention(a, p->scratch + kErrBytes + kTurnsBytes, p->num_sms, p->err(),
                               reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
