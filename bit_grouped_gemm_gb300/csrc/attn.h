// attn.h -- what the kernels of attention over a paged cache share.
#pragma once

#include "moe_internal.h"

namespace moe {

struct CacheDev {
  void *k, *v;
  const float *k_scale, *v_scale;   // e4m3 only
  int pages;
};

// ------------------------------------------------------ rotary positions ---
struct RopeArgs {
  int T, heads, kv_heads, head_dim, rotary_dim;
  bool interleaved, e4m3;
  int page_shift;
  const uint16_t *q, *k, *v;
  long long q_ld, k_ld, v_ld, o_ld;
  uint16_t* q_out;
  const int32_t *position, *slot;
  const unsigned long long* turns;   // [rotary_dim / 2] turns per position, times 2^64
  float gain;
  CacheDev cache;
};
cudaError_t launch_rope_store(const RopeArgs& a, cudaStream_t st);

// -------------------------------------------------------------- attention ---
struct AttnArgs {
  int T, heads, kv_heads, head_dim, page_shift;
  bool e4m3;
  const uint16_t* q;
  long long q_ld, o_ld;
  uint16_t* out;
  const int32_t *table, *offsets, *length;
  int table_width, requests;
  const unsigned long long* mask;
  int mask_words;
  float scale;                       // of q k^T
  CacheDev cache;
};

// Scratch: a CTA leaves the sums of at most two row tiles that it shares with
// other CTAs, each of up to 128 rows, and says which shared tile it begins.
constexpr int kAttnMaxCtas = 160;
constexpr size_t attn_scratch_bytes(int head_dim) {
  return kAttnMaxCtas * (8 + 2 * 128 * ((size_t)head_dim + 2) * 4);
}
cudaError_t launch_tree_attention(const AttnArgs& a, void* scratch, int num_sms, DevErr err,
                                  cudaStream_t st);

}  // namespace moe
