// score_topk.cuh -- one token's choice of experts by one warp, by scores with
// a balance bias and groups (moe_route_scored).
//
//   p = softmax(l) or sigmoid(l); c = p + bias (no bias: ordered by l)
//   group score = sum of the group's two largest c; the best groups stay
//   chosen: the k largest c of the groups that stay, lower index first
//   weight = p (over the chosen ones' sum) * scale
//
// The choice has to be that of 64-bit scores, but nearly every token's order
// is already certain in 32 bits: the warp works in FP32 with a bound on the
// scores' error and looks whether two neighbours in the order (or the last
// group kept and the first dropped) lie closer than twice that bound. Only
// then does it take the token's scores again in 64 bits (score_refine).
// Without a bias and groups the order is that of the logits, which is exact.
#pragma once

#include "topk.cuh"

namespace moe {

struct ScoreDev {
  int sigmoid, groups, topk_groups, renorm;
  float scale;
  const float* bias;
};

// Monotone double -> uint64 and back (no NaN, -0 already +0).
__device__ __forceinline__ unsigned long long order_key64(double f) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(f);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// Maximum over the warp, and the lowest index that holds it.
__device__ __forceinline__ void warp_best64(unsigned long long& key, int& ix) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long ok = __shfl_xor_sync(0xffffffffu, key, o);
    const int oi = __shfl_xor_sync(0xffffffffu, ix, o);
    if (ok > key || (ok == key && oi < ix)) {
      key = ok;
      ix = oi;
    }
  }
}

// The bias of expert e, -infinity where the expert is closed.
__device__ __forceinline__ float score_bias(const ScoreDev& s, int e) {
  const float b = __ldg(s.bias + e);
  return isnan(b) ? -INFINITY : b;
}

// The choice with 64-bit scores (rare; see the file comment). l[i] is the
// logit of expert lane + 32 i.
template <int VPL>
__device__ __noinline__ int score_refine(const float (&l)[VPL], int E, int k, const ScoreDev& s) {
  const int lane = threadIdx.x & 31;
  unsigned long long key[VPL];
  double z = 1.0, m = 0.0;
  if (!s.sigmoid) {
    float mf = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 32 * i < E) mf = fmaxf(mf, l[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mf = fmaxf(mf, __shfl_xor_sync(0xffffffffu, mf, o));
    m = mf;
    z = 0.0;
    for (int i = 0; i < VPL; ++i)
      if (lane + 32 * i < E) z += exp((double)l[i] - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  }
  const bool flat = !s.sigmoid && isinf(m);   // no finite maximum: p = 0
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0ull;
    if (e < E) {
      double c = s.sigmoid ? 1.0 / (1.0 + exp(-(double)l[i])) : flat ? 0.0 : exp((double)l[i] - m) / z;
      if (s.bias) c += (double)score_bias(s, e);
      key[i] = order_key64(c + 0.0);
    }
  }
  if (s.groups > 1) {
    const int gsz = E / s.groups;
    double mine = 0.0;   // lane g < groups: group g's score
    for (int g = 0; g < s.groups; ++g) {
      double sum = 0.0;
      int first = -1;
      for (int r = 0; r < (gsz > 1 ? 2 : 1); ++r) {
        unsigned long long bk = 0ull;
        int bi = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int e = lane + 32 * i;
          if (e < E && e / gsz == g && e != first && key[i] > bk) {
            bk = key[i];
            bi = e;
          }
        }
        warp_best64(bk, bi);
        first = bi;
        sum += __longlong_as_double((long long)((bk >> 63) ? (bk & 0x7FFFFFFFFFFFFFFFull) : ~bk));
      }
      if (lane == g) mine = sum;
    }
    int rank = 0;
    for (int g = 0; g < s.groups; ++g) {
      const double o = __shfl_sync(0xffffffffu, mine, g);
      rank += o > mine || (o == mine && g < lane);
    }
    const unsigned keep = __ballot_sync(0xffffffffu, lane < s.groups && rank < s.topk_groups);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !((keep >> (e / gsz)) & 1u)) key[i] = 0ull;
      // without a bias the experts rank by their logits
      else if (e < E && !s.bias) key[i] = (unsigned long long)order_key(l[i]) + 1ull;
    }
  } else if (!s.bias) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane + 32 * i < E) key[i] = (unsigned long long)order_key(l[i]) + 1ull;
  }
  int mine = 0;
  for (int j = 0; j < k; ++j) {
    unsigned long long bk = 0ull;
    int bi = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > bk) {
        bk = key[i];
        bi = lane + 32 * i;
      }
    warp_best64(bk, bi);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (bi == lane + 32 * i) key[i] = 0ull;
    if (lane == j) mine = bi;
  }
  return mine;
}

// Lane j < k gets the j-th chosen expert and its weight.
template <int VPL>
__device__ __forceinline__ void score_select(const float* __restrict__ row, int E, int k,
                                             const ScoreDev& s, int& idx, float& w) {
  const int lane = threadIdx.x & 31;
  float l[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    const float v = e < E ? __ldcg(row + e) : -INFINITY;
    l[i] = isnan(v) ? -INFINITY : v + 0.0f;   // + 0 turns -0 into +0
  }
  // softmax: maximum and sum over all experts
  float m = 0.f, z = 1.f;
  const bool need_p = s.bias || s.groups > 1 || !s.renorm;
  if (!s.sigmoid && need_p) {
    m = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
    m = key_value(__reduce_max_sync(0xffffffffu, order_key(m)));
    z = 0.f;
    if (!isinf(m)) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) z += expf(l[i] - m);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    }
  }
  auto prob = [&](float v) {
    if (s.sigmoid) return 1.0f / (1.0f + expf(-v));
    return isinf(m) ? 0.f : expf(v - m) / z;
  };
  // Bound of a score's FP32 error, twice over for a pair: expf within 2 ulp,
  // the additions and the division half an ulp each (sigmoid: below 5e-7 p);
  // softmax's argument and sum add up to 2e-6 p. p <= 1, and softmax's
  // largest p is 1 / z. The bias' addition: half an ulp of c.
  const float perr = s.sigmoid ? 1.2e-6f : 6e-6f / fmaxf(z, 1.f);
  uint32_t key[VPL];
  bool unsure = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0u;   // every real key is above 0
    if (e < E) key[i] = order_key(s.bias ? prob(l[i]) + score_bias(s, e) + 0.0f : l[i]);
  }
  if (s.groups > 1) {
    const int gsz = E / s.groups;
    float mine = 0.f;   // lane g < groups: group g's score
    float big = 0.f;    // largest finite |c| that enters one
    for (int g = 0; g < s.groups; ++g) {
      float sum = 0.f;
      int first = -1;
      for (int r = 0; r < (gsz > 1 ? 2 : 1); ++r) {
        uint32_t bk = 0u;
        int bi = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int e = lane + 32 * i;
          if (e < E && e / gsz == g && e != first && key[i] > bk) {
            bk = key[i];
            bi = e;
          }
        }
        const uint32_t mk = __reduce_max_sync(0xffffffffu, bk);
        first = (int)__reduce_min_sync(0xffffffffu, bk == mk ? (uint32_t)bi : 0xffffffffu);
        const float v = key_value(mk);
        sum += s.bias ? v : prob(v);
        if (s.bias && !isinf(v)) big = fmaxf(big, fabsf(v));
      }
      if (lane == g) mine = sum;
    }
    int rank = 0;
    for (int g = 0; g < s.groups; ++g) {
      const float o = __shfl_sync(0xffffffffu, mine, g);
      rank += o > mine || (o == mine && g < lane);
    }
    const unsigned keep = __ballot_sync(0xffffffffu, lane < s.groups && rank < s.topk_groups);
    // the last group kept and the first dropped
    const unsigned last = __ballot_sync(0xffffffffu, lane < s.groups && rank == s.topk_groups - 1);
    const unsigned next = __ballot_sync(0xffffffffu, lane < s.groups && rank == s.topk_groups);
    if (next) {
      const float a = __shfl_sync(0xffffffffu, mine, __ffs(last) - 1);
      const float b = __shfl_sync(0xffffffffu, mine, __ffs(next) - 1);
      unsure = !(a - b > 2.f * perr + 5e-7f * fmaxf(big, 1.f));
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !((keep >> (e / gsz)) & 1u)) key[i] = 0u;
    }
  }
  // k rounds, and one more where the order may be unsure
  const int rounds = s.bias ? k + 1 : k;
  float prev = INFINITY;
  int mine = 0;
  for (int j = 0; j < rounds; ++j) {
    uint32_t bk = 0u;
    int bi = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > bk) {
        bk = key[i];
        bi = lane + 32 * i;
      }
    const uint32_t mk = __reduce_max_sync(0xffffffffu, bk);
    if (mk == 0u) break;   // round k + 1 with no expert left
    const int be = (int)__reduce_min_sync(0xffffffffu, bk == mk ? (uint32_t)bi : 0xffffffffu);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (be == lane + 32 * i) key[i] = 0u;
    if (lane == j && j < k) mine = be;
    const float v = key_value(mk);
    // equal infinities are certain (closed experts, by index)
    if (s.bias && j > 0 && !(isinf(v) && v == prev) &&
        !(prev - v > perr + 2.5e-7f * fmaxf(fabsf(prev), fabsf(v))))
      unsure = true;
    prev = v;
  }
  if (unsure) mine = score_refine<VPL>(l, E, k, s);
  // the chosen experts' weights, lane j the j-th
  float lj = -INFINITY;
  bool open = false;
  if (lane < k) {
    const float v = __ldcg(row + mine);
    lj = isnan(v) ? -INFINITY : v;
    open = !s.bias || score_bias(s, mine) > -INFINITY;
  }
  float pj = 0.f;
  if (s.renorm) {
    // relative to the largest chosen logit, so that no sum underflows; a
    // sigmoid far below zero is the exponential, and below -745 (a row of
    // masks of the type's lowest value) it is 0 in 64 bits too
    const float top = key_value(__reduce_max_sync(0xffffffffu, order_key(open ? lj : -INFINITY)));
    if (open && top > (s.sigmoid ? -745.f : -INFINITY)) {
      if (s.sigmoid) pj = top < -40.f ? expf(lj - top) : 1.0f / (1.0f + expf(-lj));
      else if (!isinf(top) && !isinf(m)) pj = expf(lj - top);
    }
    float sum = 0.f;
    for (int j = 0; j < k; ++j) sum += __shfl_sync(0xffffffffu, pj, j);
    pj = sum > 0.f ? pj / sum : 0.f;
  } else if (open) {
    pj = prob(lj);
  }
  idx = mine;
  w = pj * s.scale;
}

}  // namespace moe
