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
// then does it take scores again in 64 bits: those of the experts that may be
// among the first k (one per lane), or of all where the groups are in doubt.
// Without a bias and groups the order is that of the logits, which is exact.
//
// Lane l holds experts VPL l .. VPL l + VPL - 1: its logits are two or four
// 16-byte loads, and of equal keys in several lanes the lowest lane's comes
// first.
#pragma once

#include "topk.cuh"

namespace moe {

struct ScoreDev {
  int sigmoid, groups, topk_groups, renorm;
  float scale;
  const float* bias;
};

// Monotone double -> uint64 (no NaN, -0 already +0).
__device__ __forceinline__ unsigned long long order_key64(double f) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(f);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_value64(unsigned long long k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7FFFFFFFFFFFFFFFull) : ~k));
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

__device__ __forceinline__ float clean_logit(float v) { return isnan(v) ? -INFINITY : v + 0.0f; }

// The bias of expert e, -infinity where the expert is closed.
__device__ __forceinline__ float score_bias(const ScoreDev& s, int e) {
  const float b = __ldg(s.bias + e);
  return isnan(b) ? -INFINITY : b;
}

// Softmax's maximum and sum in 64 bits (the sum 0 where p is 0 throughout).
__device__ __forceinline__ void softmax64(const float* row, int E, double& m, double& z) {
  const int lane = threadIdx.x & 31;
  float mf = -INFINITY;
  for (int e = lane; e < E; e += 32) mf = fmaxf(mf, clean_logit(__ldcg(row + e)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mf = fmaxf(mf, __shfl_xor_sync(0xffffffffu, mf, o));
  m = mf;
  z = 0.0;
  if (isinf(mf)) return;
  for (int e = lane; e < E; e += 32) z += exp((double)clean_logit(__ldcg(row + e)) - m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
}

__device__ __forceinline__ double prob64(const ScoreDev& s, float l, double m, double z) {
  if (s.sigmoid) return 1.0 / (1.0 + exp(-(double)l));
  return z > 0.0 ? exp((double)l - m) / z : 0.0;
}

// Lane j's expert of the choice, from 64-bit scores of every expert.
__device__ __noinline__ int score_exact_all(const float* row, int E, int k, const ScoreDev s) {
  const int lane = threadIdx.x & 31;
  double m = 0.0, z = 1.0;
  if (!s.sigmoid) softmax64(row, E, m, z);
  auto score = [&](int e) {
    double c = prob64(s, clean_logit(__ldcg(row + e)), m, z);
    if (s.bias) c += (double)score_bias(s, e);
    return order_key64(c + 0.0);
  };
  unsigned keep = 0xffffffffu;
  const int gsz = E / s.groups;
  if (s.groups > 1) {
    double mine = 0.0;   // lane g < groups: group g's score
    for (int g = 0; g < s.groups; ++g) {
      unsigned long long k1 = 0ull, k2 = 0ull;   // the lane's two largest
      for (int i = lane; i < gsz; i += 32) {
        const unsigned long long v = score(g * gsz + i);
        k2 = v > k1 ? k1 : v > k2 ? v : k2;
        k1 = v > k1 ? v : k1;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long a = __shfl_xor_sync(0xffffffffu, k1, o);
        const unsigned long long b = __shfl_xor_sync(0xffffffffu, k2, o);
        const unsigned long long lo = a < k1 ? a : k1, hi = b > k2 ? b : k2;
        k1 = a > k1 ? a : k1;
        k2 = lo > hi ? lo : hi;
      }
      if (lane == g) mine = key_value64(k1) + (gsz > 1 ? key_value64(k2) : 0.0);
    }
    int rank = 0;
    for (int g = 0; g < s.groups; ++g) {
      const double o = __shfl_sync(0xffffffffu, mine, g);
      rank += o > mine || (o == mine && g < lane);
    }
    keep = __ballot_sync(0xffffffffu, lane < s.groups && rank < s.topk_groups);
  }
  // k rounds, each the largest key below the last one taken (equal keys: the
  // next higher index)
  unsigned long long last = ~0ull;
  int last_e = -1, mine = 0;
  for (int j = 0; j < k; ++j) {
    unsigned long long bk = 0ull;
    int bi = 0x7fffffff;
    for (int e = lane; e < E; e += 32) {
      if (!((keep >> (e / gsz)) & 1u)) continue;
      // without a bias the experts rank by their logits
      const unsigned long long v = s.bias ? score(e) : (unsigned long long)order_key(clean_logit(__ldcg(row + e)));
      if ((v < last || (v == last && e > last_e)) && v > bk) {
        bk = v;
        bi = e;
      }
    }
    warp_best64(bk, bi);
    last = bk;
    last_e = bi;
    if (lane == j) mine = bi;
  }
  return mine;
}

// The same where only the order of the experts with an FP32 score of at least
// `thr` is in doubt, `cand` of which (bits by the lane's VPL experts) are
// eligible: at most one 64-bit score a lane. `list`: 32 ints of the warp's
// shared memory.
__device__ __noinline__ int score_exact_some(const float* row, int E, int k, const ScoreDev s,
                                             unsigned cand, int e0, int* list) {
  const int lane = threadIdx.x & 31;
  int n = __popc(cand), before = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  const int total = __shfl_sync(0xffffffffu, before, 31);
  if (total > 32) return score_exact_all(row, E, k, s);
  before -= n;
  for (; cand; cand &= cand - 1) list[before++] = e0 + __ffs(cand) - 1;
  __syncwarp();
  double m = 0.0, z = 1.0;
  if (!s.sigmoid) softmax64(row, E, m, z);
  const int e = lane < total ? list[lane] : 0;
  unsigned long long key = 0ull;
  if (lane < total)
    key = order_key64(prob64(s, clean_logit(__ldcg(row + e)), m, z) + (double)score_bias(s, e) + 0.0);
  int rank = 0;   // (the list is in index order)
  for (int j = 0; j < total; ++j) {
    const unsigned long long o = __shfl_sync(0xffffffffu, key, j);
    rank += o > key || (o == key && j < lane);
  }
  __syncwarp();
  if (lane < total) list[rank] = e;
  __syncwarp();
  return lane < k ? list[lane] : 0;
}

// Sorts a lane's 8 (key, expert) pairs: descending, the lower expert first.
__device__ __forceinline__ void sort8(uint32_t (&key)[8], int (&ix)[8]) {
  auto cswap = [&](int a, int b) {
    const bool sw = key[b] > key[a] || (key[b] == key[a] && ix[b] < ix[a]);
    const uint32_t ka = key[a], kb = key[b];
    const int ia = ix[a], ib = ix[b];
    key[a] = sw ? kb : ka;
    key[b] = sw ? ka : kb;
    ix[a] = sw ? ib : ia;
    ix[b] = sw ? ia : ib;
  };
  cswap(0, 2); cswap(1, 3); cswap(4, 6); cswap(5, 7);
  cswap(0, 4); cswap(1, 5); cswap(2, 6); cswap(3, 7);
  cswap(0, 1); cswap(2, 3); cswap(4, 5); cswap(6, 7);
  cswap(2, 4); cswap(3, 5);
  cswap(1, 4); cswap(3, 6);
  cswap(1, 2); cswap(3, 4); cswap(5, 6);
}

// Lane j < k gets the j-th chosen expert and its weight. `sm`: E floats (at
// least 32) of the warp's own shared memory.
template <int VPL>   // experts per lane, E <= 32 * VPL
__device__ __forceinline__ void score_select(const float* __restrict__ row, int E, int k,
                                             const ScoreDev& s, float* sm, int& idx, float& w) {
  const int lane = threadIdx.x & 31;
  const int e0 = VPL * lane;
  const bool live = e0 < E;   // E is a multiple of 8: a lane's 8 are all below E or none
  float l[VPL];
#pragma unroll
  for (int i = 0; i < VPL; i += 4) {
    float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (e0 + i < E) v = __ldcg(reinterpret_cast<const float4*>(row + e0 + i));
    l[i] = clean_logit(v.x);
    l[i + 1] = clean_logit(v.y);
    l[i + 2] = clean_logit(v.z);
    l[i + 3] = clean_logit(v.w);
  }
  // softmax: maximum and sum over all experts
  float m = 0.f, z = 1.f;
  if (!s.sigmoid && (s.bias || s.groups > 1 || !s.renorm)) {
    m = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, l[i]);
    m = key_value(__reduce_max_sync(0xffffffffu, order_key(m)));
    if (!isinf(m)) {
      z = 0.f;
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
  // Bound of a pair's FP32 error: expf within 2 ulp, the additions and the
  // division half an ulp each (sigmoid: below 3.6e-7 p); softmax's argument
  // and sum bring that to 2e-6 p. p <= 1, and softmax's largest p is 1 / z.
  // The bias' addition: half an ulp of c.
  const float perr = s.sigmoid ? 1.2e-6f : 6e-6f / z;
  uint32_t key[VPL];   // every real key is above 0
  int ix[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    ix[i] = e0 + i;
    key[i] = 0u;
    if (e0 + i < E) key[i] = order_key(s.bias ? prob(l[i]) + score_bias(s, e0 + i) + 0.0f : l[i]);
  }
  if constexpr (VPL == 8) sort8(key, ix);
  bool unsure_groups = false;
  if (s.groups > 1) {
    const int gsz = E / s.groups;
    // lanes per group where no lane's experts belong to two groups
    const int per = gsz / VPL;
    const bool whole = gsz % VPL == 0 && (per & (per - 1)) == 0;
    float m1 = -INFINITY, m2 = -INFINITY, big = 0.f;
    int span = per;   // lanes that hold one group's parts: group lane / span
    if (whole) {
      // a lane's two largest; without a bias their p
      if constexpr (VPL == 8) {
        m1 = key_value(key[0]);
        m2 = key_value(key[1]);
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const float v = key_value(key[i]);
          m2 = fmaxf(m2, fminf(m1, v));
          m1 = fmaxf(m1, v);
        }
      }
      if (!live) m1 = m2 = -INFINITY;
    } else {
      // through shared memory: `span` lanes a group, each every span-th expert
      int g2 = 1;
      while (g2 < s.groups) g2 <<= 1;
      span = 32 / g2;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (live && ix[i] < E) sm[ix[i]] = key_value(key[i]);
      __syncwarp();
      const int g = lane / span;
      if (g < s.groups)
        for (int i = lane % span; i < gsz; i += span) {
          const float v = sm[g * gsz + i];
          m2 = fmaxf(m2, fminf(m1, v));
          m1 = fmaxf(m1, v);
        }
      __syncwarp();
    }
    for (int o = 1; o < span; o <<= 1) {
      const float a = __shfl_xor_sync(0xffffffffu, m1, o), b = __shfl_xor_sync(0xffffffffu, m2, o);
      m2 = fmaxf(fmaxf(m2, b), fminf(m1, a));
      m1 = fmaxf(m1, a);
    }
    const int g = lane / span;
    float sum = -INFINITY;
    if (g < s.groups) {
      if (!s.bias) {
        m1 = prob(m1);
        m2 = prob(m2);
      }
      sum = gsz > 1 ? m1 + m2 : m1;
      if (!isinf(m1)) big = fabsf(m1);
      if (gsz > 1 && !isinf(m2)) big = fmaxf(big, fabsf(m2));
    }
    big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
    int rank = 0;
    for (int j = 0; j < s.groups; ++j) {
      const float o = __shfl_sync(0xffffffffu, sum, j * span);
      rank += o > sum || (o == sum && j < g);
    }
    const bool head = lane % span == 0 && g < s.groups;
    const unsigned keep = __ballot_sync(0xffffffffu, head && rank < s.topk_groups);
    // the last group kept and the first dropped: four scores' errors and the
    // sums' roundings
    const unsigned last = __ballot_sync(0xffffffffu, head && rank == s.topk_groups - 1);
    const unsigned next = __ballot_sync(0xffffffffu, head && rank == s.topk_groups);
    if (next) {
      const float a = __shfl_sync(0xffffffffu, sum, __ffs(last) - 1);
      const float b = __shfl_sync(0xffffffffu, sum, __ffs(next) - 1);
      unsure_groups = !(a - b > 2.f * perr + 5e-7f * fmaxf(big, 1.f));
    }
    if (whole) {
      if (!((keep >> (g * span)) & 1u)) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = 0u;
      }
    } else {
      if constexpr (VPL == 8) {
        // the dropped ones leave the sorted list
        int n = 0;
        uint32_t k2[8];
        int i2[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          k2[i] = 0u;
          i2[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (key[i] && ((keep >> (ix[i] / gsz * span)) & 1u)) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j == n) {
                k2[j] = key[i];
                i2[j] = ix[i];
              }
            ++n;
          }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          key[i] = k2[i];
          ix[i] = i2[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (key[i] && !((keep >> (ix[i] / gsz * span)) & 1u)) key[i] = 0u;
      }
    }
  }
  unsigned eligible = 0u;   // bits by position e0 + i, for the 64-bit path
  if (s.bias) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i]) eligible |= 1u << (ix[i] - e0);
  }
  // k rounds, and one more where the order may be unsure: lane j keeps the
  // j-th key
  const int rounds = s.bias ? k + 1 : k;
  uint32_t my_key = 0u;
  int mine = 0;
  for (int j = 0; j < rounds; ++j) {
    uint32_t top = key[0];
    int ti = ix[0];
    if constexpr (VPL > 8) {
#pragma unroll
      for (int i = 1; i < VPL; ++i)
        if (key[i] > top) {
          top = key[i];
          ti = ix[i];
        }
    }
    const uint32_t mk = __reduce_max_sync(0xffffffffu, top);
    const unsigned has = __ballot_sync(0xffffffffu, top == mk);
    const int src = __ffs(has) - 1;   // the lowest lane holds the lowest expert
    const int be = __shfl_sync(0xffffffffu, ti, src);
    if (lane == src) {
      if constexpr (VPL == 8) {
#pragma unroll
        for (int i = 0; i < 7; ++i) {
          key[i] = key[i + 1];
          ix[i] = ix[i + 1];
        }
        key[7] = 0u;
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (ix[i] == be) key[i] = 0u;
      }
    }
    if (lane == (j & 31)) {
      // (round 32 of k = 32 looks at the next key only, and lane 0 has it)
      if (j < 32) {
        my_key = mk;
        mine = be;
      }
    }
    if (j == 32 && lane == 31) sm[0] = key_value(mk), sm[1] = mk ? 1.f : 0.f;
  }
  if (s.bias) {
    // neighbours in the order: lane j against j + 1 <= k
    uint32_t nk = __shfl_down_sync(0xffffffffu, my_key, 1);
    if (k == 32) {
      __syncwarp();
      if (lane == 31) nk = sm[1] != 0.f ? order_key(sm[0]) : 0u;
      __syncwarp();
    }
    const float a = key_value(my_key), b = key_value(nk);
    // (equal infinities are certain: closed experts, by index)
    const bool close = lane < k && nk != 0u && !(isinf(a) && a == b) &&
                       !(a - b > perr + 2.5e-7f * fmaxf(fabsf(a), fabsf(b)));
    if (unsure_groups) {
      mine = score_exact_all(row, E, k, s);
    } else if (__any_sync(0xffffffffu, close)) {
      const float vk = key_value(__shfl_sync(0xffffffffu, my_key, k - 1));
      const float thr = vk - 2.f * (perr + 2.5e-7f * fabsf(vk));
      unsigned cand = 0u;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if ((eligible >> i) & 1u)
          if (!(prob(l[i]) + score_bias(s, e0 + i) < thr)) cand |= 1u << i;
      mine = score_exact_some(row, E, k, s, cand, e0, reinterpret_cast<int*>(sm));
    }
  } else if (unsure_groups) {
    mine = score_exact_all(row, E, k, s);
  }
  // the chosen experts' weights, lane j the j-th
  float lj = -INFINITY;
  bool open = false;
  if (lane < k) {
    lj = clean_logit(__ldcg(row + mine));
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
    float sum = pj;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    pj = sum > 0.f ? pj / sum : 0.f;
  } else if (open) {
    pj = prob(lj);
  }
  idx = mine;
  w = pj * s.scale;
}

}  // namespace moe
