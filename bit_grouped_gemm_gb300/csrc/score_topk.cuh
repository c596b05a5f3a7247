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
// group kept and the first dropped) lie closer than that allows. Only then does
// it look again, in pairs of floats, and in 64 bits where these cannot tell
// either. Without a bias and groups the order is that of the logits, which is
// exact.
//
// Lane l holds experts VPL l .. VPL l + VPL - 1. The choice itself takes no
// rounds: the (k + 1)-th largest of the lanes' largest keys bounds the
// (k + 1)-th largest key from below, so the few keys at or above it are put
// into a list, in index order, one per lane, and each lane counts how many of
// the list come before its own.
#pragma once

#include "topk.cuh"

namespace moe {

struct ScoreDev {
  int sigmoid, groups, topk_groups, renorm;
  float scale;
  const float* bias;
  // Groups (more than one): experts per group and the factor of a division by
  // it (e gdiv >> 20, e < 512); lanes per group, 2^span_log2, each with whole
  // experts of one group only, or (whole = 0) taking turns at its experts.
  int gsz, gdiv, span_log2, whole;
};

// The group of expert e.
__device__ __forceinline__ int group_of(const ScoreDev& s, int e) { return (e * s.gdiv) >> 20; }

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

// NaN as -infinity, -0 as +0
__device__ __forceinline__ float clean_logit(float v) { return fmaxf(v, -INFINITY) + 0.0f; }

// The bias of expert e, -infinity where the expert is closed.
__device__ __forceinline__ float score_bias(const ScoreDev& s, int e) {
  return fmaxf(__ldg(s.bias + e), -INFINITY);
}

// Softmax's maximum and sum in 64 bits (the sum 0 where p is 0 throughout).
__device__ __forceinline__ void softmax64(const float* row, int E, double& m, double& z) {
  const int lane = threadIdx.x & 31;
  float mf = -INFINITY;
  for (int e = lane; e < E; e += 32) mf = fmaxf(mf, clean_logit(__ldg(row + e)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mf = fmaxf(mf, __shfl_xor_sync(0xffffffffu, mf, o));
  m = mf;
  z = 0.0;
  if (isinf(mf)) return;
  for (int e = lane; e < E; e += 32) z += exp((double)clean_logit(__ldg(row + e)) - m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
}

__device__ __forceinline__ double prob64(const ScoreDev& s, float l, double m, double z) {
  if (s.sigmoid) return 1.0 / (1.0 + exp(-(double)l));
  return z > 0.0 ? exp((double)l - m) / z : 0.0;
}

// Lane j's expert of the choice, from 64-bit scores of every expert, each
// taken once.
template <int VPL>
__device__ __noinline__ int score_exact_all(const float* row, int E, int k, const ScoreDev s) {
  const int lane = threadIdx.x & 31, gsz = E / s.groups;
  double m = 0.0, z = 1.0;
  if (!s.sigmoid) softmax64(row, E, m, z);
  unsigned long long key[VPL];
#pragma unroll 1
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0ull;
    if (e < E) {
      double c = prob64(s, clean_logit(__ldg(row + e)), m, z);
      if (s.bias) c += (double)score_bias(s, e);
      key[i] = order_key64(c + 0.0);
    }
  }
  unsigned keep = 0xffffffffu;
  if (s.groups > 1) {
    double mine = 0.0;   // lane g < groups: group g's score
    for (int g = 0; g < s.groups; ++g) {
      unsigned long long k1 = 0ull, k2 = 0ull;   // the lane's two largest
#pragma unroll 1
      for (int i = 0; i < VPL; ++i) {
        const int e = lane + 32 * i;
        if (e >= g * gsz && e < (g + 1) * gsz) {
          const unsigned long long v = key[i];
          k2 = v > k1 ? k1 : v > k2 ? v : k2;
          k1 = v > k1 ? v : k1;
        }
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
#pragma unroll 1
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    if (e >= E) continue;
    if (!((keep >> (e / gsz)) & 1u)) key[i] = 0ull;
    // without a bias the experts rank by their logits
    else if (!s.bias) key[i] = order_key(clean_logit(__ldg(row + e)));
  }
  int mine = 0;
  for (int j = 0; j < k; ++j) {
    unsigned long long bk = 0ull;
    int bi = 0x7fffffff;
#pragma unroll 1
    for (int i = 0; i < VPL; ++i)
      if (key[i] > bk) {
        bk = key[i];
        bi = lane + 32 * i;
      }
    warp_best64(bk, bi);
#pragma unroll 1
    for (int i = 0; i < VPL; ++i)
      if (bi == lane + 32 * i) key[i] = 0ull;
    if (lane == j) mine = bi;
  }
  return mine;
}

// 1 / v to 1 ulp
__device__ __forceinline__ float rcp_1ulp(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// exp(v) in two instructions, to a relative 2^-22 + 7.5e-8 |v| (the rounding of
// v log2(e)): for ranking, where far exponents are small terms.
__device__ __forceinline__ float exp_rank(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fmul_rn(v, 1.44269504f)));
  return r;
}

// The FP32 score of an expert (without its bias) as it is ranked; softmax: from
// the row's maximum and the reciprocal of its sum (0 where p is 0 throughout).
__device__ __forceinline__ float score_prob(const ScoreDev& s, float l, float m, float rz) {
  if (s.sigmoid) return rcp_1ulp(1.0f + exp_rank(-l));
  return rz > 0.f ? __fmul_rn(exp_rank(l - m), rz) : 0.f;
}

// Writes the lane's experts e0 + i, i in the set `cand`, into `list` (32
// entries of the warp's shared memory) in index order; returns the warp's
// count, and writes nothing if that is above 32.
__device__ __forceinline__ int list_candidates(unsigned cand, int e0, int* list) {
  const int lane = threadIdx.x & 31, n = __popc(cand);
  int before = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  const int total = __shfl_sync(0xffffffffu, before, 31);
  if (total <= 32)
    for (before -= n; cand; cand &= cand - 1) list[before++] = e0 + __ffs(cand) - 1;
  __syncwarp();
  return total;
}

// ---------------------------------------------------------------------------
// Scores between FP32 and FP64. A warp's FP64 exponential takes about a
// microsecond here, so the second look is taken in pairs of floats (a value
// and what its rounding left), good to 1e-11, and only what 2e-10 cannot tell
// goes to FP64. One score per lane, of the experts in doubt alone: a look at
// every expert of the row took 8 us unrolled (its code is cold on the SM) and
// 11 us in loops (each score is one long chain). Sums and products whose rounding
// is taken up by the pair are written as rounded operations: fused into one with
// their neighbours, which the compiler may do to + and *, that rounding would count
// twice (a sigmoid off by 4.6e-9).
// ---------------------------------------------------------------------------
struct F2 {
  float h, l;
};
__device__ __forceinline__ F2 sum_ordered(float a, float b) {   // |a| >= |b| or a = 0
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ F2 sum_any(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
// c + a b for a constant c above |a b|
__device__ __forceinline__ F2 mul_add(F2 a, F2 b, float ch, float cl) {
  const float p = __fmul_rn(a.h, b.h);
  const float e = fmaf(a.h, b.h, -p) + fmaf(a.h, b.l, a.l * b.h);
  const F2 s = sum_ordered(ch, p);
  return sum_ordered(s.h, s.l + (e + cl));
}

// exp(x) to a relative 1e-11 for |x| <= 40, 4e-11 for |x| <= 80: x = n ln 2 + 2 r with ln 2 split as
// 355/512 less a remainder (n 355/512 and its difference from x are exact),
// then the exponential's series at r, |r| <= 0.174, up to r^3 in pairs and
// from r^4 in floats (r^4/24's rounding: 2e-12), squared.
__device__ __forceinline__ F2 exp_f2(float x) {
  const float n = rintf(x * 1.44269504f);
  const float t = fmaf(n, -0.693359375f, x);
  const float ch = 0x1.bd0106p-13f, cl = -0x1.cf79acp-40f;   // 355/512 - ln 2
  const float p = __fmul_rn(n, ch);
  F2 r = sum_any(t, p);
  r.l += fmaf(n, ch, -p) + n * cl;
  r.h *= 0.5f;
  r.l *= 0.5f;
  const float tail = r.h * fmaf(r.h, fmaf(r.h, fmaf(r.h, 1.f / 40320.f, 1.f / 5040.f), 1.f / 720.f), 1.f / 120.f);
  F2 g = {1.f / 24.f + tail, 0.f};
  g = mul_add(r, g, 0x1.555556p-3f, -0x1.555556p-28f);   // 1/6
  g = mul_add(r, g, 0.5f, 0.f);
  g = mul_add(r, g, 1.f, 0.f);
  g = mul_add(r, g, 1.f, 0.f);
  const float sq = __fmul_rn(g.h, g.h);
  const F2 e = sum_ordered(sq, fmaf(g.h, g.h, -sq) + 2.f * g.h * g.l);
  const float k = __int_as_float(((int)n + 127) << 23);   // 2^n, |n| <= 116
  return {e.h * k, e.l * k};
}
// a / d
__device__ __forceinline__ F2 div_f2(F2 a, F2 d) {
  const float q = a.h / d.h;
  const float r = (fmaf(-q, d.h, a.h) + a.l) - q * d.l;
  return sum_ordered(q, r / d.h);
}

// Units of 2^-40 of a score. A score is off by at most 30 of them, so two
// sums of two by 120.
constexpr long long kFineSure = 256;
__device__ __forceinline__ long long fine_units(F2 v) {
  return __float2ll_rn(v.h * 0x1p40f) + __float2ll_rn(v.l * 0x1p40f);
}

// The row's softmax sum (0 where p is 0 throughout), maximum m, four terms at
// a time.
template <int VPL>
__device__ __noinline__ F2 softmax_f2(const float* row, int E, float m) {
  const int lane = threadIdx.x & 31;
  F2 z = {0.f, 0.f};
  if (isinf(m)) return z;
  constexpr int kStep = VPL < 4 ? VPL : 4;
#pragma unroll 1
  for (int i0 = 0; i0 < VPL; i0 += kStep) {
    F2 t[kStep];
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      const int e = lane + 32 * (i0 + i);
      const float l = e < E ? clean_logit(__ldg(row + e)) : -INFINITY;
      const F2 d = sum_any(fmaxf(l, m - 80.f), -m);   // (l - m in a pair: its rounding would cost 1e-7)
      t[i] = exp_f2(fmaxf(d.h, -80.f));
      t[i].l += t[i].h * d.l;
      if (!(l - m > -80.f)) t[i] = {0.f, 0.f};
    }
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      const F2 u = sum_any(z.h, t[i].h);
      z = sum_ordered(u.h, u.l + (z.l + t[i].l));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float oh = __shfl_xor_sync(0xffffffffu, z.h, o), ol = __shfl_xor_sync(0xffffffffu, z.l, o);
    const F2 u = sum_any(z.h, oh);
    z = sum_ordered(u.h, u.l + (z.l + ol));
  }
  return z;
}

// A score (p, and the bias of an open expert) in units of 2^-40 above 2^62; 1
// for a closed expert, 0 where the bias is beyond the units.
__device__ __noinline__ unsigned long long fine_score(int sigmoid, float l, float b, float m, F2 z) {
  if (b == -INFINITY) return 1ull;
  if (!(fabsf(b) < 0x1p18f)) return 0ull;
  F2 p = {0.f, 0.f};
  const F2 d = sigmoid ? F2{fminf(fmaxf(-l, -80.f), 80.f), 0.f} : sum_any(fmaxf(l, m - 80.f), -m);
  if (sigmoid || (z.h > 0.f && l - m > -80.f)) {
    F2 x = exp_f2(d.h);
    x.l += x.h * d.l;
    F2 y = z;
    if (sigmoid) {
      const F2 u = sum_any(1.f, x.h);
      y = sum_ordered(u.h, u.l + x.l);
      x = {1.f, 0.f};
    }
    p = div_f2(x, y);
  }
  const F2 c = sum_any(p.h, b);
  return (1ull << 62) + (unsigned long long)fine_units({c.h, c.l + p.l});
}

// Lane j's expert of the choice among the `total` <= 32 listed ones, by fine
// scores; -1 in every lane where these cannot tell.
__device__ __noinline__ int fine_order(const float* row, int k, const ScoreDev s, float m, F2 z,
                                       int* list, int total) {
  const int lane = threadIdx.x & 31;
  const int e = lane < total ? list[lane] : 0;
  const float l = clean_logit(__ldg(row + e)), b = score_bias(s, e);
  const unsigned long long key = lane < total ? fine_score(s.sigmoid, l, b, m, z) : 0ull;
  // A chosen one is too close to any other that is not the same score by
  // definition (the neighbour alone would not do: equal scores may stand between).
  int rank = 0;
  bool close = false;
#pragma unroll 4
  for (int j = 0; j < total; ++j) {
    const unsigned long long o = __shfl_sync(0xffffffffu, key, j);
    const float ol = __shfl_sync(0xffffffffu, l, j), ob = __shfl_sync(0xffffffffu, b, j);
    rank += o > key || (o == key && j < lane);
    const unsigned long long gap = o > key ? o - key : key - o;
    close |= gap <= (unsigned long long)kFineSure && key > 1ull && !(l == ol && b == ob);
  }
  __syncwarp();
  if (lane < total) list[rank] = lane;
  __syncwarp();
  const int mine_lane = lane < total ? list[lane] : 0;
  __syncwarp();
  const bool bad = lane < total && (key == 0ull || (rank < k && close));
  const int mine = __shfl_sync(0xffffffffu, e, mine_lane);
  return __any_sync(0xffffffffu, bad) ? -1 : mine;
}

// Which of the doubtful groups (bits by group) stay, `want` of them, from the
// `total` <= 32 listed experts, which hold each one's two best; returns the
// kept ones' bits, 0 where fine scores cannot tell.
__device__ __noinline__ unsigned fine_groups(const float* row, int gsz, const ScoreDev s, float m, F2 z,
                                             const int* list, int total, unsigned doubt, int want) {
  const int lane = threadIdx.x & 31;
  const int e = lane < total ? list[lane] : 0, grp = lane < total ? e / gsz : -1;
  unsigned long long key = 0ull;
  if (lane < total)
    key = fine_score(s.sigmoid, clean_logit(__ldg(row + e)), s.bias ? score_bias(s, e) : 0.f, m, z);
  const bool beyond = lane < total && key == 0ull;
  long long mine = 0;   // lane g: group g's sum
  for (unsigned left = doubt; left; left &= left - 1) {
    const int g = __ffs(left) - 1;
    unsigned long long k1 = grp == g ? key : 0ull, k2 = 0ull;
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long a = __shfl_xor_sync(0xffffffffu, k1, o);
      const unsigned long long b = __shfl_xor_sync(0xffffffffu, k2, o);
      const unsigned long long lo = a < k1 ? a : k1, hi = b > k2 ? b : k2;
      k1 = a > k1 ? a : k1;
      k2 = lo > hi ? lo : hi;
    }
    // (of a group with one open logit the list has that alone, the next p is 0)
    if (!s.bias) {
      k1 = k1 > (1ull << 62) ? k1 : 1ull << 62;
      k2 = k2 > (1ull << 62) ? k2 : 1ull << 62;
    }
    // (a group with a closed expert among its two best is -infinity)
    const bool shut = k1 <= 1ull || (gsz > 1 && k2 <= 1ull);
    const long long one = 1ll << 62;
    if (lane == g)
      mine = shut ? -(1ll << 61) : ((long long)k1 - one) + (gsz > 1 ? (long long)k2 - one : 0ll);
  }
  int rank = 0;
  for (unsigned left = doubt; left; left &= left - 1) {
    const int g = __ffs(left) - 1;
    const long long o = __shfl_sync(0xffffffffu, mine, g);
    rank += o > mine || (o == mine && g < lane);
  }
  const bool in = (doubt >> lane) & 1u;
  const unsigned keep = __ballot_sync(0xffffffffu, in && rank < want);
  const unsigned last = __ballot_sync(0xffffffffu, in && rank == want - 1);
  const unsigned next = __ballot_sync(0xffffffffu, in && rank == want);
  bool bad = beyond || !last;
  if (last && next) {
    const long long a = __shfl_sync(0xffffffffu, mine, __ffs(last) - 1);
    const long long b = __shfl_sync(0xffffffffu, mine, __ffs(next) - 1);
    bad |= a - b <= kFineSure;
  }
  return __any_sync(0xffffffffu, bad) ? 0u : keep;
}

// The choice in rounds of one key each, among the keys (0: not eligible) of
// the lane's experts; lane j gets the j-th of `need`, its key and the next.
template <int VPL>
__device__ __noinline__ int choose_in_rounds(const float* row, int E, const ScoreDev s, float m, float rz,
                                             unsigned elig, int need, uint32_t& my_key,
                                             uint32_t& next_key) {
  const int lane = threadIdx.x & 31, e0 = VPL * lane;
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    key[i] = 0u;
    if ((elig >> i) & 1u) {
      const float l = clean_logit(__ldg(row + e0 + i));
      key[i] = order_key(s.bias ? score_prob(s, l, m, rz) + score_bias(s, e0 + i) : l);
    }
  }
  int mine = 0;
  my_key = next_key = 0u;
#pragma unroll 1
  for (int j = 0; j < need; ++j) {
    uint32_t hk = key[0];
    int hi = 0;
#pragma unroll
    for (int i = 1; i < VPL; ++i)
      if (key[i] > hk) {
        hk = key[i];
        hi = i;
      }
    const uint32_t mk = __reduce_max_sync(0xffffffffu, hk);
    // the lowest lane that holds it has the lowest expert
    const int src = __ffs(__ballot_sync(0xffffffffu, hk == mk)) - 1;
    const int be = __shfl_sync(0xffffffffu, e0 + hi, src);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lane == src && i == hi) key[i] = 0u;
    if (lane == j) {
      mine = be;
      my_key = mk;
    }
    if (lane == j - 1) next_key = mk;
  }
  return mine;
}

// Lane j < k gets the j-th chosen expert and its weight. `sm`: max(E, 64)
// floats of the warp's own shared memory.
template <int VPL>   // experts per lane, E <= 32 * VPL
__device__ __forceinline__ void score_select(const float* __restrict__ row, int E, int k,
                                             const ScoreDev& s, float* sm, int& idx, float& w) {
  const int lane = threadIdx.x & 31;
  const int e0 = VPL * lane;
  // the lane's logits, then its scores c (without a bias: the logits still)
  float c[VPL];
  // (through L1, where the bias stays: every token reads the same one)
  auto load_row = [&](const float* src, auto&& put) {
    if constexpr (VPL == 2) {
      float2 v = make_float2(-INFINITY, -INFINITY);
      if (e0 < E) v = __ldg(reinterpret_cast<const float2*>(src + e0));
      put(0, v.x);
      put(1, v.y);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; i += 4) {
        float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (e0 + i < E) v = __ldg(reinterpret_cast<const float4*>(src + e0 + i));
        put(i, v.x);
        put(i + 1, v.y);
        put(i + 2, v.z);
        put(i + 3, v.w);
      }
    }
  };
  load_row(row, [&](int i, float v) { c[i] = fmaxf(v, -INFINITY); });   // NaN as -infinity
  // the bias is loaded ahead where there are registers for it
  float bias[VPL];
  auto load_bias = [&] { load_row(s.bias, [&](int i, float v) { bias[i] = v; }); };
  if (VPL <= 8 && s.bias) load_bias();
  float m = 0.f, rz = 1.f;
  if (!s.sigmoid && (s.bias || s.groups > 1 || !s.renorm)) {
    m = c[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, c[i]);
    m = key_value(__reduce_max_sync(0xffffffffu, order_key(m)));
    const float mm = isinf(m) ? 0.f : m;
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const float p = exp_rank(c[i] - mm);
      if (s.bias) c[i] = p;
      z += p;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    rz = isinf(m) ? 0.f : 1.0f / z;
  }
  if (s.bias) {
    if (s.sigmoid) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = rcp_1ulp(1.0f + exp_rank(-c[i]));
    } else if (rz > 0.f) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = __fmul_rn(c[i], rz);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = 0.f;
    }
    if (VPL > 8) load_bias();
    // (a NaN bias as -infinity: lanes past E keep -infinity this way too)
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = fmaxf(__fadd_rn(c[i], bias[i]), -INFINITY);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] += 0.0f;   // -0 as +0
  }
  // Bound of a pair's FP32 error, from exp_rank's, the reciprocal's 1 ulp and
  // half an ulp for every other operation. Sigmoid: e = exp(-l) enters
  // p = 1 / (1 + e) by 1 - p, so p is off by p (1 - p) (2^-22 + 7.5e-8 |l|) +
  // 1.5 p 2^-23 < 2.6e-7. Softmax, of the largest p, 1 / z: 3.6e-7 by the
  // exponential (its argument's two roundings too) and the product, for each of
  // the two, and 1.9e-6 by 1 / z (at most 21 additions), which both share. The
  // bias' addition: half an ulp of c.
  const float perr = s.sigmoid ? 5.5e-7f : 2.8e-6f * rz;
  float top = c[0];   // the lane's largest
#pragma unroll
  for (int i = 1; i < VPL; ++i) top = fmaxf(top, c[i]);
  bool unsure_groups = false;
  constexpr unsigned kAll = (unsigned)((1ull << VPL) - 1ull);
  unsigned elig = e0 + VPL <= E ? kAll : e0 >= E ? 0u : (1u << (E - e0)) - 1u;
  if (s.groups > 1) {
    const int gsz = s.gsz, span = 1 << s.span_log2, g = lane >> s.span_log2;
    const bool whole = s.whole != 0;
    float m1 = -INFINITY, m2 = -INFINITY;   // the lane's two largest of its group
    if (whole) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        m2 = fmaxf(m2, fminf(m1, c[i]));
        m1 = fmaxf(m1, c[i]);
      }
    } else {
      // through shared memory
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (e0 + i < E) sm[e0 + i] = c[i];
      __syncwarp();
      if (g < s.groups)
        for (int i = lane & (span - 1); i < gsz; i += span) {
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
    const float low = m2 > -INFINITY ? m2 : m1;   // the second largest
    float sum = -INFINITY, big = 0.f;
    if (g < s.groups) {
      if (!s.bias) {
        m1 = score_prob(s, m1, m, rz);
        m2 = score_prob(s, m2, m, rz);
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
    const bool head = (lane & (span - 1)) == 0 && g < s.groups;
    unsigned keep = __ballot_sync(0xffffffffu, head && rank < s.topk_groups);
    // the last group kept and the first dropped: four scores' errors and the
    // sums' roundings
    const unsigned last = __ballot_sync(0xffffffffu, head && rank == s.topk_groups - 1);
    const unsigned next = __ballot_sync(0xffffffffu, head && rank == s.topk_groups);
    if (next) {
      const float a = __shfl_sync(0xffffffffu, sum, __ffs(last) - 1);
      const float b = __shfl_sync(0xffffffffu, sum, __ffs(next) - 1);
      const float wide = 2.f * perr + 5e-7f * fmaxf(big, 1.f);
      if (!(a - b > wide)) {
        // doubtful: the groups between b and a, within the bound; their experts
        // that may be among their two best go into the list
        const bool dub = head && sum >= b - wide && sum <= a + wide;
        const unsigned dheads = __ballot_sync(0xffffffffu, dub);
        unsigned doubt = 0u;
        for (unsigned left = dheads; left; left &= left - 1) doubt |= 1u << ((__ffs(left) - 1) >> s.span_log2);
        const int want = s.topk_groups - __popc(keep & ~dheads);
        unsigned cand = 0u;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int eg = group_of(s, min(e0 + i, E - 1));
          const float lw = __shfl_sync(0xffffffffu, low, eg * span);
          const float thr = s.bias ? lw - 2.f * (perr + 2.5e-7f * fabsf(lw)) : lw;
          if (e0 + i < E && ((doubt >> eg) & 1u) && !(c[i] < thr)) cand |= 1u << i;
        }
        int* list = reinterpret_cast<int*>(sm);
        const int total = list_candidates(cand, e0, list);
        unsigned kept = 0u;
        if (total <= 32) {
          F2 z2 = {1.f, 0.f};
          if (!s.sigmoid) z2 = softmax_f2<VPL>(row, E, m);
          kept = fine_groups(row, gsz, s, m, z2, list, total, doubt, want);
        }
        __syncwarp();
        unsure_groups = kept == 0u;
        keep &= ~dheads;
        for (; kept; kept &= kept - 1) keep |= 1u << ((__ffs(kept) - 1) * span);
      }
    }
    // the dropped groups' experts leave: -infinity, and not eligible
    if (whole) {
      if (!((keep >> (g * span)) & 1u)) {
        elig = 0u;
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) c[i] = -INFINITY;
      }
    } else {
      top = -INFINITY;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (e0 + i < E && !((keep >> (group_of(s, e0 + i) * span)) & 1u)) {
          c[i] = -INFINITY;
          elig &= ~(1u << i);
        }
        top = fmaxf(top, c[i]);
      }
    }
  }
  int mine = 0;
  if (unsure_groups) {
    mine = score_exact_all<VPL>(row, E, k, s);
  } else {
    // `need` scores in order: the k chosen, and with a bias the next one. The
    // lanes' need-th largest maximum bounds them from below.
    const int need = s.bias ? k + 1 : k;
    // (equal maxima count once: the bound is then lower, the list longer)
    uint32_t tk = need <= 32 ? order_key(top) : 0u, bk = 0u;
#pragma unroll 4
    for (int j = 0; j < need; ++j) {
      bk = __reduce_max_sync(0xffffffffu, tk);
      if (tk == bk) tk = 0u;
    }
    const float bound = bk ? key_value(bk) : -INFINITY;
    int* list = reinterpret_cast<int*>(sm);
    uint32_t* lkey = reinterpret_cast<uint32_t*>(sm) + 32;
    int total = 33;
    if (bound > -INFINITY) {
      unsigned cand = 0u;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (c[i] >= bound) cand |= 1u << i;
      total = list_candidates(cand, e0, list);
    }
    uint32_t my_key = 0u, next_key = 0u;
    if (total <= 32) {
      // the list's order: rank by key, then by place
      const int e = lane < total ? list[lane] : 0;
      uint32_t ck = 0u;
      if (lane < total) {
        const float v = clean_logit(__ldg(row + e));
        ck = order_key(s.bias ? __fadd_rn(score_prob(s, v, m, rz), score_bias(s, e)) : v);
      }
      int r = 0;
#pragma unroll 4
      for (int j = 0; j < total; ++j) {
        const uint32_t o = __shfl_sync(0xffffffffu, ck, j);
        r += o > ck || (o == ck && j < lane);
      }
      __syncwarp();
      if (lane < total) {
        list[r] = e;
        lkey[r] = ck;
      }
      __syncwarp();
      if (lane < total) {
        mine = list[lane];
        my_key = lkey[lane];
      }
      __syncwarp();
      next_key = __shfl_down_sync(0xffffffffu, my_key, 1);
      if (lane == 31) next_key = 0u;
    } else {
      // many equal scores, fewer open ones than needed, few lanes, or k near 32
      mine = choose_in_rounds<VPL>(row, E, s, m, rz, elig, need, my_key, next_key);
    }
    if (s.bias) {
      // neighbours in the order: equal infinities are certain (closed
      // experts, by index)
      const float a = key_value(my_key), b = key_value(next_key);
      const bool close = lane < k && next_key != 0u && !(isinf(a) && a == b) &&
                         !(a - b > perr + 2.5e-7f * fmaxf(fabsf(a), fabsf(b)));
      if (__any_sync(0xffffffffu, close)) {
        const float vk = key_value(__shfl_sync(0xffffffffu, my_key, k - 1));
        const float thr = vk - 2.f * (perr + 2.5e-7f * fabsf(vk));
        unsigned cand = 0u;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (((elig >> i) & 1u) && !(c[i] < thr)) cand |= 1u << i;
        const int n = list_candidates(cand, e0, list);
        int fine = -1;
        if (n <= 32) {
          F2 z2 = {1.f, 0.f};
          if (!s.sigmoid) z2 = softmax_f2<VPL>(row, E, m);
          fine = fine_order(row, k, s, m, z2, list, n);
        }
        mine = fine >= 0 ? fine : score_exact_all<VPL>(row, E, k, s);
      }
    }
  }
  // the chosen experts' weights, lane j the j-th
  float lj = -INFINITY;
  bool open = false;
  if (lane < k) {
    lj = clean_logit(__ldg(row + mine));
    open = !s.bias || score_bias(s, mine) > -INFINITY;
  }
  float pj = 0.f;
  if (s.renorm) {
    // relative to the largest chosen logit, so that no sum underflows; a sigmoid
    // below -20 is the exponential, to 2e-9. An exponential below -745 (masks
    // of the type's lowest value) is 0 in 64 bits too; under softmax its argument
    // is from the row's maximum, which is among the chosen without bias and groups
    const float best = key_value(__reduce_max_sync(0xffffffffu, order_key(open ? lj : -INFINITY)));
    const float arg = s.sigmoid ? best : s.bias || s.groups > 1 ? best - m : 0.f;
    if (open && best > -INFINITY && arg > -745.f) {
      if (s.sigmoid) pj = lj > -20.f ? 1.0f / (1.0f + expf(-lj)) : expf(best > -20.f ? lj : lj - best);
      else if (!isinf(best) && rz > 0.f) pj = expf(lj - best);
    }
    float sum = pj;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    pj = sum > 0.f ? pj / sum : 0.f;
  } else if (open) {
    pj = score_prob(s, lj, m, rz);
  }
  idx = mine;
  w = pj * s.scale;
}

}  // namespace moe
