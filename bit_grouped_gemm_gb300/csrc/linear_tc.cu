// linear_tc.cu -- the projection's product for more than a decode batch, on
// pairs of SMs (tcgen05 cta_group::2):
//   y[t][n] = x_scale[t] (sum_k x16[t][k] W16[n][k] + sum_r h[t][r] B[a_t][n][r])
// from the fp16 rows, the fp16 weights and the adapters' h = scale x A^T that
// the launch before it wrote (w4_linear.cu).
//
// A tile is 256 tokens x BN outputs; each CTA of the pair holds 128 token rows
// (operand A) and BN / 2 weight rows (operand B), and its 128 rows of the
// accumulator, of which TMEM holds two, so that a tile's epilogue runs under
// the next tile's MMAs. K goes by in chunks of 64.
//
// The adapters are more columns of K. For every adapter that occurs among the
// tile's tokens the tile gets rank K columns with h in A, zero in the rows of
// other tokens, and B[a] in B: the MMAs then add each token's own product,
// whatever the order of the tokens. They go by in stages of 16 columns, written
// by two groups of four warps and spread between the tile's other chunks. h goes in as two
// bf16 (the value and what its rounding left), each multiplied with B's own
// bf16: the products are exact to 16 bits of h. A zero times an infinity or a NaN
// would carry one adapter's broken B into other requests' rows, so B goes in with
// these as the largest bf16 (which is why it does not come by TMA): zero times
// that is zero, and in the adapter's own rows no ordinary number is left.
//
// Every wait is bounded, as in gemm_tc2.cu.
//
// Bound by the tensor cores at many tokens: 4096 x 2048 x 4096 44.1 us without
// adapters (1.56 PFLOP/s, conversion included), 53.2 with 8 of rank 32; the
// product alone 47 us cold (77% of the tensor pipe's time). Below 1000 tokens by
// latency: 128 x 2048 x 2048 13.6 us, of which conversion and product each wait
// for a ring of copies to fill.
#include "pair.cuh"

namespace moe {
namespace lin {

constexpr int kThreads = 480;             // TMA, 1 or 2 MMA, 2 x 4 adapter, 4 epilogue warps
constexpr int kMma2Warp = 10, kLora2Warp = 11;
constexpr int kTileM = 256;
constexpr int kOpBytes = 128 * 128;       // 128 rows x 64 16-bit columns
constexpr uint32_t kTmemCols = 512;

// An adapter stage: h and its rest (A, 128 rows x 16 bf16 each), B's BN / 2
// rows. Narrow tiles leave shared memory for four of them, where a full tile has
// two, and need them: a pair has one such tile, whose adapters all come at once.
constexpr int kLoraTile = 128 * 32;
constexpr int kMaxLoraStages = 4;

// Shared memory: the ring of operand chunks, the adapter stages, ids and runs and
// list of the tile's adapters, barriers. A copy takes up to 4,500 cycles to
// land, so a tile's pace is the ring's depth over that until its MMAs are slower:
// narrow tiles get as many chunks as fit.
constexpr int kIdsBytes = 2 * 3 * kTileM * 4;
constexpr int kBarBytes = 512;
constexpr int kSmemMax = 227 * 1024 - 1024;   // less alignment slack
constexpr int kMaxStages = 12;
inline int stage_bytes(int bn) { return kOpBytes + (bn / 2) * 128; }
inline int lora_stage_bytes(int bn) { return 2 * kLoraTile + (bn / 2) * 32; }

struct Params {
  CUtensorMap mx;       // x16 [rows][K], boxes 64 x 128
  CUtensorMap mw;       // W16 [N][K], boxes 64 x BN / 2
  LinearArgs a;
  int bn, mt, tiles;    // tile width, token tiles, all tiles
  int split;            // pairs per tile, each a part of K (a cluster is 2 x split CTAs)
  int stages, stage_bytes, lora_stages, lora_stage_bytes;
  DevErr err;
};

// Whole-warp bounded wait. kCluster: with the acquire over the cluster that the
// other CTA's own stores need; copies and MMAs that complete on the barrier do
// not, and the narrower one is cheaper.
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          const DevErr& err, int site) {
  auto look = [&](uint32_t hint) {
    if constexpr (kCluster) return try_wait_cluster(bar, parity, hint);
    else return hint ? mbar_try_wait_sleep(bar, parity, hint) : mbar_try_wait(bar, parity);
  };
  bool ok = look(0);
  if (!__all_sync(0xffffffffu, ok)) {
    const unsigned long long t0 = globaltimer_ns();
    while (!ok) {
      ok = look(100000);
      if (ok || *abort_flag || globaltimer_ns() - t0 > err.limit_ns) break;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
      if ((threadIdx.x & 31) == 0 && !*abort_flag) report_timeout(err, site);
      *abort_flag = 1;
    }
  }
  return ok;
}

__device__ __forceinline__ int token_adapter(const LinearArgs& a, int t) {
  const int id = t < a.T ? __ldcg(a.adapter + t) : -1;
  return (unsigned)id < (unsigned)a.n_adapters ? id : -1;
}

// Operand descriptor of a tile of 16 K columns: K-major, 32-byte rows with
// 32-byte swizzle (a row's two 16-byte halves change places in rows 4..7 of
// every 8), 8-row groups 256 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_sw32(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);        // start address
  d |= static_cast<uint64_t>(1u) << 16;                           // LBO (unused)
  d |= static_cast<uint64_t>(256u >> 4) << 32;                    // SBO: 8 rows * 32 B
  d |= static_cast<uint64_t>(1u) << 46;                           // descriptor version
  d |= static_cast<uint64_t>(6u) << 61;                           // 32-byte swizzle
  return d;
}

// Two bf16 with infinities and NaNs as the largest finite value of their sign.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  const uint32_t no = __vcmpeq2(w & 0x7F807F80u, 0x7F807F80u);
  return (w & ~(no & 0x7FFF7FFFu)) | (no & 0x7F7F7F7Fu);
}

// Barrier of the 128 adapter threads that tells whether all of them go on, so
// that they leave their loop together and none is waited for in vain.
__device__ __forceinline__ bool bar_and(int bar, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.and.pred q, %2, 128, p;\n"
      " selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(bar)
      : "memory");
  return r != 0;
}

// Instruction descriptor with bf16 operands (else as idesc_f16_f32).
__device__ __forceinline__ uint32_t idesc_bf16(int M, int N) {
  return idesc_f16_f32(M, N) | (1u << 7) | (1u << 10);
}

__device__ __forceinline__ void bar_sync(int bar) {
  asm volatile("bar.sync %0, 128;" ::"r"(bar) : "memory");
}

// Places of the flagged entries among 256 (thread i of 128 holds entries i
// and 128 + i) in their order, and their number. `cnt`: 8 ints.
__device__ __forceinline__ int rank_of(int bar, bool a, bool b, int i, int* cnt, int& ra, int& rb) {
  const int lane = i & 31, w = i >> 5;
  const unsigned ma = __ballot_sync(0xffffffffu, a), mb = __ballot_sync(0xffffffffu, b);
  if (lane == 0) {
    cnt[w] = __popc(ma);
    cnt[4 + w] = __popc(mb);
  }
  bar_sync(bar);
  int n = 0;
  ra = rb = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j == w) ra = n + __popc(ma & ((1u << lane) - 1u));
    if (j == 4 + w) rb = n + __popc(mb & ((1u << lane) - 1u));
    n += cnt[j];
  }
  bar_sync(bar);
  return n;
}

// kIssuers: MMA warps, 2 where a pair has one tile, else 1.
template <bool kLora, int kIssuers>
__global__ void __launch_bounds__(kThreads, 1)
    linear_tc_kernel(const __grid_constant__ Params p) {
  const int stages = p.stages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024 - (raw_addr & 1023)) & 1023);
  uint8_t* lora = smem + stages * p.stage_bytes;
  int* s_lora = reinterpret_cast<int*>(lora + p.lora_stages * p.lora_stage_bytes);   // adapter lists
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_lora + (kLora ? 2 * 3 * kTileM : 0));
  uint64_t* full = bars;                   // leader: both CTAs' operands landed
  uint64_t* empty = full + kMaxStages;              // chunk's MMAs done (both CTAs)
  uint64_t* acc_full = empty + kMaxStages;          // [2] tile's MMAs done (both CTAs)
  uint64_t* acc_empty = acc_full + 2;      // [2] leader: accumulator read by 8 warps
  uint64_t* lora_full = acc_empty + 2;     // leader: both CTAs wrote their adapter stage
  uint64_t* lora_empty = lora_full + kMaxLoraStages;   // adapter stage's MMAs done (both CTAs)
  uint64_t* list_full = lora_empty + kMaxLoraStages;   // [2] leader: the tile's adapter stages are known
  uint64_t* drain = list_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* s_steps = reinterpret_cast<volatile int*>(tmem_slot + 2);   // [2] by tile parity
  int* s_cnt2 = reinterpret_cast<int*>(tmem_slot + 4);      // [2][8] flagged entries per warp

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // CTA `rank` of pair `part` of the cluster; the pair's leader is its CTA 0
  const uint32_t crank = cluster_rank(), rank = crank & 1u, lead = crank & ~1u;
  const int part = (int)(crank >> 1), split = p.split;
  const bool leader = rank == 0;
  const int pair = (int)blockIdx.x / (2 * split), npairs = (int)gridDim.x / (2 * split);   // clusters
  auto leader_addr = [&](const void* q) { return cta_addr(q, lead); };
  auto commit_both = [&](uint64_t* bar) { mma2_commit_mask(bar, (uint16_t)(3u << lead)); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], kIssuers);
      mbar_init(&acc_empty[i], 8);
      mbar_init(&list_full[i], 1);
    }
    for (int i = 0; i < p.lora_stages; ++i) {
      mbar_init(&lora_full[i], 2);
      mbar_init(&lora_empty[i], 1);
    }
    mbar_init(drain, kIssuers);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.mx);
    tma_prefetch_desc(&p.mw);
  }
  if (warp == 1) tmem_alloc2(tmem_slot, kTmemCols);
  tc_fence_before();
  cluster_sync_all();   // barriers and TMEM of both CTAs, before any remote arrival
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // What the launch before wrote (x16, W16, h) is read after pdl_wait; the
  // adapters' ids and the rows' scales are older, as that launch waited for all
  // before it, and are read through L2.

  // this pair's chunks of K
  const int nk_all = p.a.K / 64, c_lo = part * nk_all / split, nk = (part + 1) * nk_all / split - c_lo;
  const int half = p.bn >> 1;
  const int rb = (p.a.rank + 15) >> 4;   // stages per adapter

  // warps 2 to 9: this thread's row of the tile at token place m0, its token in y
  // and scale (read where the parts' sums meet by the adapter warps too)
  bool live = false;
  int y_row = 0;
  float y_scale = 1.f;
  auto set_row = [&](int m0) {
    const int place = m0 + 128 * (int)rank + 32 * (warp & 3) + lane;
    live = place < p.a.T;
    y_row = live && kLora ? __ldcg(p.a.order + place) : place;
    if (live && p.a.x_scale) y_scale = __ldcg(p.a.x_scale + y_row);
  };

  if (warp == 0) {
    // ---------------------------------------------------- TMA, own halves
    pdl_begin();
    const uint32_t bytes = 2u * (kOpBytes + (uint32_t)half * 128u);   // of both CTAs
    int s = 0;
    uint32_t ph = 1;   // slot and the parity of its barrier's last phase
    bool ok = true;
    for (int u = pair; u < p.tiles && ok; u += npairs) {
      const int m0 = (u % p.mt) * kTileM + 128 * (int)rank;
      const int n0 = (u / p.mt) * p.bn + half * (int)rank;
      for (int c = 0; c < nk; ++c) {
        if (!(ok = warp_wait(&empty[s], ph, abort_flag, p.err, 80))) break;
        if (elect_one_sync()) {
          uint8_t* dst = smem + s * p.stage_bytes;
          if (leader) mbar_arrive_expect_tx(&full[s], bytes);
          tma_load_2d_pair(dst, &p.mx, 64 * (c_lo + c), m0, leader_addr(&full[s]));
          tma_load_2d_pair(dst + kOpBytes, &p.mw, 64 * (c_lo + c), n0, leader_addr(&full[s]));
        }
        __syncwarp();
        if (++s == stages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    if (!ok) {
      // Gave up: the copies in flight land on the leader's barriers, which the
      // other CTA cannot wait on; both leave them a millisecond.
      const unsigned long long t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
    }
  } else if (warp == 1 || warp == kMma2Warp) {
    // ------------------------------------------------- MMA issuers, leader
    // Issuing a chunk (a wait, four MMAs, a commit) takes a warp about 450
    // cycles, the MMAs themselves 2 cycles per column. With one tile per pair
    // both accumulators are free for it, so two warps take alternate chunks,
    // and alternate adapter stages, into one each, and the epilogue adds them.
    const int me = warp == 1 ? 0 : 1;
    if (leader && me < kIssuers) {
      const uint64_t ring_desc = smem_desc_sw128(smem_u32(smem));
      const uint32_t idesc = idesc_f16_f32(256, p.bn), idesc_l = idesc_bf16(256, p.bn);
      uint32_t it = 0;
      int s = me, ls = me;
      uint32_t ph = 0, lph = 0;
      if (s >= stages) s -= stages, ph ^= 1;
      bool ok = true;
      for (int u = pair; u < p.tiles && ok; u += npairs, ++it) {
        const int buf = kIssuers == 2 ? me : (int)(it & 1);
        const uint32_t acc = tmem + 256 * buf;
        if (kIssuers == 1 && !(ok = warp_wait<true>(&acc_empty[buf], ((it >> 1) & 1) ^ 1, abort_flag, p.err, 82))) break;
        tc_fence_after();
        int c = me;
        auto chunk = [&] {
          if (!(ok = warp_wait(&full[s], ph, abort_flag, p.err, 83))) return;
          tc_fence_after();
          if (elect_one_sync()) {
            // (a descriptor's low bits are the address over 16)
            const uint64_t ad = ring_desc + (uint32_t)(s * p.stage_bytes >> 4), bd = ad + (kOpBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma2_f16_ss(acc, ad + 2 * kk, bd + 2 * kk, idesc, (c != me) | (kk != 0));
            commit_both(&empty[s]);
          }
          __syncwarp();
          s += kIssuers;
          if (s >= stages) {
            s -= stages;
            ph ^= 1;
          }
        };
        // The adapter stages come evenly among the second half's chunks (fixed
        // places: the sums' order is that of every run). The first tile's list takes
        // about a microsecond and is waited for there (4096 tokens of 2048 x 2048:
        // 35.9 us, 36.9 with the wait before the first chunk).
        int nl = 0, j = me;
        if (kLora) {
          if (it == 0)
            for (; c + 1 < nk / 2 && ok; c += kIssuers) chunk();
          if (ok) ok = warp_wait(&list_full[it & 1], (it >> 1) & 1, abort_flag, p.err, 81);
          if (!ok) break;
          nl = s_steps[it & 1];
        }
        // the chunks between two of this warp's stages, and before the next one
        const int gap = nl ? (nk - nk / 2) / (nl + 1) : 0;
        int due = nk / 2 + gap * (me + 1);
        for (; c < nk; c += kIssuers) {
          chunk();
          if (!ok) break;
          while (kLora && j < nl && (c + 1 >= due || c + kIssuers >= nk)) {
            if (!(ok = warp_wait<true>(&lora_full[ls], lph, abort_flag, p.err, 84))) break;
            tc_fence_after();
            if (elect_one_sync()) {
              const uint32_t base = smem_u32(lora + ls * p.lora_stage_bytes);
              const uint64_t bd = smem_desc_sw32(base + 2 * kLoraTile);
              mma2_f16_ss(acc, smem_desc_sw32(base), bd, idesc_l, 1);
              mma2_f16_ss(acc, smem_desc_sw32(base + kLoraTile), bd, idesc_l, 1);
              commit_both(&lora_empty[ls]);
            }
            __syncwarp();
            ls += kIssuers;
            if (ls >= p.lora_stages) {
              ls -= p.lora_stages;
              lph ^= 1;
            }
            j += kIssuers;
            due += gap * kIssuers;
          }
          if (!ok) break;
        }
        if (!ok) break;
        if (elect_one_sync()) commit_both(&acc_full[kIssuers == 2 ? 0 : it & 1]);
        __syncwarp();
      }
      if (elect_one_sync()) commit_both(drain);
      __syncwarp();
    }
    // every MMA that reads this CTA's memory is done before it is released
    const unsigned long long t0 = globaltimer_ns();
    while (!try_wait_cluster(drain, 0, 100000) && globaltimer_ns() - t0 < 2 * p.err.limit_ns) {
    }
  } else if (warp < 6 || warp >= kLora2Warp) {
    // ------------------------------------------------- adapters' K columns
    if (!kLora) {
      if (split > 1) set_row((pair % p.mt) * kTileM);
    } else {
      // Two groups of four warps write alternate stages: one takes about 800
      // cycles to fill one (its barriers and proxy fence), a stage's MMAs 256
      // (128 tokens of 16 adapters, K = N = 2048: 19.7 us, with one group 21.7).
      const int grp = warp < 6 ? 0 : 1, bar = 1 + grp;
      const int i = threadIdx.x - (grp ? 32 * kLora2Warp : 64);   // 0..127: this thread's A row
      int* s_ids = s_lora + 3 * kTileM * grp;          // the tile's adapter per token
      int* s_runs = s_ids + kTileM;                    // its runs' adapters
      int* s_list = s_runs + kTileM;                   // its distinct adapters
      int* s_cnt = s_cnt2 + 8 * grp;
      int r0, r1;
      uint32_t sc = 0, it = 0;   // stages of the tiles before
      bool ok = true;
      for (int u = pair; u < p.tiles && ok; u += npairs, ++it) {
        const int m0 = (u % p.mt) * kTileM, n0 = (u / p.mt) * p.bn;
        // Are its places ordered? For the first tile found out here, as the launch
        // before does, to have the list while that still runs.
        bool ordered = true;
        if (it == 0) {
          const int blk0 = m0 / kOrderBlock * kOrderBlock, n = min(kOrderBlock, p.a.T - blk0);
          static_assert(kOrderSamples == 128, "a sample per thread");
          const int at = order_sample(i, n);
          const unsigned changes = __ballot_sync(0xffffffffu, at < n && token_adapter(p.a, blk0 + at - 1) !=
                                                                            token_adapter(p.a, blk0 + at));
          if (lane == 0) s_cnt[i >> 5] = __popc(changes);
          bar_sync(bar);
          ordered = order_rule(s_cnt[0] + s_cnt[1] + s_cnt[2] + s_cnt[3], n);
          if (ordered) pdl_wait();
        }
        // the tile's distinct adapters, in the order of their first tokens
        auto adapter_at = [&](int place) {
          if (place >= p.a.T) return -1;
          return token_adapter(p.a, ordered ? __ldcg(p.a.order + place) : place);
        };
        const int id0 = adapter_at(m0 + i), id1 = adapter_at(m0 + 128 + i);
        s_ids[i] = id0;
        s_ids[128 + i] = id1;
        bar_sync(bar);
        // where an adapter's run of tokens starts, then its first run
        const bool st0 = id0 >= 0 && (i == 0 || s_ids[i - 1] != id0);
        const bool st1 = id1 >= 0 && s_ids[127 + i] != id1;
        const int runs = rank_of(bar, st0, st1, i, s_cnt, r0, r1);
        if (st0) s_runs[r0] = id0;
        if (st1) s_runs[r1] = id1;
        bar_sync(bar);
        bool f0 = i < runs, f1 = 128 + i < runs;
        const int ru0 = f0 ? s_runs[i] : -1, ru1 = f1 ? s_runs[128 + i] : -1;
        const int upto = f1 ? 128 + i : i;
        if (f0)
          for (int e = 0; e < upto; e += 4) {
            const int4 o = *reinterpret_cast<const int4*>(s_runs + e);
            f0 &= !((o.x == ru0 && e < i) || (o.y == ru0 && e + 1 < i) || (o.z == ru0 && e + 2 < i) ||
                    (o.w == ru0 && e + 3 < i));
            f1 &= !((o.x == ru1 && e < upto) || (o.y == ru1 && e + 1 < upto) ||
                    (o.z == ru1 && e + 2 < upto) || (o.w == ru1 && e + 3 < upto));
          }
        const int nad = rank_of(bar, f0, f1, i, s_cnt, r0, r1);
        if (f0) s_list[r0] = ru0;
        if (f1) s_list[r1] = ru1;
        // of the tile's rb x nad stages every split-th is this pair's
        const int nl = (rb * nad - part + split - 1) / split;
        // The count of two tiles ago has been read once that tile is done. Only the
        // leader's first group looks, whose count the issuer waits for: for the
        // others, with no stage in a tile, nothing keeps that barrier from going on
        // past the phase they would wait for.
        const bool counts = leader && grp == 0;
        if (it >= 2 && counts) ok = warp_wait(&acc_full[it & 1], ((it >> 1) & 1) ^ 1, abort_flag, p.err, 85);
        if (!(ok = bar_and(bar, ok))) break;
        if (i == 0 && counts) {
          s_steps[it & 1] = nl;
          mbar_arrive(&list_full[it & 1]);
        }
        const int my_id = rank ? id1 : id0;
        const float* hrow = p.a.h + (size_t)min(m0 + 128 * (int)rank + i, p.a.T - 1) * p.a.rank;
        // the tile's stage g: columns 16 (g % rb) .. + 15 of adapter g / rb of
        // the list; this thread's h is loaded a stage ahead
        float4 v[4], nv[4];
        uint4 nb0, nb1;   // and B's row of this thread
        const int brow = n0 + half * (int)rank + i;
        auto load_h = [&](int j) {
#pragma unroll
          for (int e = 0; e < 4; ++e) nv[e] = make_float4(0.f, 0.f, 0.f, 0.f);
          nb0 = nb1 = make_uint4(0u, 0u, 0u, 0u);
          if (j >= nl) return;
          const int gj = part + j * split, ad = s_list[gj / rb], c = 16 * (gj % rb);
          if (i < half && brow < p.a.N) {
            const uint4* b4 = reinterpret_cast<const uint4*>(p.a.lb + ((size_t)ad * p.a.N + brow) * p.a.rank + c);
            nb0 = __ldg(b4);
            if (c + 16 <= p.a.rank) nb1 = __ldg(b4 + 1);
          }
          if (ad == my_id) {
            const float4* h4 = reinterpret_cast<const float4*>(hrow + c);
            nv[0] = __ldcg(h4);
            nv[1] = __ldcg(h4 + 1);
            if (c + 16 <= p.a.rank) {
              nv[2] = __ldcg(h4 + 2);
              nv[3] = __ldcg(h4 + 3);
            }
          }
        };
        if (it == 0) {
          pdl_wait();
          if (split > 1) set_row(m0);
        }
        // (by the count of all stages: with an even number of buffers a group then
        // has buffers of its own and meets each of their phases)
        const int j0 = (grp ^ (int)sc) & 1;
        load_h(j0);
        for (int j = j0; j < nl; j += 2) {
          const uint32_t lcnt = sc + j;
          const int ls = lcnt % p.lora_stages;
          uint8_t* stage = lora + ls * p.lora_stage_bytes;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = nv[e];
          const uint4 b0 = nb0, b1 = nb1;
          load_h(j + 2);
          if (lcnt >= (uint32_t)p.lora_stages)
            ok = warp_wait(&lora_empty[ls], ((lcnt / p.lora_stages) & 1) ^ 1, abort_flag, p.err, 86);
          if (!(ok = bar_and(bar, ok))) break;
          const float f[16] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w,
                               v[2].x, v[2].y, v[2].z, v[2].w, v[3].x, v[3].y, v[3].z, v[3].w};
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            hi[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
            lo[e] = pack_bf16x2(f[2 * e] - bf16_lo(hi[e]), f[2 * e + 1] - bf16_hi(hi[e]));
          }
          uint8_t* row = stage + i * 32;
          const int sw = ((i >> 2) & 1) << 4;
          *reinterpret_cast<uint4*>(row + sw) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(row + (16 ^ sw)) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
          *reinterpret_cast<uint4*>(row + kLoraTile + sw) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          *reinterpret_cast<uint4*>(row + kLoraTile + (16 ^ sw)) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
          if (i < half) {
            *reinterpret_cast<uint4*>(row + 2 * kLoraTile + sw) =
                make_uint4(finite2(b0.x), finite2(b0.y), finite2(b0.z), finite2(b0.w));
            *reinterpret_cast<uint4*>(row + 2 * kLoraTile + (16 ^ sw)) =
                make_uint4(finite2(b1.x), finite2(b1.y), finite2(b1.z), finite2(b1.w));
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          bar_sync(bar);
          if (i == 0) arrive_cluster_shared(leader_addr(&lora_full[ls]));
        }
        sc += nl;
        // (the next tile rewrites the list: every thread has read it)
        if (!bar_and(bar, ok)) break;
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    pdl_wait();   // (y may still be read by an older launch)
    const int quarter = warp & 3, row = 32 * quarter + lane;
    const uint32_t lane_base = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t acc_empty_l = leader_addr(acc_empty);
    const bool wide = (p.a.y_ld & 7) == 0 && (reinterpret_cast<uintptr_t>(p.a.y) & 15u) == 0;
    uint32_t it = 0;
    bool ok = true;
    for (int u = pair; u < p.tiles && ok; u += npairs, ++it) {
      const int n0 = (u / p.mt) * p.bn;
      set_row((u % p.mt) * kTileM);
      if (!(ok = warp_wait(&acc_full[it & 1], (it >> 1) & 1, abort_flag, p.err, 87))) break;
      tc_fence_after();
      for (int c0 = 0; c0 < p.bn; c0 += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tmem + lane_base + 256 * (it & 1) + c0, v);
        tmem_wait_ld();
        if (kIssuers == 2) {
          uint32_t v2[32];
          tmem_ld_32x32b_x32(tmem + lane_base + 256 + c0, v2);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            v[e] = __float_as_uint(__uint_as_float(v[e]) + __uint_as_float(v2[e]));
        }
        if (c0 + 32 >= p.bn) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_cluster_relaxed(acc_empty_l + 8 * (it & 1));
        }
        const int n = n0 + c0;
        uint16_t* o = p.a.y + y_row * p.a.y_ld + n;
        if (split > 1) {
          // this part's sums, [column][row], where the operands were (all
          // of the pair's MMAs are done)
          float* sums = reinterpret_cast<float*>(smem) + c0 * 128 + row;
#pragma unroll
          for (int e = 0; e < 32; ++e) sums[128 * e] = __uint_as_float(v[e]);
        } else if (!live) {
        } else if (wide && n + 32 <= p.a.N) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16x2(__uint_as_float(v[8 * q + 2 * e]) * y_scale,
                                 __uint_as_float(v[8 * q + 2 * e + 1]) * y_scale);
            reinterpret_cast<uint4*>(o)[q] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (n + e < p.a.N) o[e] = f32_to_bf16(__uint_as_float(v[e]) * y_scale);
        }
        __syncwarp();
      }
    }
  }
  if (split > 1) {
    // The parts' sums, added in order over distributed shared memory: pair
    // `part` writes columns part x BN / split .. of the tile, 8 warps of a CTA
    // a quarter of its rows and half of these columns each.
    __syncthreads();
    cluster_sync_all();
    if (warp >= 2 && warp < 10 && !*abort_flag) {
      const int row = 32 * (warp & 3) + lane;
      const int cols = p.bn / split, n0 = (pair / p.mt) * p.bn;
      const bool wide = (p.a.y_ld & 7) == 0 && (reinterpret_cast<uintptr_t>(p.a.y) & 15u) == 0;
      const int c_end = part * cols + (warp >= 6 ? cols : cols / 2);
      for (int c0 = part * cols + (warp >= 6 ? cols / 2 : 0); c0 < c_end; c0 += 16) {
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
        for (int q = 0; q < split; ++q) {
          const uint32_t src = cta_addr(reinterpret_cast<float*>(smem) + c0 * 128 + row, 2 * q + rank);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float o;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o) : "r"(src + 512u * e) : "memory");
            v[e] += o;
          }
        }
        const int n = n0 + c0;
        uint16_t* o = p.a.y + y_row * p.a.y_ld + n;
        if (!live) {
        } else if (wide && n + 16 <= p.a.N) {
#pragma unroll
          for (int q = 0; q < 2; ++q)
            reinterpret_cast<uint4*>(o)[q] =
                make_uint4(pack_bf16x2(v[8 * q] * y_scale, v[8 * q + 1] * y_scale),
                           pack_bf16x2(v[8 * q + 2] * y_scale, v[8 * q + 3] * y_scale),
                           pack_bf16x2(v[8 * q + 4] * y_scale, v[8 * q + 5] * y_scale),
                           pack_bf16x2(v[8 * q + 6] * y_scale, v[8 * q + 7] * y_scale));
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (n + e < p.a.N) o[e] = f32_to_bf16(v[e] * y_scale);
        }
      }
    }
  }
  __syncthreads();
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc2(tmem, kTmemCols);
  }
}

}  // namespace lin

// Tile width and parts of K, by estimated cycles: rounds of tiles over the
// pairs, each chunk at the slowest of its MMAs (2 cycles per column), its issue
// (300), its operands' copies at 75 bytes per cycle into an SM, and at 8000 out
// of L2. Of tiles that come out alike the widest is taken: fewer CTAs then read
// the same lines. Measured for the call at K = 2048 with 8 adapters of rank 16
// (widths 64, 128, 192, 224, 256): 512 x 2048 16.0, 15.2 (96: 14.8), 17.2, 18.6,
// 20.1 us; 1024 x 2048 26.7, 17.4 (160: 17.4), 18.3, 19.5, 20.9; 4096 x 2048 70.1,
// 46.0, 39.1, 39.8, 34.8; 4096 x 4096, e4m3 of rank 32, 132.0, 73.6, 58.9, 52.9,
// 54.4.
// With few tiles, two pairs of a cluster take half of K each, for the exchange of
// their sums: 128 x 2048 13.6 against 14.9 us, 200 x 1000 at K = 4096 19.9
// against 23.8; but 512 x 2048 16.4 against 15.2. (Four pairs: 19.2 against 12.3
// at 128 x 2048 without adapters; the device holds 15 clusters of 8 such CTAs.)
static void linear_shape(int T, int N, int K, int num_sms, int* bn_out, int* split_out) {
  const int mt = (T + lin::kTileM - 1) / lin::kTileM, pairs = num_sms / 2, nk = K / 64;
  double cost = 1e30;
  for (int split = 1; split <= 2; ++split)
    for (int bn = 256; bn >= 32; bn -= 32) {
      const long long tiles = (long long)mt * ((N + bn - 1) / bn);
      if (split > 1 && (bn % 64 || nk < 4 || tiles > 32)) continue;
      const double bytes = 16384.0 + 64.0 * bn, sms = 2.0 * fmin((double)(tiles * split), (double)pairs);
      const double chunk = fmax(fmax(2.0 * bn, 300.0), fmax(bytes / 75.0, bytes * sms / 8000.0));
      const double c = (double)((tiles + pairs - 1) / pairs) * chunk * ((nk + split - 1) / split) +
                       (split > 1 ? 1500.0 + 21.0 * bn : 0.0);
      if (c < cost * 0.97) {
        cost = c;
        *bn_out = bn;
        *split_out = split;
      }
    }
}

cudaError_t launch_linear_tc(const LinearArgs& a, const CUtensorMap& mx, const CUtensorMap* mw,
                             DevErr err, int num_sms, cudaStream_t st) {
  int bn = 256, split = 1;
  linear_shape(a.T, a.N, a.K, num_sms, &bn, &split);
  lin::Params p;
  p.mx = mx;
  p.mw = mw[bn / 32 - 1];
  p.split = split;
  p.a = a;
  p.bn = bn;
  p.mt = (a.T + lin::kTileM - 1) / lin::kTileM;
  p.tiles = p.mt * ((a.N + bn - 1) / bn);
  p.err = err;
  int clusters = split > 1 ? p.tiles : num_sms / 2;
  if (clusters > p.tiles) clusters = p.tiles;
  const bool two = p.tiles <= clusters && a.K >= 2 * 64 * split;
  p.stage_bytes = lin::stage_bytes(bn);
  p.lora_stage_bytes = lin::lora_stage_bytes(bn);
  // two adapter stages at least, four where the tile is narrow
  p.lora_stages = a.la ? (bn > 128 ? 2 : lin::kMaxLoraStages) : 0;   // (even: a group of writers each)
  const int fixed = (a.la ? lin::kIdsBytes : 0) + lin::kBarBytes + p.lora_stages * p.lora_stage_bytes;
  p.stages = (lin::kSmemMax - fixed) / p.stage_bytes;
  if (p.stages > lin::kMaxStages) p.stages = lin::kMaxStages;
  const int smem = fixed + p.stages * p.stage_bytes + 1024;
  auto go = [&](auto kern) {
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * split * clusters);
    cfg.blockDim = dim3(lin::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
  };
  return a.la ? (two ? go(lin::linear_tc_kernel<true, 2>) : go(lin::linear_tc_kernel<true, 1>))
              : (two ? go(lin::linear_tc_kernel<false, 2>) : go(lin::linear_tc_kernel<false, 1>));
}

}  // namespace moe
