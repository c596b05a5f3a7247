// page_map.cu -- block tables, slots, positions and ancestor masks of a batch's
// new tokens, from request lengths that only the device knows (moe_page_map).
//
// Two prefix sums over the requests (rows; pages needed and given back), then
// one row per thread: its request by bisection of the offsets, its page from the
// table or, past the pages owned, from the ring. A page that a request takes
// begins with one of its new tokens, so that token's thread enters it in the
// table. Masks and depths come from walking the parents up.
//
// Bound by latency: a dozen dependent loads and barriers. One cluster of up to 8
// CTAs: every CTA repeats the sums (they fit one pass of its threads), and one
// cluster barrier, which the rows' work hides, separates the reads of the pool's
// state from its update in place, which a grid of independent CTAs could not order.
//
// Measured (in a graph): one token 3.3 us, 256 trees of 16 5.6. The 8 CTAs take all rows,
// padding among them: 64 tokens in 4096, 65,536 and 2^20 rows 3.9, 8.3, 85 us; 65,536 and
// 2^20 rows of prompts 15.9, 226 us. A chain given as 256 parents is 256 loads one after
// the other, 41 us; without parents a chain costs nothing.
#include "moe_common.cuh"
#include "spans.h"

namespace moe {
namespace {

constexpr int kPmThreads = 512, kPmWarps = kPmThreads / 32, kPmMaxB = 4096;

struct PmParams {
  const int32_t *context, *added, *parent;
  moe_page_pool pool;
  moe_token_map out;
  int B, shift, width, M, cap, words;
};

// Exclusive sum over the CTA's threads, and the total.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v,
                                                         unsigned long long (&part)[kPmWarps],
                                                         unsigned long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  __syncthreads();   // `part` may hold the last scan's sums
  if (lane == 31) part[warp] = s;
  __syncthreads();
  unsigned long long before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kPmWarps; ++i) {
    const unsigned long long x = part[i];
    before += i < warp ? x : 0;
    total += x;
  }
  return before + s - v;
}

// The i-th of the ring's cap entries from `head` on, 0 <= i <= cap <= 2^30.
__device__ __forceinline__ int entry_of(int head, int i, int cap) { return head + i - (head + i >= cap ? cap : 0); }

// A request as the rows see it: first row, first page taken (in ring order),
// context, pages owned (negative: not served).
struct __align__(16) PmReq {
  int row, first, ctx, owned;
};

__global__ void __launch_bounds__(kPmThreads) page_map_kernel(const PmParams p) {
  pdl_begin();
  extern __shared__ PmReq req[];   // [B + 1]; the last one has only its row
  __shared__ unsigned long long s_part[kPmWarps];
  __shared__ int s_taken, s_came, s_refused, s_bad;
  const int tid = threadIdx.x, rank = blockIdx.x, nctas = gridDim.x;
  const int per = (p.B + kPmThreads - 1) / kPmThreads, b0 = tid * per;
  if (tid == 0) {
    s_taken = s_came = s_refused = s_bad = 0;
    if (rank == 0) p.out.status[4] = 0;   // before the cluster's barrier
  }
  const int cap = p.cap;
  const int head = (int)((unsigned)p.pool.ring_pos[0] % (unsigned)cap);
  const int free_pages = min(max(p.pool.ring_pos[1], 0), cap);

  // (the first request's, the only one of up to 512, before the first sum waits)
  const bool some = b0 < p.B;
  const int add0 = some ? p.added[b0] : 0, ctx0 = some ? p.context[b0] : 0, own0 = some ? p.pool.owned[b0] : 0;

  // rows: sums of up to 4096 lengths below 2^31 fit 64 bits
  unsigned long long mine = max(add0, 0), total_rows = 0;
  for (int i = 1; i < per && b0 + i < p.B; ++i) mine += max(p.added[b0 + i], 0);
  unsigned long long row = block_scan(mine, s_part, total_rows);
  // pages needed (low half) and given back (high half), each at most B * width <= 2^30
  unsigned long long pages = 0;
  for (int i = 0; i < per && b0 + i < p.B; ++i) {
    const int b = b0 + i, add = i ? p.added[b] : add0, ctx = i ? p.context[b] : ctx0,
              own = i ? p.pool.owned[b] : own0;
    const long long n = max(add, 0), len = ctx + n;
    const int want = (int)min((len + (1 << p.shift) - 1) >> p.shift, (long long)p.width + 1);
    const bool owns = own >= 0 && own <= p.width;
    const bool sound = add >= 0 && ctx >= 0 && owns && want <= p.width &&
                       ctx <= ((long long)own << p.shift) && row + n <= (unsigned)p.M &&
                       (!p.words || n <= 64 * p.words);
    const bool ended = add < 0 && owns;
    req[b] = {(int)min(row, (unsigned long long)p.M), sound ? max(want - own, 0) : 0, ctx,
              sound ? own : ended ? -2 - own : -1};
    if (sound) pages += max(want - own, 0);
    if (ended) pages += (unsigned long long)own << 32;
    row += n;
  }
  unsigned long long total_pages = 0;
  unsigned long long at = block_scan(pages, s_part, total_pages);
  const int rows = (int)min(total_rows, (unsigned long long)p.M);
  if (tid == 0) req[p.B] = {rows, 0, 0, -1};
  int taken = 0, came = 0, refused = 0;
  for (int i = 0; i < per && b0 + i < p.B; ++i) {
    PmReq r = req[b0 + i];
    const int need = r.first, upto = (int)(unsigned)at + need;
    if (r.owned >= 0) {
      r.first = (int)(unsigned)at;
      at += need;
      if (need && upto > free_pages) {
        r.owned = -1;
      } else if (need) {
        taken = upto;
      }
    } else if (r.owned <= -2) {
      const int back = -2 - r.owned, from = (int)(at >> 32);
      at += (unsigned long long)back << 32;
      r.first = from;
      if (from + back <= cap - free_pages) {
        came = max(came, from + back);
      } else {
        r.owned = -1;
      }
    }
    refused += r.owned == -1;
    req[b0 + i] = r;
  }
  if (taken) atomicMax(&s_taken, taken);
  if (came) atomicMax(&s_came, came);
  if (refused) atomicAdd(&s_refused, refused);
  __syncthreads();
  // What the CTAs read and others update in place, owned and ring_pos, is read. (Pages
  // given back go to entries of the ring that no row takes.)
  if (nctas > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  // ------------------------------------------------------------- the rows
  int bad = 0;
  const int page = 1 << p.shift;
  for (int t = rank * kPmThreads + tid; t < p.M; t += nctas * kPmThreads) {
    int slot = -1, pos = 0;
    unsigned long long bits[4] = {0, 0, 0, 0};
    if (t < rows) {
      int lo = 0, hi = p.B;   // the last request whose first row is at most t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (req[mid].row <= t) lo = mid; else hi = mid;
      }
      const PmReq r = req[lo];
      if (r.owned >= 0) {
        const int i = t - r.row, j = r.ctx + i, pg = j >> p.shift;
        int32_t* entry = p.pool.table + (long long)lo * p.width + pg;
        int id;
        if (pg < r.owned) {
          id = *entry;
        } else {
          id = p.pool.ring[entry_of(head, r.first + pg - r.owned, cap)];
          if ((j & (page - 1)) == 0) *entry = id;
        }
        if (id >= 0 && id <= (0x7fffffff >> p.shift) - 1) slot = (id << p.shift) | (j & (page - 1));
        int depth = i;
        if (p.parent) {
          const int32_t* par = p.parent + r.row;
          depth = -1;
          for (int a = i; a >= 0;) {   // (each step goes to a smaller index)
            const unsigned long long bit = 1ull << (a & 63);
#pragma unroll
            for (int w = 0; w < 4; ++w)
              if (a >> 6 == w) bits[w] |= bit;
            ++depth;
            const int up = __ldg(par + a);
            const bool ok = up >= -1 && up < a;
            bad += !ok && a == i;
            a = ok ? up : -1;
          }
        } else if (p.words) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int k = i + 1 - 64 * w;
            bits[w] = k >= 64 ? ~0ull : k > 0 ? (1ull << k) - 1 : 0;
          }
        }
        pos = r.ctx + depth;
      }
    }
    p.out.slot[t] = slot;
    p.out.position[t] = pos;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      if (w < p.words) p.out.mask[(long long)t * p.words + w] = bits[w];
  }
  if (bad) atomicAdd(&s_bad, bad);

  // ------------------------------------- the pool's state, all reads done
  __syncthreads();
  if (nctas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  for (int b = rank * kPmThreads + tid; b <= p.B; b += nctas * kPmThreads) {
    const PmReq r = req[b];
    p.out.offsets[b] = r.row;
    if (b == p.B) break;
    const int n = max(p.added[b], 0), own = p.pool.owned[b];
    const int want = (int)(((long long)r.ctx + n + page - 1) >> p.shift);
    p.out.length[b] = r.owned >= 0 ? r.ctx + n : 0;
    p.pool.owned_out[b] = r.owned >= 0 ? max(own, want) : r.owned <= -2 ? 0 : own;
  }
  const int warp = tid >> 5, lane = tid & 31;
  if (s_came)
    for (int b = rank * kPmWarps + warp; b < p.B; b += nctas * kPmWarps) {
      const PmReq r = req[b];
      if (r.owned > -2) continue;
      // (8 loads under way: one at a time took 4 us for 1000 pages)
      const int back = -2 - r.owned;
      const int32_t* from = p.pool.table + (long long)b * p.width;
      for (int i0 = lane; i0 < back; i0 += 32 * 8) {
        int id[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) id[j] = i0 + 32 * j < back ? from[i0 + 32 * j] : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i0 + 32 * j < back) p.pool.ring[entry_of(head, free_pages + r.first + i0 + 32 * j, cap)] = id[j];
      }
    }
  if (tid == 0) {
    if (s_bad) atomicAdd(p.out.status + 4, s_bad);
    if (rank == 0) {
      const long long lack = (long long)(total_pages & 0xffffffffu) - free_pages;
      p.pool.ring_pos_out[0] = entry_of(head, s_taken, cap);
      p.pool.ring_pos_out[1] = free_pages - s_taken + s_came;
      p.out.status[0] = rows;
      p.out.status[1] = s_taken;
      p.out.status[2] = s_refused;
      p.out.status[3] = (int)max(lack, 0ll);
    }
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_page_map(const moe_page_desc* d, const int32_t* context,
                                   const int32_t* added, const int32_t* parent,
                                   const moe_page_pool* pool, const moe_token_map* out,
                                   moe_stream_t stream) {
  if (!d || !context || !added || !pool || !out) return MOE_ERR_INVALID_ARG;
  if (d->requests < 1 || d->table_width < 1 || d->max_tokens < 1 || d->ring_size < 1 ||
      d->mask_words < 0 || d->page_size < 1)
    return MOE_ERR_INVALID_ARG;
  int shift = 4;
  while (shift < 9 && (1 << shift) != d->page_size) ++shift;
  if (shift == 9 || d->requests > kPmMaxB || d->table_width > (1 << 18) ||
      d->max_tokens > (1 << 20) || d->ring_size > (1 << 30) || d->mask_words > 4)
    return MOE_ERR_UNSUPPORTED;
  if (!pool->table || !pool->ring || !pool->owned || !pool->owned_out || !pool->ring_pos ||
      !pool->ring_pos_out || !out->length || !out->offsets || !out->slot || !out->position ||
      !out->status)
    return MOE_ERR_INVALID_ARG;
  if ((d->mask_words > 0) != (out->mask != nullptr) || (parent && !d->mask_words))
    return MOE_ERR_INVALID_ARG;
  const size_t B = d->requests, M = d->max_tokens, W = d->table_width;
  // written first, then what is only read
  const Span s[] = {{pool->table, 4 * B * W}, {pool->ring, 4 * (size_t)d->ring_size},
                    {pool->owned_out, 4 * B}, {pool->ring_pos_out, 8},
                    {out->length, 4 * B}, {out->offsets, 4 * (B + 1)},
                    {out->slot, 4 * M}, {out->position, 4 * M},
                    {out->status, 20}, {out->mask, 8 * M * d->mask_words},
                    {pool->owned, 4 * B}, {pool->ring_pos, 8},
                    {context, 4 * B}, {added, 4 * B},
                    {parent, 4}};   // (as many parents as there are rows, which the device knows)
  constexpr int kWritten = 10, kAll = 15;
  for (int i = 0; i < kAll; ++i)
    if (!is_aligned(s[i].p, s[i].p == out->mask ? 8 : 4)) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < kWritten; ++i)
    for (int j = i + 1; j < kAll; ++j) {
      // the state in place: the same array, not a shifted one
      if ((i == 2 && j == 10) || (i == 3 && j == 11))
        if (s[i].p == s[j].p) continue;
      if (clash(s[i], s[j])) return MOE_ERR_INVALID_ARG;
    }
  PmParams p{context, added, parent, *pool, *out, d->requests, shift, d->table_width,
             d->max_tokens, d->ring_size, d->mask_words};
  const int smem = (d->requests + 1) * (int)sizeof(PmReq);
  const void* kern = reinterpret_cast<const void*>(page_map_kernel);
  if (smem > 40 * 1024 && allow_smem(kern, smem) != cudaSuccess) return MOE_ERR_CUDA;
  int ctas = (d->max_tokens + kPmThreads - 1) / kPmThreads;
  ctas = ctas > 4 ? 8 : ctas > 2 ? 4 : ctas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, page_map_kernel, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
