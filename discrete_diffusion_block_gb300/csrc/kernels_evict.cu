// Eviction from the paged KV cache by accumulated attention weight: of a
// sequence's L > budget cached tokens each KV head keeps the first `sinks`, the
// last `recent`, and of those between them the budget - sinks - recent of the
// largest weight (equal ones by ascending slot); what is kept moves together, in
// order, to the slots 0 .. of the pages of out_tables.
//
// What bounds it: the weights are read once (4 L bytes a head), the kept rows of K
// and V read and written once (8 hd bytes a row): the memory's bandwidth, for few
// sequences the latency of the chain weights -> choice -> rows.
//
// A cluster of 1 to 8 blocks takes one KV head of one sequence.  Each of its blocks
// makes the whole choice for itself (reading L weights from L2 costs less than
// passing counts between blocks): a radix select, 11, 11 and 10 bits at a time over
// histograms in shared memory, gives the smallest kept weight and how many of its
// equals stay; then a bit per slot says what is kept, and a running count per word
// of bits finds the d-th kept slot by bisection.  The blocks take turns of
// kEvictTurn rows each; a warp moves K and V of its rows through registers (the
// 16-byte chunks of a row change places with slot % 8), all loads before all stores.
//
// In place (out_tables holds the sequence's own pages) this order is what makes it
// safe: the d-th kept slot is never before d, so the rows that a turn reads lie
// behind all that earlier turns wrote, and a cluster barrier between a turn's loads
// and its stores keeps those from overtaking the loads of the same turn.
#include <algorithm>

#include "gemm_tc.cuh"
#include "internal.h"

namespace dg {

namespace {

constexpr int kEvictThreads = 512;
constexpr int kEvictRows = 16;                               // rows of a warp in a turn
constexpr int kEvictTurn = kEvictThreads / 32 * kEvictRows;  // of a block
constexpr int kEvictKeys = 32768;                            // weights kept in shared memory; later ones are read again
constexpr int kEvictBins = 2048;

struct EvictArgs {
  CacheEvict a;
  int words;  // words of bits that the shared memory holds: a sequence may have 32 times as many slots
  int keys;   // weights that it holds
  int *err;
};

// A weight as an integer of the same order: NaN below all, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  if (w != w) return 0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sum of v over the threads before this one; total: over all.  scratch: 17 ints.
__device__ __forceinline__ int block_scan(int v, int *scratch, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int x = lane < kEvictThreads / 32 ? scratch[lane] : 0;
#pragma unroll
    for (int o = 1; o < kEvictThreads / 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane < kEvictThreads / 32) scratch[lane] = x;
  }
  __syncthreads();
  *total = scratch[kEvictThreads / 32 - 1];
  const int before = warp ? scratch[warp - 1] : 0;
  __syncthreads();
  return before + incl - v;
}

// The n-th (from 0) set bit of w.
__device__ __forceinline__ int nth_bit(uint32_t w, int n) {
  int at = 0;
#pragma unroll
  for (int half = 16; half; half >>= 1) {
    const int c = __popc(w & ((1u << half) - 1));
    if (n >= c) {
      n -= c;
      at += half;
      w >>= half;
    }
  }
  return at;
}

template <int HD>
__global__ void __launch_bounds__(kEvictThreads, 1) cache_evict_kernel(const __grid_constant__ EvictArgs p) {
  extern __shared__ uint32_t smem[];
  __shared__ int scan[20], hist[kEvictBins], found[2], flags;
  uint32_t *bits = smem, *equal = bits + p.words, *keys = equal + p.words;
  int *before = (int *)equal;  // kept slots before a word (once `equal` is done with)
  const CacheEvict &a = p.a;
  const int C = cluster_ctas(), rank = blockIdx.x % C, unit = blockIdx.x / C;
  const int b = unit / a.Hkv, g = unit - b * a.Hkv, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int L = a.lens[b], n_out = min(L, a.budget);
  const int *table = a.page_tables + (size_t)b * a.max_pages, *out_table = a.out_tables + (size_t)b * a.out_max_pages;
  int *kept = a.kept ? a.kept + ((size_t)b * a.Hkv + g) * a.budget : nullptr;

  // Sequences that the call cannot move are left alone; the same in all blocks.
  if (tid == 0) flags = 0;
  __syncthreads();
  const bool bad_length = L < 0 || (long long)L > (long long)a.max_pages * a.pg || (L + 31) / 32 > p.words ||
                          (long long)n_out > (long long)a.out_max_pages * a.pg;
  if (!bad_length) {
    int f = 0;
    const int n_pages = ceil_div(L, a.pg), n_out_pages = ceil_div(n_out, a.pg);
    for (int i = tid; i < n_pages; i += kEvictThreads) {
      const int src = table[i], dst = i < n_out_pages ? out_table[i] : -1;
      if (src < 0 || src >= a.n_pages || (i < n_out_pages && (dst < 0 || dst >= a.n_pages))) f |= 1;
      if (src == dst) f |= 2;  // in place
    }
    if (f) atomicOr(&flags, f);
  }
  __syncthreads();
  const bool bad = bad_length || (flags & 1), in_place = flags & 2;
  if (bad) {
    if (tid == 0 && p.err) atomicExch(p.err + 1, bad_length ? kBadSequence : kBadPage);
    if (tid == 0 && rank == 0 && g == 0) a.out_lens[b] = -1;
    if (kept && rank == 0)
      for (int d = tid; d < a.budget; d += kEvictThreads) kept[d] = -1;
    return;
  }
  if (tid == 0 && rank == 0 && g == 0) a.out_lens[b] = n_out;
  const int words = (L + 31) / 32;

  // ---- the choice
  if (L > a.budget) {
    auto weight = [&](int j) { return order_key(__ldcg(a.mass + ((size_t)table[j / a.pg] * a.Hkv + g) * a.pg + j % a.pg)); };
    const int lo = a.sinks, hi = L - a.recent;
    const int cached = min(L, p.keys);
    for (int j = tid; j < cached; j += kEvictThreads) keys[j] = weight(j);
    auto key = [&](int j) { return j < cached ? keys[j] : weight(j); };
    uint32_t least = 0xffffffffu, mask = 0;
    int left = a.budget - a.sinks - a.recent;  // equals of `least` that stay
    if (left > 0) {
      least = 0;
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
        for (int i = tid; i < bins; i += kEvictThreads) hist[i] = 0;
        __syncthreads();
        for (int j0 = lo + 32 * warp; j0 < hi; j0 += kEvictThreads) {
          const int j = j0 + lane;
          const uint32_t k = j < hi ? key(j) : 0;
          const bool in = j < hi && (k & mask) == least;
          const int bin = (k >> shift) & (bins - 1);
          // (weights that nothing looked at are all 0: one addition for a warp of equals)
          int same;
          __match_all_sync(0xffffffffu, in ? bin : -1, &same);
          if (same) {
            if (lane == 0 && in) atomicAdd(&hist[bin], 32);
          } else if (in) {
            atomicAdd(&hist[bin], 1);
          }
        }
        __syncthreads();
        // from the top: the bin in which the count reaches `left`
        const int per = bins / kEvictThreads, top = bins - 1 - tid * per;
        int n = 0, total;
        for (int i = 0; i < per; ++i) n += hist[top - i];
        int above = block_scan(n, scan, &total);
        if (above < left && above + n >= left) {
          int bin = top;
          while (above + hist[bin] < left) above += hist[bin--];
          found[0] = bin;
          found[1] = left - above;
        }
        __syncthreads();
        least |= (uint32_t)found[0] << shift;
        left = found[1];
        mask |= (uint32_t)(bins - 1) << shift;
        __syncthreads();
      }
    } else {
      __syncthreads();
    }
    // bits of the slots that stay whatever their equals do, and of the equals
    for (int w = warp; w < words; w += kEvictThreads / 32) {
      const int j = 32 * w + lane;
      const bool there = j < L, always = there && (j < lo || j >= hi);
      const uint32_t k = there ? key(j) : 0;
      const uint32_t more = __ballot_sync(0xffffffffu, always || (there && k > least));
      const uint32_t same = __ballot_sync(0xffffffffu, there && !always && k == least);
      if (lane == 0) {
        bits[w] = more;
        equal[w] = same;
      }
    }
    __syncthreads();
    // of the equals the first `left`
    const int per = ceil_div(words, kEvictThreads), w0 = min(words, tid * per), w1 = min(words, w0 + per);
    int n = 0, total;
    for (int w = w0; w < w1; ++w) n += __popc(equal[w]);
    int at = block_scan(n, scan, &total);
    for (int w = w0; w < w1 && at < left; ++w) {
      const uint32_t e = equal[w];
      const int c = __popc(e);
      bits[w] |= at + c <= left ? e : e & ((1u << nth_bit(e, left - at)) - 1);
      at += c;
    }
    __syncthreads();
    n = 0;
    for (int w = w0; w < w1; ++w) n += __popc(bits[w]);
    at = block_scan(n, scan, &total);
    for (int w = w0; w < w1; ++w) {
      before[w] = at;
      at += __popc(bits[w]);
    }
    __syncthreads();
  }

  // ---- the move
  constexpr int kLanes = HD / 8;        // lanes of a row of K, and of V
  constexpr int kSide = 32 / (2 * kLanes);  // rows of K and V that the warp moves at once
  const int half = lane & (2 * kLanes - 1), v_side = half / kLanes, c = half % kLanes;
  const bf16 *pool = v_side ? a.v_pool : a.k_pool;
  bf16 *out = v_side ? a.v_pool : a.k_pool;
  const size_t sub = (size_t)(c >> 3) * a.pg * 64;
  for (int d0 = 0; d0 < n_out; d0 += C * kEvictTurn) {
    const int first = d0 + (rank * (kEvictThreads / 32) + warp) * kEvictRows;
    // row `first + lane` of the warp's: where it lies and where it goes
    int src = -1, src_slot = 0, dst_slot = 0;
    size_t src_at = 0, dst_at = 0;
    float w = 0.0f;
    if (lane < kEvictRows && first + lane < n_out) {
      const int d = first + lane;
      src = d;
      if (L > a.budget) {
        int l = 0, r = words - 1;  // the last word with before <= d
        while (l < r) {
          const int m = (l + r + 1) >> 1;
          if (before[m] <= d) l = m;
          else r = m - 1;
        }
        src = 32 * l + nth_bit(bits[l], d - before[l]);
      }
      const int sp = src / a.pg, dp = d / a.pg;
      src_slot = src - sp * a.pg;
      dst_slot = d - dp * a.pg;
      src_at = ((size_t)table[sp] * a.Hkv + g) * a.pg;
      dst_at = ((size_t)out_table[dp] * a.Hkv + g) * a.pg;
      w = __ldcg(a.mass + src_at + src_slot);
      if (kept) kept[d] = src;
    }
    uint4 row[kEvictRows / kSide];
#pragma unroll
    for (int i = 0; i < kEvictRows / kSide; ++i) {
      const int from = i * kSide + lane / (2 * kLanes);
      const int s = __shfl_sync(0xffffffffu, src_slot, from);
      const size_t at = __shfl_sync(0xffffffffu, (unsigned long long)src_at, from);
      if (first + from < n_out) row[i] = __ldcg((const uint4 *)(pool + at * HD + sub + (size_t)s * 64 + (((c & 7) ^ (s & 7)) << 3)));
    }
    if (in_place) {
      if (C > 1) tc::cluster_sync();
      else __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kEvictRows / kSide; ++i) {
      const int from = i * kSide + lane / (2 * kLanes);
      const int s = __shfl_sync(0xffffffffu, dst_slot, from);
      const size_t at = __shfl_sync(0xffffffffu, (unsigned long long)dst_at, from);
      const bool moved = __shfl_sync(0xffffffffu, (int)(src_at != dst_at || src_slot != dst_slot), from);
      if (first + from < n_out && moved) *(uint4 *)(out + at * HD + sub + (size_t)s * 64 + (((c & 7) ^ (s & 7)) << 3)) = row[i];
    }
    if (src >= 0) a.mass[dst_at + dst_slot] = w;
  }
  if (kept && rank == 0)
    for (int d = n_out + tid; d < a.budget; d += kEvictThreads) kept[d] = -1;
}

template <int HD>
cudaError_t launch_evict(const EvictArgs &p, int cluster, size_t smem, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(cache_evict_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.a.n_seqs * p.a.Hkv * cluster);
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_evict_kernel<HD>, p);
}

}  // namespace

cudaError_t cache_evict(const CacheEvict &a, int *err, cudaStream_t st) {
  if (a.n_seqs == 0) return cudaSuccess;
  EvictArgs p{};
  p.a = a;
  p.err = err;
  const int slots = (int)(std::min)((long long)a.max_pages * a.pg, (long long)kEvictMostSlots);
  p.words = ceil_div(slots, 32);
  p.keys = (std::min)(slots, kEvictKeys);
  // Blocks for all SMs where there are few heads of few sequences, as far as the
  // kept rows give each block of a cluster a turn.
  int cluster = 1;
  while (cluster < 8 && a.n_seqs * a.Hkv * cluster < 152 && cluster * kEvictTurn < a.budget) cluster *= 2;
  const size_t smem = ((size_t)2 * p.words + p.keys) * 4;
  return a.hd == 128 ? launch_evict<128>(p, cluster, smem, st) : launch_evict<64>(p, cluster, smem, st);
}

}  // namespace dg
