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
// The choice, by a block of 1024 threads: a radix select, 11, 11 and 10 bits at a time over
// histograms in shared memory, gives the smallest kept weight and how many of its equals
// stay; then a bit per slot says what is kept, and running counts of the bits give every
// kept slot its place in the list.  The move, by a cluster of up to 8 blocks: the blocks
// take turns of some rows a warp; a warp moves K and V of its rows through registers (the
// 16-byte chunks of a row change places with slot % 8), all loads before all stores.  Small
// calls are one launch, in which each block makes the choice for itself, others two, the
// choices and the moves (launch_evict has the rule and both sides' times).
//
// Measured in captured graphs (8 KV heads of 128): 12 sequences of up to 32k slots to 8k 124
// us, 70% of the copy bandwidth (the move alone 95 us, the choice 27); 29 of up to 2900 to
// 1111 (4 heads of 64) 19.5 us, the choice 8.5 and the rows 9 of a block; one of 2176 to 2048
// 12.6, a chain of latencies: lengths and tables 1.1 us, weights 0.8, three passes 3.5, bits
// and lists 2.0, rows 3.6, launch and end 1.6 (clock stamps of a block).  In place the small
// ones take as long, the large one 111 where it takes 133 (calls one by one, caches cold):
// its rows before the first that goes are not moved.  Not kept:
// passes that end early where all that is left of a bin stays (0.1 us less); the move's
// launch begun under the choice (0.5 us less of the small ones, 4 more of the large).
//
// In place (out_tables holds the sequence's own pages) this order is what makes it
// safe: the d-th kept slot is never before d, so the rows that a turn reads lie
// behind all that earlier turns wrote, and a cluster barrier between a turn's loads
// and its stores keeps those from overtaking the loads of the same turn.
#include <algorithm>
#include <atomic>

#include "gemm_tc.cuh"
#include "internal.h"

namespace dg {

namespace {

constexpr int kEvictThreads = 1024;  // of the choice
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 16;                              // rows of a warp in a turn
constexpr int kMoveTurn = kMoveThreads / 32 * kMoveRows;   // of a block
constexpr int kBothRows = 8, kBothTurn = kEvictThreads / 32 * kBothRows;  // the same, in one launch with the choice
constexpr int kEvictKeys = 32768;    // weights kept in shared memory; later ones are read again
constexpr int kEvictBins = 2048;
constexpr int kFewUnits = 152;  // (KV head, sequence) pairs of a call in one launch
constexpr int kChoiceBytes = (2 * (kEvictMostSlots / 32) + kEvictKeys) * 4;  // most of its dynamic shared memory
static_assert(kEvictMostSlots % 128 == 0 && kChoiceBytes <= 212992, "shared memory of the choice");
constexpr int kEvictPages = 1024;    // entries of the page table kept in shared memory

struct EvictArgs {
  CacheEvict a;
  int words;  // words of bits that the shared memory holds: a sequence may have 32 times as many slots
  int keys;   // weights that it holds
  int pg_shift, vec;  // log2 of the page size (-1: no power of two); weights can be loaded four at a time
  int *err;
};

// A weight as an integer of the same order: NaN below all (1), -0 as 0.  kStays: above
// all; 0: no slot of the sequence.
constexpr uint32_t kStays = 0xffffffffu;
__device__ __forceinline__ uint32_t order_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  if (w != w) return 1u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sum of v over the threads before this one; total: over all.  scratch: 32 ints.
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

// The choice for KV head g of sequence b, by a block; `lists`: it writes the call's lists
// and lengths.  Returns the number of slots kept, -1 where the sequence is left alone.
// slots (or NULL): the slots kept of a sequence beyond the budget, once more in shared
// memory (in place of the weights).
__device__ __forceinline__ int choose(const EvictArgs &p, int b, int g, bool lists, uint32_t *smem, int *slots) {
  __shared__ int scan[32], hist[kEvictBins], found[2], flags, entries[kEvictPages];
  uint32_t *bits = smem, *equal = bits + p.words, *keys = equal + p.words;
  const CacheEvict &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int L = a.lens[b], n_out = min(L, a.budget);
  const int *table = a.page_tables + (size_t)b * a.max_pages, *out_table = a.out_tables + (size_t)b * a.out_max_pages;
  int *kept = a.kept + ((size_t)b * a.Hkv + g) * a.budget;
  // -1 behind the last kept slot (budgets go up to 2^31 - 1: unsigned, so that the last step does not wrap)
  auto fill = [&](int from) {
    for (unsigned d = from + tid; lists && d < (unsigned)a.budget; d += kEvictThreads) kept[d] = -1;
  };

  // Sequences that the call cannot move are left alone; the same in all blocks.
  if (tid == 0) flags = 0;
  __syncthreads();
  // (lengths and page sizes go up to 2^31 - 1: nothing is added to them)
  const bool bad_length = L < 0 || L > 32 * p.words || (long long)L > (long long)a.max_pages * a.pg ||
                          (long long)n_out > (long long)a.out_max_pages * a.pg;
  auto pages_for = [&](int n) { return n / a.pg + (n % a.pg != 0); };
  const int n_pages = bad_length ? 0 : pages_for(L);
  if (!bad_length) {
    bool f = false;
    const int n_out_pages = pages_for(n_out);
    for (int i = tid; i < n_pages; i += kEvictThreads) {
      const int src = table[i], dst = i < n_out_pages ? out_table[i] : 0;
      if (i < kEvictPages) entries[i] = src;
      f |= src < 0 || src >= a.n_pages || dst < 0 || dst >= a.n_pages;
    }
    if (f) flags = 1;
  }
  __syncthreads();
  const bool bad = bad_length || flags;
  if (bad) {
    if (tid == 0 && p.err) atomicExch(p.err + 1, bad_length ? kBadSequence : kBadPage);
    if (tid == 0 && g == 0 && lists) a.out_lens[b] = -1;
    fill(0);
    return -1;
  }
  if (tid == 0 && g == 0 && lists) a.out_lens[b] = n_out;
  fill(n_out);
  if (L <= a.budget) {
    for (int d = tid; d < L && lists; d += kEvictThreads) kept[d] = d;
    return L;
  }
  const int words = (L + 31) / 32;

  const int *pages = n_pages <= kEvictPages ? entries : table;
  auto place = [&](int j) {
    const int page = p.pg_shift >= 0 ? j >> p.pg_shift : j / a.pg;
    return a.mass + ((size_t)pages[page] * a.Hkv + g) * a.pg + (j - page * a.pg);
  };
  auto key_of = [&](int j, float w) { return j >= L ? 0u : j < a.sinks || j >= L - a.recent ? kStays : order_key(w); };
  // four slots, from a multiple of four on
  auto load4 = [&](int j) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (p.vec) {  // (the fours behind the last slot lie in its page)
      v = __ldcg((const float4 *)place(j));
    } else {
      v.x = __ldcg(place(j));
      if (j + 1 < L) v.y = __ldcg(place(j + 1));
      if (j + 2 < L) v.z = __ldcg(place(j + 2));
      if (j + 3 < L) v.w = __ldcg(place(j + 3));
    }
    return make_uint4(key_of(j, v.x), key_of(j + 1, v.y), key_of(j + 2, v.z), key_of(j + 3, v.w));
  };
  const int cached = min(128 * ceil_div(L, 128), p.keys);
#pragma unroll 8
  for (int j = 4 * tid; j < cached; j += 4 * kEvictThreads) *(uint4 *)(keys + j) = j < L ? load4(j) : make_uint4(0u, 0u, 0u, 0u);
  auto key4 = [&](int j) { return j < cached ? *(const uint4 *)(keys + j) : j < L ? load4(j) : make_uint4(0u, 0u, 0u, 0u); };
  // the budget's largest, those that stay in any case among them: the least of them, and
  // how many of its equals stay (`left`)
  uint32_t least = 0, mask = 0;
  int left = a.budget;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    for (int i = tid; i < bins; i += kEvictThreads) hist[i] = 0;
    __syncthreads();
#pragma unroll 1
    for (int j0 = 128 * warp; j0 < L; j0 += 4 * kEvictThreads) {
      const uint4 k = key4(j0 + 4 * lane);
      const bool in[4] = {(k.x & mask) == least && k.x, (k.y & mask) == least && k.y, (k.z & mask) == least && k.z, (k.w & mask) == least && k.w};
      if (!__any_sync(0xffffffffu, in[0] || in[1] || in[2] || in[3])) continue;
      const int bin[4] = {(int)(k.x >> shift) & (bins - 1), (int)(k.y >> shift) & (bins - 1), (int)(k.z >> shift) & (bins - 1),
                          (int)(k.w >> shift) & (bins - 1)};
      // (weights that nothing looked at are all 0, and many stay: one addition for a warp of equals)
      const bool equal4 = in[0] && in[1] && in[2] && in[3] && bin[0] == bin[1] && bin[0] == bin[2] && bin[0] == bin[3];
      const int bin0 = __shfl_sync(0xffffffffu, bin[0], 0);
      if (__all_sync(0xffffffffu, equal4 && bin[0] == bin0)) {
        if (lane == 0) atomicAdd(&hist[bin[0]], 128);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (in[i]) atomicAdd(&hist[bin[i]], 1);
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
  }
  // bits of the slots above it, and of its equals: a lane has four slots, eight lanes a word
#pragma unroll 1
  for (int j0 = 128 * warp; j0 < L; j0 += 4 * kEvictThreads) {
    const uint4 k = key4(j0 + 4 * lane);
    const int at = 4 * (lane & 7);
    uint32_t more = ((k.x > least ? 1u : 0u) | (k.y > least ? 2u : 0u) | (k.z > least ? 4u : 0u) | (k.w > least ? 8u : 0u)) << at;
    uint32_t same = ((k.x == least ? 1u : 0u) | (k.y == least ? 2u : 0u) | (k.z == least ? 4u : 0u) | (k.w == least ? 8u : 0u)) << at;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      more |= __shfl_xor_sync(0xffffffffu, more, o);
      same |= __shfl_xor_sync(0xffffffffu, same, o);
    }
    if ((lane & 7) == 0) {
      bits[j0 / 32 + lane / 8] = more;
      equal[j0 / 32 + lane / 8] = same;
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
  // kept slots before each word, then the list
  n = 0;
  for (int w = w0; w < w1; ++w) n += __popc(bits[w]);
  at = block_scan(n, scan, &total);
  int *before = (int *)equal;  // (done with)
  for (int w = w0; w < w1; ++w) {
    before[w] = at;
    at += __popc(bits[w]);
  }
  __syncthreads();
  for (int w = warp; w < words && (lists || slots); w += kEvictThreads / 32) {
    const uint32_t e = bits[w];
    const int d = before[w] + __popc(e & ((1u << lane) - 1));
    if (e >> lane & 1) {
      if (lists) kept[d] = 32 * w + lane;
      if (slots) slots[d] = 32 * w + lane;
    }
  }
  return n_out;
}

__global__ void __launch_bounds__(kEvictThreads, 1) evict_choice_kernel(const __grid_constant__ EvictArgs p) {
  extern __shared__ uint32_t smem[];
  const int b = blockIdx.x / p.a.Hkv;
  choose(p, b, blockIdx.x - b * p.a.Hkv, true, smem, nullptr);
}

// Whether sequence b, of one slot or more, stays as it is: within the budget, in place.
__device__ __forceinline__ bool stays(const EvictArgs &p, int b) {
  const CacheEvict &a = p.a;
  return a.lens[b] <= a.budget && a.page_tables[(size_t)b * a.max_pages] == a.out_tables[(size_t)b * a.out_max_pages];
}

// Moves the n_out > 0 kept rows of a KV head, K, V and weights, by a cluster of C blocks of
// WARPS warps, ROWS rows a warp in a turn; slot_of(d): the slot that the d-th had.
template <int HD, int WARPS, int ROWS, class SlotOf>
__device__ __forceinline__ void move_rows(const EvictArgs &p, int b, int g, int n_out, int C, int rank, SlotOf slot_of) {
  const CacheEvict &a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int *table = a.page_tables + (size_t)b * a.max_pages, *out_table = a.out_tables + (size_t)b * a.out_max_pages;
  const bool in_place = table[0] == out_table[0];
  constexpr int kLanes = HD / 8;        // lanes of a row of K, and of V
  constexpr int kSide = 32 / (2 * kLanes);  // rows of K and V that the warp moves at once
  const int half = lane & (2 * kLanes - 1), v_side = half / kLanes, c = half % kLanes;
  const bf16 *pool = v_side ? a.v_pool : a.k_pool;
  bf16 *out = v_side ? a.v_pool : a.k_pool;
  const size_t sub = (size_t)(c >> 3) * a.pg * 64;
  for (int d0 = 0; d0 < n_out; d0 += C * WARPS * ROWS) {
    const int first = d0 + (rank * WARPS + warp) * ROWS;
    // row `first + lane` of the warp's: where it lies and where it goes
    int src = -1, src_slot = 0, dst_slot = 0;
    size_t src_at = 0, dst_at = 0;
    float w = 0.0f;
    if (lane < ROWS && first + lane < n_out) {
      const int d = first + lane;
      src = slot_of(d);
      const int sp = p.pg_shift >= 0 ? src >> p.pg_shift : src / a.pg, dp = p.pg_shift >= 0 ? d >> p.pg_shift : d / a.pg;
      src_slot = src - sp * a.pg;
      dst_slot = d - dp * a.pg;
      src_at = ((size_t)table[sp] * a.Hkv + g) * a.pg;
      dst_at = ((size_t)out_table[dp] * a.Hkv + g) * a.pg;
      w = __ldcg(a.mass + src_at + src_slot);
    }
    // (in place the rows before the first that goes stay where they are)
    const unsigned moving = __ballot_sync(0xffffffffu, src >= 0 && (src_at != dst_at || src_slot != dst_slot));
    uint4 row[ROWS / kSide];
#pragma unroll
    for (int i = 0; i < ROWS / kSide; ++i) {
      const int from = i * kSide + lane / (2 * kLanes);
      const int s = __shfl_sync(0xffffffffu, src_slot, from);
      const size_t at = __shfl_sync(0xffffffffu, (unsigned long long)src_at, from);
      if (moving >> from & 1) row[i] = __ldcg((const uint4 *)(pool + at * HD + sub + (size_t)s * 64 + (((c & 7) ^ (s & 7)) << 3)));
    }
    if (in_place) {
      if (C > 1) tc::cluster_sync();
      else __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < ROWS / kSide; ++i) {
      const int from = i * kSide + lane / (2 * kLanes);
      const int s = __shfl_sync(0xffffffffu, dst_slot, from);
      const size_t at = __shfl_sync(0xffffffffu, (unsigned long long)dst_at, from);
      if (moving >> from & 1) *(uint4 *)(out + at * HD + sub + (size_t)s * 64 + (((c & 7) ^ (s & 7)) << 3)) = row[i];
    }
    if (moving >> lane & 1) a.mass[dst_at + dst_slot] = w;
  }
}

template <int HD>
__global__ void __launch_bounds__(kMoveThreads, 2) evict_move_kernel(const __grid_constant__ EvictArgs p) {
  const CacheEvict &a = p.a;
  const int C = cluster_ctas(), rank = blockIdx.x % C, unit = blockIdx.x / C, b = unit / a.Hkv, g = unit - b * a.Hkv;
  const int n_out = a.out_lens[b];
  if (n_out <= 0 || stays(p, b)) return;  // (the same in all blocks of a cluster)
  const int *kept = a.kept + ((size_t)b * a.Hkv + g) * a.budget;
  move_rows<HD, kMoveThreads / 32, kMoveRows>(p, b, g, n_out, C, rank, [&](int d) { return kept[d]; });
}

// Both in one launch: every block of the cluster makes the choice for itself.
template <int HD>
__global__ void __launch_bounds__(kEvictThreads, 1) evict_kernel(const __grid_constant__ EvictArgs p) {
  extern __shared__ uint32_t smem[];
  const int C = cluster_ctas(), rank = blockIdx.x % C, unit = blockIdx.x / C, b = unit / p.a.Hkv, g = unit - b * p.a.Hkv;
  int *slots = (int *)(smem + 2 * p.words);
  const int n_out = choose(p, b, g, rank == 0, smem, slots);
  if (n_out <= 0 || stays(p, b)) return;  // (the same in all blocks of a cluster)
  const bool all = p.a.lens[b] <= p.a.budget;
  __syncthreads();
  move_rows<HD, kEvictThreads / 32, kBothRows>(p, b, g, n_out, C, rank, [&](int d) { return all ? d : slots[d]; });
}

// Lets a kernel use as much shared memory as any call needs, once per device.
template <void (*KERNEL)(const EvictArgs)>
cudaError_t choice_memory() {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev].load()) {
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, kChoiceBytes);
    if (e != cudaSuccess) return e;
    done[dev].store(true);
  }
  return cudaSuccess;
}

cudaError_t launch_clusters(void (*kernel)(const EvictArgs), const EvictArgs &p, int cluster, int threads, size_t smem, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.a.n_seqs * p.a.Hkv * cluster);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int HD>
cudaError_t launch_evict(const EvictArgs &p, int slots, cudaStream_t st) {
  const CacheEvict &a = p.a;
  const size_t smem = ((size_t)2 * p.words + p.keys) * 4;
  const long long units = (long long)a.n_seqs * a.Hkv;
  int cluster = 1;  // as many blocks as the kept rows have turns for
  // One launch while there is little to move and little to choose from: it saves a launch
  // and a round through the lists, but every block of a cluster makes the choice, and 1024
  // threads that hold a choice keep fewer rows on their way.  Measured, calls in a row, one
  // launch and two (8 heads of 128 unless stated): 1 sequence of 2176 slots to 2048 14.5 and
  // 18.6 us, of 8192 to 7000 (29 MB) 29.0 and 37.1; 29 of 2900 to 1111, 4 heads of 64, 20.9
  // and 30.1; 4 of 8192 to 2048 (34 MB) 26.8 and 30.9, of 4096 to 4000 (66 MB) 35.1 and 38.5;
  // 16 of 2300 to 2048 (134 MB) 59.4 and 59.5, in a graph 57.2 and 55.5; 19 of 4500 to 4096
  // 120 and 117; 12 of 32k to 8k 134 and 128.
  if (units <= kFewUnits && slots <= 8192 && units * a.budget * HD * 4 <= 96 << 20) {
    while (cluster < 8 && 2 * units * cluster <= kFewUnits && cluster * kBothTurn < a.budget) cluster *= 2;
    const cudaError_t e = choice_memory<evict_kernel<HD>>();
    return e != cudaSuccess ? e : launch_clusters(evict_kernel<HD>, p, cluster, kEvictThreads, smem, st);
  }
  cudaError_t e = choice_memory<evict_choice_kernel>();
  if (e != cudaSuccess) return e;
  evict_choice_kernel<<<a.n_seqs * a.Hkv, kEvictThreads, smem, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  while (cluster < 8 && cluster * kMoveTurn < a.budget) cluster *= 2;
  return launch_clusters(evict_move_kernel<HD>, p, cluster, kMoveThreads, 0, st);
}

}  // namespace

cudaError_t cache_evict(const CacheEvict &a, int *err, cudaStream_t st) {
  if (a.n_seqs == 0) return cudaSuccess;
  EvictArgs p{};
  p.a = a;
  p.err = err;
  const int slots = (int)(std::min)((long long)a.max_pages * a.pg, (long long)kEvictMostSlots);
  p.words = 4 * ceil_div(slots, 128);  // (whole groups of 128 slots)
  p.keys = (std::min)(32 * p.words, kEvictKeys);
  p.pg_shift = (a.pg & (a.pg - 1)) ? -1 : __builtin_ctz(a.pg);
  p.vec = a.pg % 4 == 0 && (uintptr_t)a.mass % 16 == 0;
  return a.hd == 128 ? launch_evict<128>(p, slots, st) : launch_evict<64>(p, slots, st);
}

}  // namespace dg
