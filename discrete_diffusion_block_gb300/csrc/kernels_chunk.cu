// Windowed attention for chunks of many new tokens (a prompt's, a long draft's); the
// tree attention's kernel has the window for batches of few rows.
//   out[t][h] = sum_j p_j v_j,  p = softmax_j(scale q[t][h] . k_j),  lse = log sum_j e^{scale q . k_j}
// over slots j <= s = prefix + t with j > s - window or j < sinks.
//
// What bounds it: 4 hd flops per (row, key) pair on the tensor cores, one exponential
// per pair beside them.  A unit is two tiles of up to 128 rows (tokens x heads of the
// group, consecutive tokens) of a (sequence, KV head): both use every tile of 128 keys
// that is brought into shared memory, each with scores and output sums of its own in
// tensor memory, so that one tile's products run under the other's softmax.  Blocks
// take equal ranges of the batch's (unit, key tile) pairs (ranges.cuh); a unit that
// spans several blocks leaves fp32 output sums, maxima and sums of each in the
// workspace, and the block whose piece arrives last joins them, in the order of the
// keys: no block waits, results repeat bit for bit.
//
// Roles of a block (384 threads): warp 0 copies keys and values out of the
// pre-swizzled pages, warp 2 the rows; warps 1 and 3 issue the products of one row tile
// each, from one thread, taking turns (without turns both tiles' products run at once, and
// then both softmaxes run at once and the tensor core waits); warps 4-7 and 8-11 do the
// softmax of one row tile each (thread = row).  A row's 128 scores are loaded at once
// (tensor memory answers late while products run), for which the other warps give
// registers away (with 168 for all threads 2048 tokens over 30k keys took 4% longer).
//
// Measured (16 query and 8 KV heads of 128): 2048 tokens over 30k keys 370 to 402 us, by
// machine, 68 to 74% of the measured product rate; 16384 tokens with windows of 1024 172 to
// 176 us, 41%: a tenth of a row
// tile's steps are the first tokens', two tenths half masked, and a unit's beginning and
// end (its lengths, first scores, output) take as long as four of its ten steps.
//
// Roundings: P is rounded to bf16 for the second product, whose operands are bf16 as V is
// (the row sum adds the unrounded values; against 64 bits the output, bf16 too, is off by
// 2.0e-3 of its norm, by 1.7e-3 with everything in fp32 up to its own rounding); scores, sums,
// accumulators and partial sums are fp32.
#include <algorithm>
#include <atomic>

#include "attn_tc.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "ranges.cuh"
#include "window.cuh"

namespace dg {

namespace {

constexpr int kChunkThreads = 384;
constexpr int kChunkCtas = 152;    // most blocks: one per SM
constexpr int kChunkGaveUp = 80;   // status code of a block that gave up after an earlier kernel
// Registers of a thread: 168 at the launch, of which the first four warps give 64 each.
constexpr int kChunkFewRegs = 104, kChunkManyRegs = 200;
static_assert(128 * kChunkFewRegs + 256 * kChunkManyRegs <= kChunkThreads * 168, "registers of the block");
constexpr int kChunkKept = 80;     // bytes of a ChunkKept
constexpr int kChunkFlags = 8;     // key tiles whose bad-page flags are kept: more than are ever in flight

struct ChunkArgs {
  CUtensorMap q_map;  // rows [n_tok][Hq][hd], box 64 x G x T
  TreeAttention a;
  int G, T, ctas;     // T: tokens of a row tile
  int wide;           // rows of out begin at multiples of 32 bytes: stored 32 at a time (16384 tokens of 1024 171 us, 176 with 16)
  float scale_log2;
  float4 *part;               // [2 kChunkCtas][2 row tiles][hd / 4][128 rows]
  float2 *state;              // [2 kChunkCtas][2][128]: (m, l) of each row
  unsigned long long *count;  // [2][kChunkCtas]: pieces that have arrived of the unit that ends in block c
  unsigned long long ticket;
  int *err;
};

template <int HD>
struct ChunkSmem {
  static constexpr int HB = HD / 64;
  static constexpr int KR = HD == 128 ? 5 : 10;            // ring depth: tiles of K and V in turn
  static constexpr size_t tile = (size_t)HB * 16384;       // 128 keys or rows
  static constexpr size_t q = 0;                           // [2]
  static constexpr size_t ring = q + 2 * tile;
  static constexpr size_t flags = ring + KR * tile;        // [kChunkFlags] bad halves of a key tile (2 bits)
  static constexpr size_t bars = flags + kChunkFlags * 4;
  // full[KR], empty[KR]; of each row tile: q_full, q_empty, s_full, p_full, pv_done, o_empty, turn, drained; p_half[2]
  static constexpr int n_bars = 2 * KR + 2 * 8 + 2;
  static constexpr size_t kept = bars + n_bars * 8;        // ChunkKept of the 8 softmax warps
  static constexpr size_t slot = kept + 8 * kChunkKept;
  static constexpr size_t bytes = slot + 16;
};

// Units of a sequence: pairs of row tiles; items: key tiles.
struct ChunkList {
  const ChunkArgs &p;
  struct Seq {
    int row0, n, pre, units;
    bool bad;
    __device__ __forceinline__ int visits() const { return units; }
  };
  static constexpr int kUnitCost = 2;
  __device__ __forceinline__ Seq load(int b) const {
    Seq s;
    const int o0 = p.a.offsets[b], o1 = p.a.offsets[b + 1];
    s.row0 = o0;
    s.pre = p.a.prefix_lens[b];
    const long long n = (long long)o1 - o0, keys = (long long)s.pre + n;
    const long long room = min((long long)p.a.max_pages * p.a.pg, (long long)0x7fffff00);
    s.bad = n != 0 && (o0 < 0 || n < 0 || o1 > p.a.n_tok || s.pre < 0 || keys > room);
    s.n = s.bad ? 0 : (int)n;
    s.units = ceil_div(s.n, 2 * p.T);
    return s;
  }
  __device__ __forceinline__ bool even(const Seq &) const { return false; }
  // Key tiles of unit u: item i is key tile i for i < sink, else i - sink + first.
  struct Keys {
    int sink, first, count, low, end;  // the unit's first window begins at slot low, its keys end before slot `end`
  };
  __device__ __forceinline__ Keys keys(const Seq &s, int u) const {
    Keys k;
    const int t0 = u * 2 * p.T;
    k.low = max(0, s.pre + t0 - p.a.window + 1);
    k.end = s.pre + min(s.n, t0 + 2 * p.T);
    k.first = k.low >> 7;
    k.sink = min((p.a.sinks + 127) >> 7, k.first);
    k.count = k.sink + ((k.end + 127) >> 7) - k.first;
    return k;
  }
  __device__ __forceinline__ int items(const Seq &s, int u) const { return keys(s, u).count; }
};
typedef RangeWalk<ChunkList> ChunkWalk;

// What a softmax warp uses only at a piece's beginning and end.  Its steps take all
// registers; left to the compiler this lies in local memory, with parts of what the steps
// use (2048 tokens over 30k keys: 413 us instead of 402).
struct ChunkKept {
  ChunkWalk w;
  int rows, t0, steps, number, piece;
  uint32_t status;
};
static_assert(sizeof(ChunkKept) <= kChunkKept, "");

// Row tile t of the walk's unit within its piece: tokens [t0, t0 + n), and the items
// whose key tiles a row of it sees: below `sink` and in [lo, hi).
struct RowTile {
  int t0, n, sink, lo, hi, steps;
  __device__ __forceinline__ bool live(int i) const { return i < sink || (i >= lo && i < hi); }
};
__device__ __forceinline__ RowTile row_tile(const ChunkList &list, const ChunkWalk &w, const ChunkList::Keys &k, int t) {
  const ChunkArgs &p = list.p;
  RowTile r;
  r.t0 = (2 * w.u + t) * p.T;
  r.n = max(0, min(p.T, w.s.n - r.t0));
  const int low = max(0, w.s.pre + r.t0 - p.a.window + 1) >> 7, end = (w.s.pre + r.t0 + r.n + 127) >> 7;
  r.sink = k.sink;
  // (where the first tokens reach into the window's tiles all are taken; the masks hide what is not seen)
  r.lo = k.sink + ((p.a.sinks + 127) >> 7 > k.first ? 0 : low - k.first);
  r.hi = k.sink + end - k.first;
  if (r.n == 0) r.sink = r.hi = 0;
  r.steps = max(0, min(w.i1, r.sink) - w.i0) + max(0, min(w.i1, r.hi) - max(w.i0, max(r.lo, r.sink)));
  return r;
}

// A bounded wait that costs one test when the phase is over already.
__device__ __forceinline__ bool chunk_wait(uint64_t *b, uint32_t parity, int *err, int code, volatile int *abort) {
  return tc::mbar_try_wait(b, parity) || tc::mbar_wait(b, parity, err, code, abort);
}

template <int HD>
__global__ void __launch_bounds__(kChunkThreads, 1) chunk_attn_kernel(const __grid_constant__ ChunkArgs p) {
  using S = ChunkSmem<HD>;
  constexpr int HB = S::HB, KR = S::KR;
  extern __shared__ __align__(1024) unsigned char base[];
  uint64_t *full = (uint64_t *)(base + S::bars), *empty = full + KR, *tile_bars = empty + KR;
  uint32_t *tmem_slot = (uint32_t *)(base + S::slot);
  volatile int *abort = (volatile int *)(tmem_slot + 1), *last = abort + 1;  // last: [2]
  int *flags = (int *)(base + S::flags);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (tc::smem_u32(base) & 1023u) {  // the operand tiles' swizzle needs it: the same in every block
    if (threadIdx.x == 0 && p.err) atomicExch(p.err, kShapeErrorBase + 7);
    return;
  }
  if (threadIdx.x == 0) {
    *abort = 0;
    for (int i = 0; i < KR; ++i) {
      tc::mbar_init(full + i, 1);
      tc::mbar_init(empty + i, 2);  // both row tiles are done with it
    }
    for (int i = 0; i < 2; ++i) {
      uint64_t *b = tile_bars + 8 * i;
      tc::mbar_init(b, 1);
      tc::mbar_init(b + 1, 1);
      tc::mbar_init(b + 2, 1);
      tc::mbar_init(b + 3, 4);  // one arrival per softmax warp
      tc::mbar_init(b + 4, 1);
      tc::mbar_init(b + 5, 4);
      tc::mbar_init(b + 6, 1);
      tc::mbar_init(b + 7, 1);
      tc::mbar_init(tile_bars + 16 + i, 4);
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  }
  const ChunkList list{p};
  const BlockRange range = block_range(list, p.a.n_seqs, p.a.Hkv, p.ctas, p.err, lane);  // the same in every warp
  ChunkWalk w;
  if (range.count <= 0 || !w.begin(list, range, p.a.n_seqs, p.a.Hkv, lane)) return;
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(tc::smem_u32(tmem_slot)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  unsigned long long status = 0;
  if (warp == 4 || warp == 8)
    if (p.err) asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];\n" : "=l"(status) : "l"(p.err - 1) : "memory");
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (status >> 32) *abort = 1;  // an earlier kernel gave up
  // Row tile t: S at columns 128 t, P (bf16 pairs) over the first 64 of them once S has
  // been read, O at 256 + 128 t.
  const uint32_t tmem = *tmem_slot;

  // Key tiles are numbered through the block's pieces (item number); K of tile n is the
  // ring's 2 n-th tile, V its 2 n + 1-st.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kChunkFewRegs));
    if (warp == 0) {
      // ---- keys and values: lane = 64-key half of a run of up to 16 key tiles -----------
      int slot = 0, phase = 0, issued = 0, number = 0;
      bool ok = true, more = true;
      ChunkList::Keys ks = list.keys(w.s, w.u);
      auto half_key = [&](int i) {
        const int n = i + (lane >> 1);
        return 128 * (n < ks.sink ? n : n - ks.sink + ks.first) + 64 * (lane & 1);
      };
      // the half's entry of the page table; kNotRead where no row sees a key of it (its page is not touched)
      auto entry_of = [&](int i) {
        const int key = half_key(i);
        return i + (lane >> 1) < w.i1 && key < ks.end && (key + 64 > ks.low || key < p.a.sinks)
                   ? table_entry(p.a.page_tables, (size_t)w.b * p.a.max_pages + key / p.a.pg) : kNotRead;
      };
      int i = w.i0, page = entry_of(i);
      while (ok && more) {
        const int n = min(16, w.i1 - i), key = half_key(i);
        const bool off = page != kNotRead && (page < 0 || page >= p.a.n_pages);
        if (off && p.err) atomicExch(p.err + 1, kBadPage);
        const unsigned bad = __ballot_sync(0xffffffffu, off);
        // rows [0, e) of the half are keys, those in [sink, low) are not seen by any row
        const int e = page < 0 || off ? 0 : min(64, ks.end - key);
        const int sink = min(max(p.a.sinks - key, 0), e), low = max(sink, min(max(ks.low - key, 0), e));
        const size_t at = e ? ((size_t)page * p.a.Hkv + w.g) * p.a.pg * HD + (size_t)(key % p.a.pg) * 64 : 0;
        i += n;
        if (i >= w.i1) {
          more = w.next(list, p.a.n_seqs, p.a.Hkv);
          if (more) {
            ks = list.keys(w.s, w.u);
            i = w.i0;
          }
        }
        if (more) page = entry_of(i);
#pragma unroll 1
        for (int j = 0; ok && j < 2 * n; ++j) {
          const bool is_v = j & 1;
          if (lane == 0) {
            if (issued >= KR) ok = chunk_wait(empty + slot, phase ^ 1, p.err, 81, abort);
            if (*abort) ok = false;
            if (ok) {
              if (!is_v) flags[number & (kChunkFlags - 1)] = (int)(bad >> j) & 3;
              tc::mbar_expect_tx(full + slot, (uint32_t)S::tile);
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          if ((lane >> 1) == (j >> 1)) {
            unsigned char *d = base + S::ring + (size_t)slot * S::tile + (lane & 1) * kAttnSlotHalfBytes;
            const bf16 *src = (is_v ? p.a.v_pool : p.a.k_pool) + at;
            // K: the page's other slots too (their scores are masked); V: zeros in place of
            // rows that nothing sees (0 times anything must be 0)
            const int a = e == 0 ? 0 : is_v ? (low > sink ? sink : e) : 64, c = is_v ? low : 64, z = is_v ? e : 64;
#pragma unroll
            for (int blk = 0; blk < HB; ++blk) {
              unsigned char *db = d + (size_t)blk * 16384;
              const bf16 *sb = src + (size_t)blk * p.a.pg * 64;
              if (a > 0) tc::bulk_load(db, sb, 128u * a, full + slot);
              if (a < 64) {  // (a: e, or sink with [low, e) to come)
                const int zero_to = a < z && c > a ? c : 64;
                tc::bulk_load(db + 128 * a, g_zero_half, 128u * (zero_to - a), full + slot);
                if (zero_to < 64) {
                  if (z > c) tc::bulk_load(db + 128 * c, sb + 64 * c, 128u * (z - c), full + slot);
                  if (z < 64) tc::bulk_load(db + 128 * z, g_zero_half, 128u * (64 - z), full + slot);
                }
              }
            }
          }
          __syncwarp();
          number += is_v;
          ++issued;
          if (++slot == KR) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok && lane == 0) {  // gave up: wait (bounded) for the copies in flight
        for (int k = issued - 1; k >= 0 && k >= issued - KR; --k) {
          const long long t0 = clock64();
          while (!tc::mbar_try_wait(full + k % KR, (k / KR) & 1) && clock64() - t0 < tc::kWaitCycles) {
          }
        }
      }
    } else if (warp == 2) {
      // ---- rows ------------------------------------------------------------------------
      if (tc::elect_one()) {
        bool ok = true, more = true;
        int pieces[2] = {0, 0};
        while (ok && more) {
          const ChunkList::Keys ks = list.keys(w.s, w.u);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const RowTile r = row_tile(list, w, ks, t);
            if (r.steps == 0) continue;
            uint64_t *q_full = tile_bars + 8 * t, *q_empty = q_full + 1;
            if (pieces[t]) ok = ok && chunk_wait(q_empty, (pieces[t] - 1) & 1, p.err, 82, abort);
            if (*abort) ok = false;
            if (!ok) break;
            ++pieces[t];
            tc::mbar_expect_tx(q_full, HB * 128u * p.T * p.G);
#pragma unroll
            for (int blk = 0; blk < HB; ++blk)
              tc::tma_load_3d(base + S::q + t * S::tile + (size_t)blk * 16384, &p.q_map, 64 * blk, w.g * p.G, w.s.row0 + r.t0, q_full);
          }
          more = ok && w.next(list, p.a.n_seqs, p.a.Hkv);
        }
        if (!ok) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const long long t0 = clock64();
            while (pieces[t] && !tc::mbar_try_wait(tile_bars + 8 * t, (pieces[t] - 1) & 1) && clock64() - t0 < tc::kWaitCycles) {
            }
          }
        }
      }
    } else {
      // ---- products of row tile t: P V of its step, then S of its next -------------------
      const int t = warp >> 1;  // warps 1 and 3
      uint64_t *q_full = tile_bars + 8 * t, *q_empty = q_full + 1, *s_full = q_full + 2, *p_full = q_full + 3, *pv_done = q_full + 4,
               *o_empty = q_full + 5, *turn = q_full + 6, *drained = q_full + 7, *other_turn = tile_bars + 8 * (t ^ 1) + 6, *p_half = tile_bars + 16 + t;
      const uint32_t t_s = tmem + 128 * t, t_o = tmem + 256 + 128 * t;
      if (tc::elect_one()) {
        bool ok = true, more = true;
        int k_slot = 0, k_phase = 0, pieces = 0, steps = 0, turns = 0;  // (K of the next item)
        const uint32_t a = (uint32_t)tc::sw128_desc(tc::smem_u32(base + S::q + t * S::tile));
        const uint32_t kdesc = (uint32_t)tc::sw128_desc(tc::smem_u32(base + S::ring)), vdesc = (uint32_t)mn_desc(tc::smem_u32(base + S::ring));
        const uint64_t k_high = tc::sw128_desc(0) & 0xffffffff00000000ull, v_high = mn_desc(0) & 0xffffffff00000000ull;
        auto next_slot = [&](int &slot, int &phase) {
          if (++slot == KR) {
            slot = 0;
            phase ^= 1;
          }
        };
        if (t == 0) attn_arrive(turn);  // the first turn
        while (ok && more) {
          const RowTile r = row_tile(list, w, list.keys(w.s, w.u), t);
          const int i0 = w.i0, i1 = w.i1;
          more = w.next(list, p.a.n_seqs, p.a.Hkv);
          int s_left = r.steps;
          bool had = false, pv = false;  // the piece has had a step; P V of the item before is due
          int v_slot = 0, v_phase = 0;   // V of the item before
#pragma unroll 1
          for (int i = i0; i <= i1; ++i) {
            const bool s = i < i1 && r.live(i);
            // what the turn's products need: V of the item before, K of this one; the
            // softmax has read S, and written P over it; the sums are free; the rows
            ok = (i == i0 || chunk_wait(full + v_slot, v_phase, p.err, 85, abort)) && (i == i1 || chunk_wait(full + k_slot, k_phase, p.err, 84, abort)) &&
                 (!pv || (chunk_wait(p_half, steps & 1, p.err, 92, abort) && (had || !pieces || chunk_wait(o_empty, (pieces - 1) & 1, p.err, 87, abort)))) &&
                 (!s || s_left < r.steps || chunk_wait(q_full, pieces & 1, p.err, 83, abort)) && chunk_wait(turn, turns & 1, p.err, 91, abort);
            if (!ok) break;
            ++turns;
            tc::fence_after();
            if (pv) {
              const uint32_t b = vdesc + v_slot * (uint32_t)(S::tile >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)  // 128 keys, 16 (8 columns of P) per MMA; half of them
                mma_bf16_tmem_a(t_o, t_s + 8 * kk, v_high | (b + kk * (2048 >> 4)), tc::idesc_bf16(128, HD) | (1u << 16), had || kk ? 1u : 0u);
              ok = chunk_wait(p_full, steps & 1, p.err, 86, abort);
              if (!ok) break;
              tc::fence_after();
#pragma unroll
              for (int kk = 4; kk < 8; ++kk)
                mma_bf16_tmem_a(t_o, t_s + 8 * kk, v_high | (b + kk * (2048 >> 4)), tc::idesc_bf16(128, HD) | (1u << 16), 1u);
              tc::mma_commit(pv_done);
              had = true;
              // S may be written again (and O rescaled) once P has been read
              ok = chunk_wait(pv_done, steps & 1, p.err, 88, abort);
              if (!ok) break;
              ++steps;
            }
            if (s) {
              const uint32_t b = kdesc + k_slot * (uint32_t)(S::tile >> 4);
#pragma unroll
              for (int kk = 0; kk < HD / 16; ++kk) {
                const uint32_t o = (kk >> 2) * 1024 + 2 * (kk & 3);
                tc::mma_bf16(t_s, k_high | (a + o), k_high | (b + o), tc::idesc_bf16(128, 128), kk ? 1u : 0u);
              }
            }
            attn_arrive(other_turn);
            if (s) {
              tc::mma_commit(s_full);
              if (--s_left == 0) tc::mma_commit(q_empty);
            }
            if (i > i0) attn_arrive(empty + v_slot);  // (P V is done)
            if (i < i1) {
              if (s) tc::mma_commit(empty + k_slot);
              else attn_arrive(empty + k_slot);
              next_slot(k_slot, k_phase);
              v_slot = k_slot;
              v_phase = k_phase;
              next_slot(k_slot, k_phase);
            }
            pv = s;
          }
          if (r.steps) ++pieces;
        }
        if (!ok) {  // gave up: wait (bounded) for the products in flight
          tc::mma_commit(drained);
          const long long t0 = clock64();
          while (!tc::mbar_try_wait(drained, 0) && clock64() - t0 < tc::kWaitCycles) {
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kChunkManyRegs));
    // ---- softmax of row tile t: thread = row -------------------------------------------
    const int t = warp >= 8, q4 = warp & 3, row = threadIdx.x & 127;
    uint64_t *s_full = tile_bars + 8 * t + 2, *p_full = s_full + 1, *pv_done = s_full + 2, *o_empty = s_full + 3, *p_half = tile_bars + 16 + t;
    const float NEG = __int_as_float(0xff800000);
    const uint32_t t_s = tmem + 128 * t + ((uint32_t)(32 * q4) << 16), t_o = t_s + 256;
    const f32x2 scale2 = pair(p.scale_log2, p.scale_log2);
    int step = 0, number = 0, piece = 0;
    ChunkKept &kept = *(ChunkKept *)(base + S::kept + (warp - 4) * kChunkKept);
    do {
      int at, up, low, sinks, jump, key_base, item, skip, steps;
      bool active;
      {
        const ChunkList::Keys ks = list.keys(w.s, w.u);
        const RowTile r = row_tile(list, w, ks, t);
        const int rows = r.n * p.G;
        active = 32 * q4 < rows;
        at = row < rows ? w.s.pre + r.t0 + row / p.G : -1;  // the row's slot
        // The piece's steps: `sinks` key tiles from key_base on, then others, `jump` keys and `skip` items later.
        const int item1 = max(w.i0, max(r.lo, r.sink));
        sinks = max(0, min(w.i1, r.sink) - w.i0);
        key_base = 128 * w.i0;
        jump = 128 * (item1 - ks.sink + ks.first - sinks - w.i0);
        skip = item1 - w.i0 - sinks;
        item = number;
        // masks: keys behind the slot of the warp's first row, or before its last row's window
        up = w.s.pre + r.t0 + 32 * q4 / p.G - 127;
        low = w.s.pre + r.t0 + min(r.n, (32 * q4 + 31) / p.G + 1) - p.a.window;
        steps = r.steps;
        number += w.i1 - w.i0;
        if (lane == 0) kept = ChunkKept{w, rows, r.t0, r.steps, number, piece, (uint32_t)status};
        __syncwarp();
      }
      float m = NEG, l = 0.0f;
#pragma unroll 1
      for (int n = 0; n < steps; ++n, ++step, ++item, key_base += 128) {
        if (n == sinks) {
          key_base += jump;
          item += skip;
        }
        chunk_wait(s_full, step & 1, p.err, 89, abort);
        __syncwarp();
        if (!active) {
          if (lane == 0) {
            attn_arrive(p_half);
            attn_arrive(p_full);
          }
          continue;
        }
        tc::fence_after();
        uint32_t x[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::tmem_ld32(t_s + 32 * c, x[c]);
        const int bad = flags[item & (kChunkFlags - 1)];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::tmem_ld_wait(x[c]);  // ties every loaded register to the wait
        if (key_base > up || (key_base < low && key_base + 128 > p.a.sinks) || bad) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const unsigned long long see = (bad >> h & 1) || at < 0 ? 0ull : window_bits(at, key_base + 64 * h, p.a.window, p.a.sinks);
            // (a warp's rows are few tokens: one or two of the four columns' ranges need masks)
#pragma unroll
            for (int c = 2 * h; c < 2 * h + 2; ++c) {
              const uint32_t bits = (uint32_t)(see >> 32 * (c & 1));
              if (__all_sync(0xffffffffu, bits == 0xffffffffu)) continue;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!(bits >> j & 1u)) x[c][j] = 0xff800000u;
            }
          }
        }
        // maximum of the raw scores (the scale is positive): four chains
        float a0 = NEG, a1 = NEG, a2 = NEG, a3 = NEG;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            a0 = fmaxf(fmaxf(a0, __uint_as_float(x[c][j])), __uint_as_float(x[c][j + 1]));
            a1 = fmaxf(fmaxf(a1, __uint_as_float(x[c][j + 2])), __uint_as_float(x[c][j + 3]));
            a2 = fmaxf(fmaxf(a2, __uint_as_float(x[c][j + 4])), __uint_as_float(x[c][j + 5]));
            a3 = fmaxf(fmaxf(a3, __uint_as_float(x[c][j + 6])), __uint_as_float(x[c][j + 7]));
          }
        const float tmax = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3)) * p.scale_log2;
        const float m_new = fmaxf(m, tmax), m_old = m;
        const bool grow = m_new > m + kRescaleLog2;  // false while both are -inf
        if (grow) m = m_new;
        const float nmu = m == NEG ? 0.0f : -m;
        const f32x2 nmu2 = pair(nmu, nmu);
        // rows whose maximum grew: O (and l) to the new reference, O <- O 2^(m_old - m)
        // (P V of every earlier step is done)
        float f = 1.0f;
        if (n && __any_sync(0xffffffffu, grow)) {
          f = grow ? ex2(m_old - m) : 1.0f;  // m_old = -inf: 0 (O holds zeros)
#pragma unroll 1
          for (int c = 0; c < HD; c += 32) {
            uint32_t o[32];
            tc::tmem_ld32(t_o + c, o);
            tc::tmem_ld_wait(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st32(t_o + c, o);
          }
        }
        f32x2 sum0 = pair(0.0f, 0.0f), sum1 = sum0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 d = split(fma2(pair(__uint_as_float(x[c][j]), __uint_as_float(x[c][j + 1])), scale2, nmu2));
            const float p0 = ex2(d.x), p1 = ex2(d.y);
            pk[j >> 1] = pack_bf16(p0, p1);
            if (j & 2) sum1 = add2(sum1, pair(p0, p1));
            else sum0 = add2(sum0, pair(p0, p1));
          }
          tmem_st16(t_s + 16 * c, pk);
          if (c == 1) {  // P V of the first 64 keys may begin (the whole tile's at once: 16384 tokens of 1024 2.5% more)
            asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
            tc::fence_before();
            __syncwarp();
            if (lane == 0) attn_arrive(p_half);
            __syncwarp();  // (the next store takes all lanes together)
          }
        }
        const float2 sum = split(add2(sum0, sum1));
        l = l * f + (sum.x + sum.y);
        asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");  // P (and O) written before the release
        tc::fence_before();
        __syncwarp();
        if (lane == 0) attn_arrive(p_full);
      }
      w = kept.w;
      number = kept.number;
      piece = kept.piece;
      steps = kept.steps;
      status = kept.status;
      const int rows = kept.rows, token = kept.t0 + row / p.G, head = w.g * p.G + row % p.G;
      const bool whole = w.i0 == 0 && w.i1 == w.items;
      const int slot = 2 * blockIdx.x + (piece++ ? 1 : 0);
      __syncwarp();
      if (rows == 0) continue;
      if (steps) chunk_wait(pv_done, (step - 1) & 1, p.err, 90, abort);
      __syncwarp();
      bf16 *dst = p.a.out + (size_t)(w.s.row0 + token) * p.a.out_stride + (size_t)head * HD;
      float *lse = p.a.lse ? p.a.lse + (size_t)(w.s.row0 + token) * p.a.Hq + head : nullptr;
      if (active) {
        tc::fence_after();
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        float4 *part = p.part + (size_t)(2 * slot + t) * (HD / 4) * 128 + row;
        if (steps) {
#pragma unroll 1
          for (int c = 0; c < HD; c += 32) {
            uint32_t v[32];
            tc::tmem_ld32(t_o + c, v);
            tc::tmem_ld_wait(v);
            if (row < rows && whole) {
#pragma unroll
              for (int j = 0; j < 32; j += 16) {
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = pack_bf16(__uint_as_float(v[j + 2 * i]) * inv, __uint_as_float(v[j + 2 * i + 1]) * inv);
                if (p.wide) {
                  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst + c + j), "r"(o[0]), "r"(o[1]), "r"(o[2]),
                               "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                               : "memory");
                } else {
                  *(uint4 *)(dst + c + j) = make_uint4(o[0], o[1], o[2], o[3]);
                  *(uint4 *)(dst + c + j + 8) = make_uint4(o[4], o[5], o[6], o[7]);
                }
              }
            } else if (row < rows) {
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                part[(size_t)((c + j) >> 2) * 128] = make_float4(__uint_as_float(v[j]), __uint_as_float(v[j + 1]), __uint_as_float(v[j + 2]),
                                                                 __uint_as_float(v[j + 3]));
            }
            __syncwarp();  // (the next load takes all lanes together)
          }
          tc::fence_before();
        }
        if (row < rows) {
          if (!whole) p.state[(size_t)(2 * slot + t) * 128 + row] = make_float2(l == l ? m : -NEG, l);  // (a NaN row: see the tree attention)
          else if (lse) *lse = fmaf(m, kLn2, logf(l));
        }
      }
      __syncwarp();
      if (steps && lane == 0) attn_arrive(o_empty);
      if (whole) continue;
      // ---- a piece: the last block to arrive joins the unit's rows of this tile
      const UnitBlocks blocks = unit_blocks(w, range.per);
      __threadfence();
      asm volatile("barrier.sync %0, 128;\n" ::"r"(1 + t) : "memory");
      if (row == 0)
        last[t] = !*abort && arrive_last(p.count + (size_t)t * kChunkCtas + blocks.last, p.ticket + (uint32_t)status, blocks.last - blocks.first + 1);
      asm volatile("barrier.sync %0, 128;\n" ::"r"(1 + t) : "memory");
      if (!last[t] || row >= rows) continue;
      __threadfence();
      // (32 columns at a time: as one stretch of code for all, 16384 tokens of 1024 took 3% more)
      float top = NEG, L = 0.0f;
      for (int b = blocks.first; b <= blocks.last; ++b) top = fmaxf(top, __ldcg(&p.state[(size_t)(2 * blocks.slot(b) + t) * 128 + row].x));
#pragma unroll 1
      for (int c = 0; c < HD / 4; c += 8) {
        float4 acc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        L = 0.0f;
#pragma unroll 1
        for (int b = blocks.first; b <= blocks.last; ++b) {
          const size_t piece_at = (size_t)(2 * blocks.slot(b) + t);
          const float2 ml = __ldcg(p.state + piece_at * 128 + row);
          const float f = ml.x == NEG ? 0.0f : ex2(ml.x - top);
          if (f == 0.0f) continue;  // (a tile that saw none of the piece's keys has left no sums)
          L += f * ml.y;
          const float4 *src = p.part + (piece_at * (HD / 4) + c) * 128 + row;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 v = __ldcg(src + (size_t)j * 128);
            acc[j].x += f * v.x;
            acc[j].y += f * v.y;
            acc[j].z += f * v.z;
            acc[j].w += f * v.w;
          }
        }
        const float inv = L > 0.0f ? 1.0f / L : L == L ? 0.0f : L;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          uint4 o;
          o.x = pack_bf16(acc[j].x * inv, acc[j].y * inv);
          o.y = pack_bf16(acc[j].z * inv, acc[j].w * inv);
          o.z = pack_bf16(acc[j + 1].x * inv, acc[j + 1].y * inv);
          o.w = pack_bf16(acc[j + 1].z * inv, acc[j + 1].w * inv);
          *(uint4 *)(dst + 4 * (c + j)) = o;
        }
      }
      if (lse) *lse = fmaf(top, kLn2, logf(L));
    } while (w.next(list, p.a.n_seqs, p.a.Hkv));
  }
  __syncwarp();  // lone-thread roles above: reconverge before the block-wide barrier
  tc::fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort && p.err) atomicCAS(p.err, 0, kChunkGaveUp);
  if (warp == 1) {
    tc::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512u));
  }
}

struct ChunkWorkspace {
  size_t part, state, count, bytes;
};
ChunkWorkspace chunk_workspace(int hd) {
  ChunkWorkspace w;
  w.part = 0;
  w.state = w.part + (size_t)2 * kChunkCtas * 2 * 128 * hd * 4;
  w.count = w.state + (size_t)2 * kChunkCtas * 2 * 128 * sizeof(float2);
  w.bytes = w.count + (size_t)2 * kChunkCtas * 8;
  return w;
}

// Blocks of a launch on the current device, asked once.
template <int HD>
cudaError_t chunk_ctas(int *out) {
  static std::atomic<int> ctas[64];
  static_assert(ChunkSmem<HD>::bytes <= 232448, "shared memory of the chunk attention kernel");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int n = ctas[dev].load();
  if (!n) {
    e = cudaFuncSetAttribute(chunk_attn_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ChunkSmem<HD>::bytes);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    n = n < kChunkCtas ? n : kChunkCtas;
    ctas[dev].store(n);
  }
  *out = n;
  return cudaSuccess;
}

template <int HD>
cudaError_t launch_chunk(ChunkArgs &p, cudaStream_t st) {
  const cudaError_t e = chunk_ctas<HD>(&p.ctas);
  if (e != cudaSuccess) return e;
  chunk_attn_kernel<HD><<<p.ctas, kChunkThreads, ChunkSmem<HD>::bytes, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

// Which kernel: this file's takes pairs of row tiles, and is ahead where there are more
// tiles of 128 rows than blocks (the tree attention's kernel gives each block one until
// then) and sequences fill a tile.  Measured, this kernel and the tree attention's (16 and
// 8 heads of 128): one of 1300 tokens, windows of 1024 (168 tiles) 36 and 45; of 2048 (256)
// 42 and 61; one of 4096, all keys 76 and 117; 8 of 512 over 2k 84 and 103; 13 of 100,
// windows of 512 (208) 34 and 33, 16 of 100 (256) 36 and 41; 64 of 100, windows of 1024 105
// and 140.  One of 1024 tokens (128 tiles), windows of 1024 33 and 24, over 16k keys 118 and
// 129 (the host does not know which); one of 256 over 16k 63 and 47; 64 of 64 tokens,
// windows of 1024 (512, one tile to a unit) 97 and 86; one of 2048 among 64 single ones, 4k
// keys each 276 and 245, windows of 1024 102 and 124.
static bool blocks_full(int n_tok, int Hq) { return (long long)n_tok * Hq > kChunkCtas * 128; }
static bool many_rows(int n_tok, int n_seqs, int Hq, int Hkv) {
  return blocks_full(n_tok, Hq) && (long long)n_tok * (Hq / Hkv) > 128ll * n_seqs;
}

// What is enough for n_tok rows is so for fewer, in however many sequences.
size_t window_attention_workspace_bytes(int n_tok, int n_seqs, int Hq, int Hkv, int hd) {
  const size_t tree = tree_attention_workspace_bytes(n_tok, n_seqs, Hq, Hkv, hd);
  return blocks_full(n_tok, Hq) ? std::max(tree, chunk_workspace(hd).bytes) : tree;
}

cudaError_t window_attention(const TreeAttention &a, void *ws, int *err, cudaStream_t st) {
  if (a.n_tok == 0 || a.n_seqs == 0) return cudaSuccess;
  if (!many_rows(a.n_tok, a.n_seqs, a.Hq, a.Hkv)) return tree_attention(a, ws, err, st);
  const ChunkWorkspace w = chunk_workspace(a.hd);
  ChunkArgs p{};
  p.a = a;
  p.G = a.Hq / a.Hkv;
  p.T = 128 / p.G;
  p.wide = (uintptr_t)a.out % 32 == 0 && a.out_stride % 16 == 0;
  p.scale_log2 = (float)(1.4426950408889634 * (double)a.scale);
  p.part = (float4 *)((unsigned char *)ws + w.part);
  p.state = (float2 *)((unsigned char *)ws + w.state);
  p.count = (unsigned long long *)((unsigned char *)ws + w.count);
  p.ticket = new_ticket();
  p.err = err;
  const cudaError_t e = rows_map(&p.q_map, a.q, a.q_stride, a.n_tok, a.Hq, a.hd, p.G, p.T);
  if (e != cudaSuccess) return e;
  return a.hd == 128 ? launch_chunk<128>(p, st) : launch_chunk<64>(p, st);
}

}  // namespace dg
