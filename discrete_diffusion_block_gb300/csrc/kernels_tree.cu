// Attention of drafted tokens over the paged KV cache, for a batch of uneven
// sequences: token t of sequence b (row offsets[b] + t) sees the sequence's
// prefix_lens[b] cached keys and those of its drafted keys whose bit is set in
// its mask words (without masks: the drafted keys up to itself).
//   out[t][h] = sum_j p_j v_j,  p = softmax_j(scale q[t][h] . k_j)
// over the keys it sees; a row that sees none is zero.
// The same kernel with WIN: windowed attention of batches of few rows (kernels_chunk.cu
// has those of many).  Token t lies at slot prefix + t and sees itself, the window - 1
// slots before it and the first `sinks`; a unit's key tiles are those of the sinks and
// those from its first row's window on, numbered without the gap between them.
//
// What bounds it: every key and value is read once for the n G rows of its
// sequence and KV head (G = Hq / Hkv), 4 n G flops per element of K and V, so
// up to ~275 rows per KV head the cache's bytes are the floor.  The rows of a
// (sequence, KV head) are packed into tiles of 128 (the MMA's M); one tile and
// its sequence's keys, in tiles of 128, are a unit.  Lengths live on the
// device: every block adds up the units' key tiles, and all blocks take equal
// ranges of that sum (a range may end inside a unit, and hold several small
// ones), so that the memory pipes of all SMs stay equally busy however uneven
// the batch is; or, with few units, a part of one unit each (block_range).  A unit
// that lies in one range is written out by its block.  Of
// one that spans several, each block leaves fp32 partial sums and softmax
// states in the workspace and raises a flag; after its own work, each joins a
// share of the unit's rows, once all the unit's flags are up.  The blocks wait
// for one another (for a bounded time), so the launch is cooperative.  Pieces
// are added in the order of the keys: results repeat bit for bit.
//
// Roles of a block (384 threads, as in the canvas attention): warps 0 and 6
// stream K and V tiles through rings of bulk copies out of the pre-swizzled
// pages, across the ends of units; warps 1 and 11 issue S = Q K^T and O += P V
// from one thread each; warps 2-5 and 7-10 do the softmax, two warps per
// quarter of the tile's rows (thread = row, half of a tile's keys each), and
// stage the next unit's rows as soon as the last S of a unit is done.  Quarters
// without rows (a few drafted tokens fill one) skip the arithmetic.
//
// Measured (16 query and 8 KV heads of 128 unless stated): 64 sequences of 24
// tokens over 16k keys 261 us, 6.4 TB/s; 40 ragged sequences of 5 tokens (12 and 4
// heads of 64) 25.4 us; one of 61 tokens over 32k 36 us, of which the keys' stream
// takes 19, at 7.1 TB/s, and launch (2), start (3.5), the last tile and the join (8)
// most of the rest; one token over 2k keys 11.3 to 12.1 us (by machine), all of it
// latency; 16 sequences of one token over 2k 28.8 us.  With WIN: one token of 4096 keys
// 14.1 us, 64 sequences of one token 146 us (6.1 TB/s), one of 1024 tokens, windows of
// 1024, 24 us.
// Slower and not kept: the pieces joined over a cluster's shared memory, or by a
// kernel of their own; rows copied into idle quarters of a tile; no range shorter
// than 3 tiles (one token over 2k: 0.3 us more); the join's code gone through
// beforehand by the idle producers (2 us more).
//
// Roundings: P is rounded to bf16 for the second product (the row sum adds the
// unrounded values); scores, sums, accumulators and partial sums are fp32.
#include <atomic>
#include <chrono>
#include <mutex>

#include "attn_tc.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "window.cuh"

namespace dg {

namespace {

constexpr int kTreeThreads = 384;
constexpr int kTreePvWarp = 11;
constexpr int kTreeCtas = 152;      // most blocks: one per SM
constexpr int kTreeGaveUp = 63;     // status code of a join that gave up, or of a block that did after an earlier kernel
constexpr int kTreeFlags = 8;       // K tiles whose bad-page flags are kept: more than are ever in flight

struct TreeArgs {
  TreeAttention a;
  int G, ctas, may_part;  // may_part: units may be no more than blocks
  float scale_log2, inv_ctas;
  float *part;       // [2 kTreeCtas] slots of [hd / 4][128 rows] float4: block c's first piece in 2 c, its last in 2 c + 1
  float2 *state;     // [2 kTreeCtas][128]: (m, l) of each row
  unsigned long long *flags;  // [2 kTreeCtas]: the launch's value (BlockShare) while the slot holds a piece of this launch
  int *joined;       // [kTreeCtas]: warps that have seen all flags of the unit that ends in block c
  unsigned long long ticket;  // this call's own number
  int *err;
};

template <int HD>
struct TreeSmem {
  static constexpr int HB = HD / 64;
  static constexpr int KR = HD == 128 ? 3 : 6;             // ring depths: 96 KB each for K and V
  static constexpr size_t tile = (size_t)HB * 16384;
  static constexpr size_t q = 0;
  static constexpr size_t kring = q + tile;
  static constexpr size_t vring = kring + KR * tile;
  static constexpr size_t xch = vring + KR * tile;         // [2 buffers][2 halves][128 rows] fp32
  static constexpr size_t flags = xch + 2 * 2 * 128 * 4;       // [kTreeFlags] bad halves of a K tile (2 bits)
  static constexpr size_t bars = flags + kTreeFlags * 4;
  // q_full, k_full[KR], k_empty[KR], v_full[KR], v_empty[KR], s_full[2],
  // s_empty[2], p_full[2], p_empty[2], o_full, o_empty, drained[2]
  static constexpr int n_bars = 1 + 4 * KR + 8 + 4;
  static constexpr size_t share = bars + n_bars * 8 + 16;  // BlockShare
  static constexpr size_t bytes = share + 80;
};

// Rows and keys of one sequence; n = 0 when it has nothing to do or its rows
// or slots lie outside the call's arrays.
struct Seq {
  int row0, n, pre, key_tiles, row_tiles;
  bool bad;
};

__device__ __forceinline__ Seq load_seq(const TreeArgs &p, int b) {
  Seq s;
  const int o0 = p.a.offsets[b], o1 = p.a.offsets[b + 1];
  s.row0 = o0;
  s.pre = p.a.prefix_lens[b];
  const long long n = (long long)o1 - o0, keys = (long long)s.pre + n;
  const long long room = min((long long)p.a.max_pages * p.a.pg, (long long)0x7fffff00);
  s.bad = n != 0 && (o0 < 0 || n < 0 || o1 > p.a.n_tok || s.pre < 0 || keys > room);
  s.n = s.bad ? 0 : (int)n;
  s.key_tiles = s.n ? (int)((keys + 127) >> 7) : 0;
  s.row_tiles = (int)(((long long)s.n * p.G + 127) >> 7);
  return s;
}

// The key tiles of a row tile (tokens t0 .. t1 - 1 of its sequence): without a
// window all of the sequence's; with one those of the first tokens that stay
// visible, then those between the first token's window and the last token.
struct Keys {
  int sink, first, count;  // tile i is key tile i for i < sink, else i - sink + first
  int low, at, end;        // the first token lies at slot `at`, its window begins at slot low; keys end before slot `end`
};
template <bool WIN>
__device__ __forceinline__ Keys unit_keys(const TreeArgs &p, const Seq &s, int rt) {
  Keys k;
  if constexpr (!WIN) {
    k.sink = k.first = k.low = k.at = 0;
    k.count = s.key_tiles;
    k.end = s.pre + s.n;
  } else {
    const int t0 = 128 * rt / p.G, t1 = min(s.n, ceil_div(128 * (rt + 1), p.G));
    k.at = s.pre + t0;
    k.low = max(0, k.at - p.a.window + 1);
    k.end = s.pre + t1;
    k.first = k.low >> 7;
    k.sink = min((p.a.sinks + 127) >> 7, k.first);
    k.count = k.sink + ((k.end + 127) >> 7) - k.first;
  }
  return k;
}

// The cost of a unit in key tiles, for the equal ranges: its tiles, and
// kTreeUnitCost more for starting it (rows staged, the first tile's way through
// all stages, sums written out and joined).  A range's tiles are those of its
// cost units that lie behind the start-up of their unit.  Measured with 2, 3, 4, 5
// in its place: 40 ragged sequences of 5 tokens 24.9, 24.8, 25.5, 26.2 us; 15 of 22
// over 5.5k 20.2, 20.6, 19.4, 20.2; 30 of 6 over 4.7k 18.1, 17.4, 16.9, 16.8; 64 of
// 24 over 16k 260 with each.

// Its units, and the cost of them all; the host has checked that a batch's sum fits 31 bits.
__device__ __forceinline__ int seq_units(const TreeArgs &p, const Seq &s) { return s.n ? p.a.Hkv * s.row_tiles : 0; }
template <bool WIN>
__device__ __forceinline__ int head_cost(const TreeArgs &p, const Seq &s) {  // of one KV head
  if constexpr (!WIN) return s.row_tiles * (s.key_tiles + kTreeUnitCost);
  int sum = 0;
#pragma unroll 1
  for (int rt = 0; rt < s.row_tiles; ++rt) sum += unit_keys<WIN>(p, s, rt).count + kTreeUnitCost;
  return sum;
}
template <bool WIN>
__device__ __forceinline__ int seq_cost(const TreeArgs &p, const Seq &s) {
  return s.n ? p.a.Hkv * head_cost<WIN>(p, s) : 0;
}
// The most key tiles that a unit of the sequence has (with a window: no fewer).
template <bool WIN>
__device__ __forceinline__ int seq_longest(const TreeArgs &p, const Seq &s) {
  if (!WIN || s.n == 0) return s.key_tiles;
  if (s.row_tiles == 1) return unit_keys<WIN>(p, s, 0).count;
  return (int)min((long long)s.key_tiles, ((long long)p.a.window + p.a.sinks + 127 / p.G + 1 + 2 * 127 + 127) >> 7);
}

// The pieces of a block's range: the key tiles [kt0, kt1) of unit (b, g, rt).
// at: where the unit begins, relative to the range; left: what the range holds
// behind the piece's end.
template <bool WIN>
struct Walk {
  Seq s;
  Keys keys;
  int b, g, rt, kt0, kt1, at, left;
  __device__ __forceinline__ int key_tile(int kt) const { return !WIN || kt < keys.sink ? kt : kt - keys.sink + keys.first; }
  __device__ __forceinline__ int tiles() const { return WIN ? keys.count : s.key_tiles; }
  __device__ __forceinline__ int end() const { return WIN ? keys.end : s.pre + s.n; }
  __device__ __forceinline__ void clip(int from, int n) {  // cost units [from, from + n) of the unit
    const int end = min(tiles() + kTreeUnitCost, from + n);
    kt0 = max(0, from - kTreeUnitCost);
    kt1 = max(0, end - kTreeUnitCost);
    left = n - (end - from);
  }
  // one of k equal parts of the sequence's unit u; false: it holds no tile
  __device__ __forceinline__ bool begin_part(const TreeArgs &p, int b_, int u, int part, int k) {
    b = b_;
    s = load_seq(p, b);
    g = u;
    rt = 0;
    if (s.row_tiles > 1) {
      g = u / s.row_tiles;
      rt = u - g * s.row_tiles;
    }
    keys = unit_keys<WIN>(p, s, rt);
    const int each = ceil_div(tiles(), k);
    kt0 = part * each;
    kt1 = min(tiles(), kt0 + each);
    at = left = 0;
    return kt0 < kt1;
  }
  // false: the range holds no tile
  __device__ __forceinline__ bool begin(const TreeArgs &p, int b_, int from, int n) {
    b = b_;
    s = load_seq(p, b);
    if (!WIN || s.row_tiles == 1) {
      keys = unit_keys<WIN>(p, s, 0);
      const int cost = tiles() + kTreeUnitCost, u = from / cost;
      g = u / s.row_tiles;
      rt = u - g * s.row_tiles;
      at = u * cost - from;
    } else {  // (the last unit ends behind `from`)
      const int head = head_cost<WIN>(p, s);
      g = from / head;
      at = g * head - from;
      rt = 0;
      keys = unit_keys<WIN>(p, s, 0);
#pragma unroll 1
      while (at + keys.count + kTreeUnitCost <= 0) {
        at += keys.count + kTreeUnitCost;
        keys = unit_keys<WIN>(p, s, ++rt);
      }
    }
    clip(-at, n);
    return kt0 < kt1 || next(p);
  }
  __device__ __forceinline__ bool next(const TreeArgs &p) {
    do {
      if (left <= 0) return false;
      at += tiles() + kTreeUnitCost;
      if (++rt == s.row_tiles) {
        rt = 0;
        if (++g == p.a.Hkv) {
          g = 0;
          do {
            if (++b >= p.a.n_seqs) return false;
            s = load_seq(p, b);
          } while (s.n == 0);
        }
      }
      keys = unit_keys<WIN>(p, s, rt);
      clip(0, left);
    } while (kt0 == kt1);
    return true;
  }
};

constexpr int kFewPieces = 8;  // pieces of a unit that are joined without barriers
constexpr float kWholeTiles = 4;  // key tiles of a unit that is not worth splitting

// A block's share of the batch: `count` cost units from unit `at` of sequence b
// on, of the equal ranges of `per`; or (k > 0) the part-th of k parts of one unit
// of rows, the at-th of the sequence; unit: its number.  Found by every warp for
// itself: each lane adds up a run of sequences, a scan over the lanes finds the
// sequence in which the share begins.
//
// Equal ranges keep every block busy whatever the lengths, but most blocks end
// one unit and begin another, and a unit's pieces are many.  Where every unit can
// have blocks of its own (there are no more units than blocks) and parts of the
// longest are hardly larger than the equal ranges, a block takes one part: 16
// sequences of one token over 2k keys 32.2 -> 28.9 us, two of 61 over 8k 29.8 ->
// 24.5, one token over 2k 11.7 -> 11.3.  8 parts at most if that is enough, as they
// are joined without barriers; and units of up to 4 tiles stay whole, as a join
// takes as long as 4 tiles (4 sequences of 45 tokens over 273: 13.4 -> 10.5 us).  The
// choice itself costs batches of single tiles 0.2 to 0.4 us.
struct Range {
  int b, at, count, per, k, unit, part;
};
template <bool WIN>
__device__ __forceinline__ Range block_range(const TreeArgs &p, int lane) {
  const int run = ceil_div(p.a.n_seqs, 32), lo = min(p.a.n_seqs, lane * run), hi = min(p.a.n_seqs, lo + run);
  constexpr int kMost = 1 << 30;  // more than an ascending batch's sum: offsets that overlap stop here
  int mine = 0, units = 0, longest = 0;
#pragma unroll 4
  for (int b = lo; b < hi; ++b) {
    const Seq s = load_seq(p, b);
    mine = (int)min((unsigned)mine + (unsigned)seq_cost<WIN>(p, s), (unsigned)kMost);
    units = min(units + min(seq_units(p, s), kTreeCtas + 1), kTreeCtas + 1);
    longest = max(longest, seq_longest<WIN>(p, s));
    if (s.bad && blockIdx.x == 0 && threadIdx.x < 32 && p.err) atomicExch(p.err + 1, kBadSequence);
  }
  Range r;
  r.k = 0;
  if (p.may_part) {
    const int all = __reduce_add_sync(0xffffffffu, units);
    if (all <= p.ctas && all > 0) {
      // (in floating point: the choice need not be exact, only the same everywhere)
      const float cost = (float)__reduce_add_sync(0xffffffffu, (unsigned)mine), most = (float)__reduce_max_sync(0xffffffffu, longest);
      const int k = (int)__fdividef((float)p.ctas + 0.5f, (float)all), few = most <= kWholeTiles ? 1 : min(k, kFewPieces);
      const float limit = cost * p.inv_ctas + 1.5f;
      r.k = most <= max(limit, kWholeTiles) * few ? few : most <= limit * k ? k : 0;
    }
  }
  if (r.k) mine = units;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl = (int)min((unsigned)incl + (unsigned)v, (unsigned)kMost);
  }
  const int total = __shfl_sync(0xffffffffu, incl, 31);
  long long first;
  if (r.k) {
    r.per = 1;
    r.unit = (int)__fdividef((float)blockIdx.x + 0.5f, (float)r.k);  // blocks and parts are few: exact
    r.part = blockIdx.x - r.unit * r.k;
    first = r.unit;
  } else {
    r.per = (int)(((unsigned)total + (unsigned)p.ctas - 1) / (unsigned)p.ctas);
    first = (long long)r.per * blockIdx.x;
  }
  r.count = (int)min((long long)r.per, total - first);
  r.b = -1;
  r.at = 0;
  const int start = (int)min(first, (long long)total);
  int at = __shfl_up_sync(0xffffffffu, incl, 1);  // those of the lanes before
  if (lane == 0) at = 0;
  const bool here = start >= at && start < incl;
  if (here) {
    for (int b = lo; b < hi; ++b) {
      const Seq s = load_seq(p, b);
      const int n = r.k ? seq_units(p, s) : seq_cost<WIN>(p, s);
      if (start < at + n) {
        r.b = b;
        r.at = start - at;
        break;
      }
      at += n;
    }
  }
  const int src = max(0, __ffs(__ballot_sync(0xffffffffu, here)) - 1);
  r.b = __shfl_sync(0xffffffffu, r.b, src);
  r.at = __shfl_sync(0xffffffffu, r.at, src);
  if (r.b < 0) r.count = 0;
  return r;
}

// A bounded wait that costs one test when the phase is over already.
__device__ __forceinline__ bool tree_wait(uint64_t *b, uint32_t parity, int *err, int code, volatile int *abort) {
  return tc::mbar_try_wait(b, parity) || tc::mbar_wait(b, parity, err, code, abort);
}

// The same for a whole warp, whose threads may leave the wait at different
// times: they are together again afterwards, as the tensor-memory instructions
// behind it ask.
__device__ __forceinline__ void warp_wait(uint64_t *b, uint32_t parity, int *err, int code, volatile int *abort) {
  tree_wait(b, parity, err, code, abort);
  __syncwarp();
}

// 64 mask bits of a row from drafted key d0 on (d0 may be negative: prefix
// keys, seen), keys past the row's last one cleared.
__device__ __forceinline__ unsigned long long row_bits(const TreeArgs &p, const Seq &s, int t, int d0) {
  const int nv = s.n - d0;  // keys of the sequence from d0 on
  if (nv <= 0) return 0ull;
  unsigned long long v;
  if (d0 <= -64) {
    v = ~0ull;
  } else if (!p.a.mask) {
    const int k = t + 1 - d0;
    v = k >= 64 ? ~0ull : k <= 0 ? 0ull : (1ull << k) - 1;
  } else {
    const unsigned long long *w = p.a.mask + (size_t)(s.row0 + t) * p.a.mask_words;
    if (d0 < 0) {
      v = (w[0] << -d0) | ((1ull << -d0) - 1);
    } else {
      const int i = d0 >> 6, sh = d0 & 63;
      v = i < p.a.mask_words ? w[i] >> sh : 0ull;
      if (sh && i + 1 < p.a.mask_words) v |= w[i + 1] << (64 - sh);
    }
  }
  return nv >= 64 ? v : v & ((1ull << nv) - 1);
}

__device__ __forceinline__ void st_flag(unsigned long long *p, unsigned long long v) {
  asm volatile("st.relaxed.gpu.global.u64 [%0], %1;\n" ::"l"(p), "l"(v) : "memory");  // after a fence
}
__device__ __forceinline__ unsigned long long ld_flag(const unsigned long long *p) {
  unsigned long long v;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];\n" : "=l"(v) : "l"(p) : "memory");
  return v;
}

// The eight softmax warps meet (the form of the barrier that does not ask a
// warp's threads to arrive together).
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.sync 6, 256;\n" ::: "memory"); }

// A unit that spans the blocks first .. last: its pieces are slot first_slot and
// slot 2 c of the blocks behind the first; row r0 + i is token row0 + (r0 + i) / G.
struct Span {
  int first, last, first_slot, row0, r0, g;
  int shares, i0, rows;  // blocks with a share of its rows; this block's: rows i0 .. i0 + rows - 1
  __device__ __forceinline__ int slot(int s) const { return s == 0 ? first_slot : 2 * (first + s); }
};
// The span of the walk's unit in the block's range.
template <bool WIN>
__device__ __forceinline__ Span unit_span(const TreeArgs &p, const Walk<WIN> &w, const Range &r) {
  Span u;
  if (r.k) {
    u.first = r.unit * r.k;
    u.last = u.first + (w.tiles() - 1) / ceil_div(w.tiles(), r.k);
    u.first_slot = 2 * u.first;
  } else {
    const int begin = r.per * (int)blockIdx.x + w.at, tiles = begin + kTreeUnitCost;
    u.first = tiles / r.per;
    u.last = (tiles + w.tiles() - 1) / r.per;
    u.first_slot = 2 * u.first + (begin > u.first * r.per ? 1 : 0);  // a piece of the unit before comes first there
  }
  u.row0 = w.s.row0;
  u.r0 = 128 * w.rt;
  u.g = w.g;
  const int n_rows = min(128, w.s.n * p.G - u.r0), each = ceil_div(n_rows, u.last - u.first + 1);
  u.shares = ceil_div(n_rows, each);
  u.i0 = min(n_rows, ((int)blockIdx.x - u.first) * each);
  u.rows = min(n_rows, u.i0 + each) - u.i0;
  return u;
}

// What the softmax warps need at their end, kept in shared memory: registers are
// short in their loop.
struct BlockShare {
  // A raised flag of this launch: the call's ticket, plus the epoch of the status
  // word.  A launch that gives up may leave flags up, and a captured call has the
  // same ticket in every replay; but a launch that gives up also leaves its code in
  // the status word, later launches give up while that is set, and dg_op_status,
  // which clears it, moves the epoch on first.  So no launch takes an earlier one's
  // flags for its own.
  unsigned long long up;
  Range range;
  Span head;  // of the first unit
};
static_assert(sizeof(BlockShare) <= 80, "shared memory");

// The status word (in the high half: 0, or what an earlier kernel gave up with) and
// its epoch (low half) in one load: a clear status is never seen with the epoch
// before the clearing.
__device__ __forceinline__ unsigned long long ld_status(const int *err) {
  unsigned long long v = 0;
  if (err) asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];\n" : "=l"(v) : "l"(err - 1) : "memory");
  return v;
}

// The join's scratch, in the idle rings.
struct JoinSmem {
  float2 state[512];      // [rows of the share][pieces], 128 + kTreeCtas at most: (m, l); .x becomes the weight
  float4 sum[256];        // a thread's sum, where several threads share a column's pieces
  float4 piece[32][256];  // [k][thread]: the pieces a thread adds up, copied by itself
};

// Waits (bounded) until the unit's pieces are there, flag s in lane s, s + 32 ..;
// run by every softmax warp for itself.  False: given up.
__device__ __forceinline__ bool pieces_ready(const TreeArgs &p, const Span &u, int n, int lane, unsigned long long up,
                                             volatile int *abort) {
  for (int s = lane; s < n; s += 32) {
    const unsigned long long *flag = p.flags + u.slot(s);
    const long long t0 = clock64();
    while (ld_flag(flag) != up && !*abort) {
      if (clock64() - t0 > tc::kWaitCycles) {
        if (p.err) atomicExch(p.err, kTreeGaveUp);
        *abort = 1;
      }
    }
  }
  __syncwarp();
  return !__any_sync(0xffffffffu, *abort);
}

__device__ __forceinline__ void store_row4(const TreeArgs &p, const Span &u, int i, int hd, int col, float4 v, float inv) {
  const int rg = u.r0 + i, t = rg / p.G, h = u.g * p.G + rg - t * p.G;
  *(uint2 *)(p.a.out + (size_t)(u.row0 + t) * p.a.out_stride + (size_t)h * hd + 4 * col) =
      make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
}

// The log-sum-exp of row i: l the sum of 2^(score - m).
__device__ __forceinline__ void store_lse(const TreeArgs &p, const Span &u, int i, float m, float l) {
  const int rg = u.r0 + i, t = rg / p.G, h = u.g * p.G + rg - t * p.G;
  p.a.lse[(size_t)(u.row0 + t) * p.a.Hq + h] = fmaf(m, kLn2, logf(l));
}

// This block's share of a unit's rows, out of the pieces of all its blocks:
// weights 2^(m_s - m*), pieces in the order of the keys.  Run by 2^lt of the
// softmax threads (tid of them; 256 for more than kFewPieces) after the block's
// last piece.  The last warp to have seen the unit's flags takes them down: the
// next replay of a captured call, whose ticket is the same, has to find them down.
// Latency bound, and run once a launch: what is loaded is loaded together, and
// the code is kept short (straight-line variants for each shape spent more time
// on fetching instructions).
template <int HD, bool WIN>
__device__ __forceinline__ void join_unit(const TreeArgs &p, const Span &u, JoinSmem *scratch, int tid, int lt,
                                          unsigned long long up, volatile int *abort) {
  constexpr int C = HD / 4, LC = HD == 128 ? 5 : 4;  // float4 columns of a row
  const int n = u.last - u.first + 1, i0 = u.i0, rows = u.rows, lane = tid & 31;
  if (rows <= 0) return;
  bool ready = pieces_ready(p, u, n, lane, up, abort);
  static_assert(sizeof(JoinSmem) <= 2 * TreeSmem<HD>::KR * TreeSmem<HD>::tile, "the rings");
  const int mine = 256 >> lt;  // a share counts 8, whether 8 warps join it or 4
  int seen = 0;
  if (lane == 0 && ready) seen = atomicAdd(p.joined + u.last, mine) + mine;
  const float NEG = __int_as_float(0xff800000);
  const float4 *src = (const float4 *)p.part + (size_t)(2 * u.first) * C * 128 + i0;
  const float2 *state = p.state + (size_t)(2 * u.first) * 128 + i0;
  const int odd = u.first_slot & 1;  // the first block's slot is the second of its two
  if (n <= kFewPieces) {
    // 2^(lt - LC) rows abreast; a thread holds all (2^lb or fewer) pieces of 8 >> lb rows at a time
    const int la = lt - LC, r = tid & ((1 << la) - 1), col = tid >> la, lb = n <= 2 ? 1 : n <= 4 ? 2 : 3;
    for (int b0 = 0; ready && b0 < rows; b0 += (8 >> lb) << la) {
      float4 o[8];
      float2 ml[8];
      float mx[8], w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = b0 + r + ((k >> lb) << la), s = k & ((1 << lb) - 1), slot = 2 * s + (s ? 0 : odd);
        ml[k] = make_float2(NEG, 0.0f);
        if (i < rows && s < n) {
          o[k] = __ldcg(src + ((size_t)slot * C + col) * 128 + i);
          ml[k] = __ldcg(state + (size_t)slot * 128 + i);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) mx[k] = ml[k].x;
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) {
        if (d >> lb) break;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (!(k & d)) mx[k] = mx[k | d] = fmaxf(mx[k], mx[k | d]);
      }
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float L = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = b0 + r + ((k >> lb) << la), s = k & ((1 << lb) - 1);
        w[k] = ml[k].x == NEG ? 0.0f : ex2(ml[k].x - mx[k]);
        if (w[k] != 0.0f) {  // (NaN too)
          L += w[k] * ml[k].y;
          acc.x += w[k] * o[k].x;
          acc.y += w[k] * o[k].y;
          acc.z += w[k] * o[k].z;
          acc.w += w[k] * o[k].w;
        }
        if (s == (1 << lb) - 1) {
          if (i < rows) store_row4(p, u, i0 + i, HD, col, acc, L > 0.0f ? 1.0f / L : 0.0f);
          if (WIN && i < rows && col == 0 && p.a.lse) store_lse(p, u, i0 + i, mx[k], L);
          acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          L = 0.0f;
        }
      }
    }
  } else {
    // Many pieces, few rows (128 / n of them in a share): 2^lr rows abreast x C
    // columns x groups of threads that share the pieces.  A thread copies all its
    // pieces to shared memory at once (32 at most: 63 pieces of 3 rows); the rows'
    // weights and the groups' sums go there too.
    int lr = 0;
    while ((1 << lr) < rows && lr < 8 - LC) ++lr;
    const int r = tid & ((1 << lr) - 1), col = (tid >> lr) & (C - 1), group = tid >> (lr + LC), lg = 8 - LC - lr;
    const int per = (n + (1 << lg) - 1) >> lg, s0 = group * per, s1 = min(n, s0 + per);
    int k = 0;
    for (int i = r; ready && i < rows; i += 1 << lr) {
#pragma unroll 4
      for (int s = s0; s < s1; ++s, ++k)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(tc::smem_u32(&scratch->piece[k][tid])),
                     "l"(src + ((size_t)(2 * s + (s ? 0 : odd)) * C + col) * 128 + i)
                     : "memory");
    }
    // the weights, while the pieces are in flight: a warp a row
    float2 *st = scratch->state;
    for (int q = tid >> 5; q < rows; q += 8) {
      float mx = NEG, L = 0.0f;
#pragma unroll 1
      for (int s = lane; s < n; s += 32) {
        float2 v = make_float2(NEG, 0.0f);
        if (ready) v = __ldcg(state + (size_t)(2 * s + (s ? 0 : odd)) * 128 + q);
        st[q * n + s] = v;
        mx = fmaxf(mx, v.x);
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
#pragma unroll 1
      for (int s = lane; s < n; s += 32) {
        const float2 v = st[q * n + s];
        const float f = v.x == NEG ? 0.0f : ex2(v.x - mx);
        L += f * v.y;
        st[q * n + s].x = f;
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
      if (WIN && ready && lane == 0 && p.a.lse) store_lse(p, u, i0 + q, mx, L);
      const float inv = L > 0.0f ? 1.0f / L : 0.0f;
#pragma unroll 1
      for (int s = lane; s < n; s += 32) st[q * n + s].x *= inv;
    }
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    softmax_sync();
    k = 0;
    // (the rounds count the same in every thread: there is a barrier inside)
    for (int b0 = 0; b0 < rows; b0 += 1 << lr) {
      const int i = b0 + r;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (ready && i < rows) {
#pragma unroll 4
        for (int s = s0; s < s1; ++s, ++k) {
          const float f = st[i * n + s].x;
          const float4 v = scratch->piece[k][tid];
          acc.x += f * v.x;
          acc.y += f * v.y;
          acc.z += f * v.z;
          acc.w += f * v.w;
        }
      }
      if (lg) {  // (one round of rows then)
        scratch->sum[tid] = acc;
        softmax_sync();
        if (group == 0) {
#pragma unroll 1
          for (int g = 1; g < 1 << lg; ++g) {
            const float4 v = scratch->sum[tid + (g << (lr + LC))];
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
          }
        }
      }
      if (ready && group == 0 && i < rows) store_row4(p, u, i0 + i, HD, col, acc, 1.0f);
    }
    softmax_sync();  // the scratch is free again
  }
  if (lane == 0 && ready && seen == 8 * u.shares) {
#pragma unroll 1
    for (int s = 0; s < n; ++s) p.flags[u.slot(s)] = 0;
  }
}

template <int HD, bool WIN>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_attn_kernel(const __grid_constant__ TreeArgs p) {
  using S = TreeSmem<HD>;
  constexpr int HB = S::HB, KR = S::KR;
  extern __shared__ __align__(1024) unsigned char base[];
  uint64_t *q_full = (uint64_t *)(base + S::bars);
  uint64_t *k_full = q_full + 1, *k_empty = k_full + KR;
  uint64_t *v_full = k_empty + KR, *v_empty = v_full + KR;
  uint64_t *s_full = v_empty + KR, *s_empty = s_full + 2;
  uint64_t *p_full = s_empty + 2, *p_empty = p_full + 2;
  uint64_t *o_full = p_empty + 2, *o_empty = o_full + 1, *drained = o_empty + 1;
  uint32_t *tmem_slot = (uint32_t *)(drained + 2);
  volatile int *abort = (volatile int *)(tmem_slot + 1);
  int *flags = (int *)(base + S::flags);
  auto k_tile = [&](int slot) { return base + S::kring + (size_t)slot * S::tile; };
  auto v_tile = [&](int slot) { return base + S::vring + (size_t)slot * S::tile; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (tc::smem_u32(base) & 1023u) {  // the operand tiles' swizzle needs it: the same in every block
    if (threadIdx.x == 0 && p.err) atomicExch(p.err, kShapeErrorBase + 5);
    return;
  }
  // Barriers and tensor memory are set up by warps 0 and 1 while every warp
  // finds the block's range; the K producer (warp 0) goes on without waiting
  // for the others.
  if (warp == 0 && lane == 0) {
    *abort = 0;
    tc::mbar_init(q_full, 8);
    for (int i = 0; i < KR; ++i) {
      tc::mbar_init(k_full + i, 1);
      tc::mbar_init(k_empty + i, 1);
      tc::mbar_init(v_full + i, 1);
      tc::mbar_init(v_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(s_full + i, 1);
      tc::mbar_init(s_empty + i, 8);  // one arrival per softmax warp
      tc::mbar_init(p_full + i, 8);
      tc::mbar_init(p_empty + i, 1);
      tc::mbar_init(drained + i, 1);
    }
    tc::mbar_init(o_full, 1);
    tc::mbar_init(o_empty, 8);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  }
  const Range range = block_range<WIN>(p, lane);  // the same in every warp
  Walk<WIN> w;
  if (range.count <= 0 || !(range.k ? w.begin_part(p, range.b, range.at, range.part, range.k)
                                    : w.begin(p, range.b, range.at, range.count)))
    return;
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     tc::smem_u32(tmem_slot)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  // Barriers, `abort` and the tensor memory's address are there after this.
  auto set_up = [&]() {
    tc::fence_before();
    __syncwarp();
    asm volatile("bar.sync 5, %0;\n" ::"n"(kTreeThreads) : "memory");
    tc::fence_after();
  };
  // S double buffer: columns [0, 128) [128, 256); O: [256, 256 + HD); P double
  // buffer (bf16 pairs): [384, 448) [448, 512)

  // Tiles are numbered through all pieces of the block: tile i uses ring slot
  // i % KR and S and P buffer i & 1.
  if (warp == 0 || warp == 6) {
    // ---- K (warp 0) and V (warp 6) producers ---------------------------------
    const bool is_k = warp == 0;
    const bf16 *pool = is_k ? p.a.k_pool : p.a.v_pool;
    unsigned char *ring = base + (is_k ? S::kring : S::vring);
    uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
    int issued = 0, slot = 0, phase = 0;
    bool ok = true;
    int err_seen = 0;
    if (is_k) {
      __syncwarp();
      err_seen = ld_err_word(p.err);
      asm volatile("bar.arrive 5, %0;\n" ::"n"(kTreeThreads) : "memory");
    } else {
      set_up();
    }
    // Of a run of up to 16 tiles each lane holds one 64-key half: its page,
    // kNotRead past the last key.  The next run's entries of the page table (and
    // the next unit's lengths) are loaded while this one's tiles are copied.
    auto half_key = [&](const Walk<WIN> &u, int kt) {
      return WIN ? 128 * u.key_tile(kt + (lane >> 1)) + 64 * (lane & 1) : 128 * kt + 64 * lane;
    };
    auto pages_of = [&](const Walk<WIN> &u, int kt) {
      const int key = half_key(u, kt);
      // (halves that no row sees are not read, nor their entries of the table)
      return kt + (lane >> 1) < u.kt1 && key < u.end() && (!WIN || key + 64 > u.keys.low || key < p.a.sinks)
                 ? table_entry(p.a.page_tables, (size_t)u.b * p.a.max_pages + key / p.a.pg) : kNotRead;
    };
    int kt = w.kt0, page = pages_of(w, kt);
    bool more = true;
    do {
      // Where the half's rows are and how many are copied (the rest of it becomes
      // zero).  K: the page's slots past the last key too (their scores are
      // masked); V: the sequence's own rows only (0 times anything must be 0), with a
      // window those up to row `sink` and from row `low` on.
      const int n = min(16, w.kt1 - kt), key = half_key(w, kt);
      const bool off = page != kNotRead && (page < 0 || page >= p.a.n_pages);
      const int rows = page == kNotRead || off ? 0 : is_k ? 64 : min(64, w.end() - key);
      int sink = 0, low = 0;
      if (WIN && !is_k) {
        sink = min(max(p.a.sinks - key, 0), rows);
        low = max(sink, min(max(w.keys.low - key, 0), rows));
      }
      const bf16 *src = rows ? pool + ((size_t)page * p.a.Hkv + w.g) * p.a.pg * HD + (size_t)(key % p.a.pg) * 64 : pool;
      if (off && p.err) atomicExch(p.err + 1, kBadPage);
      const unsigned bad = __ballot_sync(0xffffffffu, off);  // lanes whose page is outside the pools
      Walk<WIN> nw = w;
      int next_page = 0;
      for (int j = 0; ok && j < n; ++j) {
        if (lane == 0) {
          if (issued >= KR) ok = tree_wait(empty + slot, phase ^ 1, p.err, is_k ? 51 : 50, abort);
          if (*abort) ok = false;
          if (ok) {
            if (is_k) flags[issued & (kTreeFlags - 1)] = (int)(bad >> (2 * j)) & 3;
            tc::mbar_expect_tx(full + slot, (uint32_t)S::tile);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (ok) {
          if ((lane >> 1) == j) {
            unsigned char *d = ring + (size_t)slot * S::tile + (lane & 1) * kAttnSlotHalfBytes;
#pragma unroll
            for (int b = 0; b < HB; ++b) {
              unsigned char *db = d + (size_t)b * 16384;
              const bf16 *sb = src + (size_t)b * p.a.pg * 64;
              if (WIN && low > sink) {
                if (sink > 0) tc::bulk_load(db, sb, 128u * sink, full + slot);
                tc::bulk_load(db + 128 * sink, g_zero_half, 128u * (low - sink), full + slot);
                if (rows > low) tc::bulk_load(db + 128 * low, sb + 64 * low, 128u * (rows - low), full + slot);
              } else if (rows > 0) {
                tc::bulk_load(db, sb, 128u * rows, full + slot);
              }
              if (rows < 64) tc::bulk_load(d + (size_t)b * 16384 + 128 * rows, g_zero_half, 128u * (64 - rows), full + slot);
            }
          }
          if (++issued == 1 && err_seen) *abort = 1;  // an earlier kernel gave up
          if (++slot == KR) {
            slot = 0;
            phase ^= 1;
          }
        }
        __syncwarp();
        if (j == 0) {
          kt += n;
          if (kt >= nw.kt1) {
            more = nw.next(p);
            kt = nw.kt0;
          }
          if (more) next_page = pages_of(nw, kt);
        }
      }
      w = nw;
      page = next_page;
    } while (ok && more);
    if (!ok && lane == 0) {  // gave up: wait (bounded) for the copies in flight
      for (int i = issued - 1; i >= 0 && i >= issued - KR; --i) {
        const long long t0 = clock64();
        while (!tc::mbar_try_wait(full + i % KR, (i / KR) & 1) && clock64() - t0 < tc::kWaitCycles) {
        }
      }
    }
  } else if (warp == 1 || warp == kTreePvWarp) {
    set_up();
    const uint32_t tmem = *tmem_slot, t_s = tmem, t_o = tmem + 256, t_p = tmem + 384;
    if (tc::elect_one()) {
      bool ok = true;
      int i = 0, slot = 0, phase = 0, piece = 0;
      if (warp == 1) {  // ---- S = Q K^T
        const uint32_t idesc = tc::idesc_bf16(128, 128);
        do {
          ok = tree_wait(q_full, piece & 1, p.err, 52, abort);
          for (int kt = w.kt0; ok && kt < w.kt1; ++kt, ++i) {
            const int buf = i & 1;
            if (i >= 2) ok = tree_wait(s_empty + buf, ((i >> 1) - 1) & 1, p.err, 53, abort);
            ok = ok && tree_wait(k_full + slot, phase, p.err, 54, abort);
            if (!ok) break;
            tc::fence_after();
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
              const uint64_t adesc = tc::sw128_desc(tc::smem_u32(base + S::q + (size_t)(kk >> 2) * 16384)) + 2 * (kk & 3);
              const uint64_t bdesc = tc::sw128_desc(tc::smem_u32(k_tile(slot) + (size_t)(kk >> 2) * 16384)) + 2 * (kk & 3);
              tc::mma_bf16(t_s + buf * 128, adesc, bdesc, idesc, kk ? 1u : 0u);
            }
            tc::mma_commit(s_full + buf);
            tc::mma_commit(k_empty + slot);
            if (++slot == KR) {
              slot = 0;
              phase ^= 1;
            }
          }
          ++piece;
        } while (ok && w.next(p));
      } else {  // ---- O += P V
        const uint32_t idesc = tc::idesc_bf16(128, HD) | (1u << 16);  // B (V) N-contiguous
        do {
          if (piece) ok = tree_wait(o_empty, (piece - 1) & 1, p.err, 55, abort);
          for (int kt = w.kt0; ok && kt < w.kt1; ++kt, ++i) {
            const int buf = i & 1;
            ok = tree_wait(p_full + buf, (i >> 1) & 1, p.err, 56, abort) &&
                 tree_wait(v_full + slot, phase, p.err, 57, abort);
            if (!ok) break;
            tc::fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {  // 128 keys, 16 (8 columns of P) per MMA
              const uint64_t bdesc = mn_desc(tc::smem_u32(v_tile(slot))) + (uint64_t)kk * (2048 >> 4);
              mma_bf16_tmem_a(t_o, t_p + 64 * buf + 8 * kk, bdesc, idesc, (kt > w.kt0 || kk) ? 1u : 0u);
            }
            tc::mma_commit(p_empty + buf);
            tc::mma_commit(v_empty + slot);
            if (++slot == KR) {
              slot = 0;
              phase ^= 1;
            }
          }
          if (ok) tc::mma_commit(o_full);
          ++piece;
        } while (ok && w.next(p));
      }
      if (!ok) {  // gave up: wait (bounded) for the MMAs in flight
        uint64_t *bar = drained + (warp == 1 ? 0 : 1);
        tc::mma_commit(bar);
        const long long t0 = clock64();
        while (!tc::mbar_try_wait(bar, 0) && clock64() - t0 < tc::kWaitCycles) {
        }
      }
    }
  } else {
    // ---- softmax warps --------------------------------------------------------
    const int half = warp >= 7 ? 1 : 0;
    const int q4 = warp & 3, row = 32 * q4 + lane;
    const int tid = (warp - (half ? 3 : 2)) * 32 + lane;  // 0 .. 255
    const float NEG = __int_as_float(0xff800000);
    const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
    float *xch = (float *)(base + S::xch);  // [2 buffers][2 halves][128 rows]
    auto pair_sync = [&]() {
      __syncwarp();
      asm volatile("bar.sync %0, 64;\n" ::"r"(1 + q4) : "memory");
    };
    // The piece's query rows into the operand tile (row r: token r / G, head g G + r % G).
    auto stage_q = [&](const Walk<WIN> &u) {
      const int rows = min(128, u.s.n * p.G - 128 * u.rt);
      constexpr int kN = 128 * (HD / 8) / 256;  // chunks of a thread in a full tile
      const int c = tid & (HD / 8 - 1);
      uint4 v[kN];
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int r = (tid + 256 * k) / (HD / 8);
        if (r < rows) {
          const int rg = 128 * u.rt + r, t = rg / p.G, h = u.g * p.G + rg - t * p.G;
          v[k] = *(const uint4 *)(p.a.q + (size_t)(u.s.row0 + t) * p.a.q_stride + (size_t)h * HD + 8 * c);
        }
      }
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int r = (tid + 256 * k) / (HD / 8);
        if (r < rows) *(uint4 *)(base + S::q + (size_t)(c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v[k];
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      __syncwarp();
    };
    // A line of 128 bytes a thread: all of a tile's rows (two lines of HD = 128).
    auto request_q = [&](const Walk<WIN> &u) {
      const int rows = min(128, u.s.n * p.G - 128 * u.rt), r = tid / HB;
      if (r < rows) {
        const int rg = 128 * u.rt + r, t = rg / p.G, h = u.g * p.G + rg - t * p.G;
        asm volatile("prefetch.global.L1 [%0];\n" ::"l"(p.a.q + (size_t)(u.s.row0 + t) * p.a.q_stride + (size_t)h * HD +
                                                        64 * (tid % HB)));
      }
    };
    BlockShare *share = (BlockShare *)(base + S::share);
    const unsigned long long status = tid == 0 ? ld_status(p.err) : 0;
    if (tid == 0) share->range = range;
    stage_q(w);
    set_up();
    if (tid == 0) {
      share->up = p.ticket + (uint32_t)status;  // (read behind a softmax_sync, as the head)
      if (status >> 32) *abort = 1;
    }
    if (lane == 0) attn_arrive(q_full);
    if (tid == 0) share->head = unit_span(p, w, range);  // (read behind a softmax_sync)
    const uint32_t tmem = *tmem_slot, t_s = tmem, t_o = tmem + 256, t_p = tmem + 384;
    // the first unit, if it lies in earlier blocks too, and the last, if it goes
    // on in later ones, are joined at the end (they may be the same)
    const bool join_head = w.kt0 > 0;
    int i = 0, piece = 0;
    while (true) {
      const int rows = min(128, w.s.n * p.G - 128 * w.rt);
      const bool active = 32 * q4 < rows;  // the same in both warps of the quarter
      const int rg = 128 * w.rt + row, t = row < rows ? rg / p.G : 0, h = w.g * p.G + rg - t * p.G;
      float m = NEG, l = 0.0f;  // l: this half's share of the row sum
      // the next piece, found while this one's first keys are on their way, and
      // its rows requested: staging them later must not wait for memory
      Walk<WIN> nx = w;
      const bool more = nx.next(p);  // the same in all softmax warps (never cut short: they meet at named barriers)
      if (more) request_q(nx);
      for (int kt = w.kt0; kt < w.kt1; ++kt, ++i) {
        const int buf = i & 1;
        warp_wait(s_full + buf, (i >> 1) & 1, p.err, 58, abort);
        if (!active) {
          // nothing to compute: the arrivals alone, P's after the buffer's last use
          if (lane == 0) attn_arrive(s_empty + buf);
          if (i >= 2) warp_wait(p_empty + buf, ((i >> 1) - 1) & 1, p.err, 59, abort);
          __syncwarp();
          if (lane == 0) attn_arrive(p_full + buf);
          continue;
        }
        tc::fence_after();
        const int key_base = 128 * w.key_tile(kt) + 64 * half;
        uint32_t x[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tc::tmem_ld32(t_s + buf * 128 + lane_off + 64 * half + 32 * c, x[c]);
#pragma unroll
        for (int c = 0; c < 2; ++c) tc::tmem_ld_wait(x[c]);  // ties every loaded register to the wait
        const int bad = flags[i & (kTreeFlags - 1)];
        tc::fence_before();
        __syncwarp();
        if (lane == 0) attn_arrive(s_empty + buf);
        // keys the row must not see are -inf: only where drafted keys begin, or a page was bad
        // (with a window: where keys are behind the first row's, or before the last row's window)
        const bool some = WIN ? key_base + 64 > w.keys.at + 1 ||
                                    (key_base < w.keys.end - p.a.window && key_base + 64 > p.a.sinks)
                              : key_base + 64 > w.s.pre;
        if (some || bad) {
          unsigned long long see = (bad >> half) & 1 ? 0ull
                                   : WIN             ? window_bits(w.s.pre + t, key_base, p.a.window, p.a.sinks)
                                                     : row_bits(p, w.s, t, key_base - w.s.pre);
          if (row >= rows) see = 0ull;
          const uint32_t lo = (uint32_t)see, hi = (uint32_t)(see >> 32);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (!((lo >> j) & 1u)) x[0][j] = 0xff800000u;
            if (!((hi >> j) & 1u)) x[1][j] = 0xff800000u;
          }
        }
        // maximum of the raw scores (the scale is positive): four chains, then the pair's
        float a0 = NEG, a1 = NEG, a2 = NEG, a3 = NEG;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            a0 = fmaxf(fmaxf(a0, __uint_as_float(x[c][j])), __uint_as_float(x[c][j + 1]));
            a1 = fmaxf(fmaxf(a1, __uint_as_float(x[c][j + 2])), __uint_as_float(x[c][j + 3]));
            a2 = fmaxf(fmaxf(a2, __uint_as_float(x[c][j + 4])), __uint_as_float(x[c][j + 5]));
            a3 = fmaxf(fmaxf(a3, __uint_as_float(x[c][j + 6])), __uint_as_float(x[c][j + 7]));
          }
        const float hmax = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3));
        float *ex = xch + buf * 256;  // the other buffer is in use until both have passed this sync
        ex[half * 128 + row] = hmax;
        pair_sync();
        const float tmax = fmaxf(hmax, ex[(half ^ 1) * 128 + row]) * p.scale_log2;
        const float m_new = fmaxf(m, tmax);
        const bool grow = m_new > m + kRescaleLog2;  // false while both are -inf; the same in both halves
        // P buffer i & 1 is free once P V of tile i - 2 is done
        if (i >= 2) warp_wait(p_empty + buf, ((i >> 1) - 1) & 1, p.err, 60, abort);
        const float m_old = m;
        if (grow) m = m_new;
        const float nmu = m == NEG ? 0.0f : -m;
        const f32x2 scale2 = pair(p.scale_log2, p.scale_log2), nmu2 = pair(nmu, nmu);
        f32x2 sum0 = pair(0.0f, 0.0f), sum1 = sum0;
        const uint32_t prow = t_p + 64 * buf + 32 * half + lane_off;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 d = split(fma2(pair(__uint_as_float(x[c][j]), __uint_as_float(x[c][j + 1])), scale2, nmu2));
            const float p0 = ex2(d.x), p1 = ex2(d.y);
            pk[j >> 1] = pack_bf16(p0, p1);
            if (j & 2) sum1 = add2(sum1, pair(p0, p1));
            else sum0 = add2(sum0, pair(p0, p1));
          }
          tmem_st16(prow + 16 * c, pk);
        }
        const float2 sum = split(add2(sum0, sum1));
        // rows whose maximum grew: O (and l) to the new reference, O <- O 2^(m_old - m);
        // each half rescales its half of the O columns
        float f = 1.0f;
        if (__any_sync(0xffffffffu, grow) && kt > w.kt0) {
          // O must hold P V of every earlier tile of the piece: wait for tile i - 1's
          warp_wait(p_empty + (buf ^ 1), ((i - 1) >> 1) & 1, p.err, 61, abort);
          tc::fence_after();
          f = grow ? ex2(m_old - m) : 1.0f;  // m_old = -inf: 0 (O holds zeros)
#pragma unroll 1
          for (int c = half * (HD / 64); c < (half + 1) * (HD / 64); ++c) {
            uint32_t o[32];
            tc::tmem_ld32(t_o + lane_off + 32 * c, o);
            tc::tmem_ld_wait(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st32(t_o + lane_off + 32 * c, o);
          }
        }
        l = l * f + (sum.x + sum.y);
        asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");  // P (and O) written before the release
        tc::fence_before();
        __syncwarp();
        if (lane == 0) attn_arrive(p_full + buf);
      }
      // every S of this piece is done (its last s_full): the next piece's rows
      if (more) {
        stage_q(nx);
        if (lane == 0) attn_arrive(q_full);
      }
      const bool full_unit = w.kt0 == 0 && w.kt1 == w.tiles();
      const int slot = 2 * blockIdx.x + (piece ? 1 : 0);
      warp_wait(o_full, piece & 1, p.err, 62, abort);  // inactive warps too: o_empty counts one arrival of each a piece
      if (active) {  // the row sum of both halves
        float *ex = xch + (i & 1) * 256;  // as the next tile's maxima
        ex[half * 128 + row] = l;
        pair_sync();
        const float lt = half ? ex[row] + l : l + ex[128 + row];  // keys 0-63 first
        pair_sync();
        tc::fence_after();
        const float inv = lt > 0.0f ? 1.0f / lt : 0.0f;
        bf16 *dst = p.a.out + (size_t)(w.s.row0 + t) * p.a.out_stride + (size_t)h * HD;
        float4 *part = (float4 *)p.part + (size_t)slot * 128 * (HD / 4) + row;
#pragma unroll 1
        for (int c = half * (HD / 64); c < (half + 1) * (HD / 64); ++c) {
          uint32_t v[32];
          __syncwarp();  // the load takes all lanes together (rows of nobody's leave the loop's last turn early)
          tc::tmem_ld32(t_o + lane_off + 32 * c, v);
          tc::tmem_ld_wait(v);
          if (row >= rows) continue;
          if (full_unit) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              uint4 o;
              o.x = pack_bf16(__uint_as_float(v[j]) * inv, __uint_as_float(v[j + 1]) * inv);
              o.y = pack_bf16(__uint_as_float(v[j + 2]) * inv, __uint_as_float(v[j + 3]) * inv);
              o.z = pack_bf16(__uint_as_float(v[j + 4]) * inv, __uint_as_float(v[j + 5]) * inv);
              o.w = pack_bf16(__uint_as_float(v[j + 6]) * inv, __uint_as_float(v[j + 7]) * inv);
              *(uint4 *)(dst + 32 * c + j) = o;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              part[(size_t)(8 * c + (j >> 2)) * 128] = make_float4(__uint_as_float(v[j]), __uint_as_float(v[j + 1]),
                                                                   __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
          }
        }
        // (a row whose sum is NaN: its weight in the join is inf - inf, so the row is NaN)
        if (WIN && full_unit && half == 0 && row < rows && p.a.lse)
          p.a.lse[(size_t)(w.s.row0 + t) * p.a.Hq + h] = fmaf(m, kLn2, logf(lt));
        if (!full_unit && half == 0 && row < rows) p.state[(size_t)slot * 128 + row] = make_float2(lt == lt ? m : -NEG, lt);
        tc::fence_before();
      }
      __syncwarp();
      if (lane == 0) attn_arrive(o_empty);
      if (!more) {
        // At the end, once (a fence in mid-stream waits for every store and load
        // in flight, and the rings run dry): the flags of the first and the last
        // piece, then this block's shares of the units they belong to.
        const bool join_tail = w.kt1 < w.tiles() && (piece || !join_head);
        const Span tail = unit_span(p, w, share->range);
        if (join_head || join_tail) {
          // counted from here by those who see the flag
          if (tid == 0 && join_head && share->head.last == (int)blockIdx.x) p.joined[blockIdx.x] = 0;
          // (found out while the fence waits)
          asm volatile("" ::"r"(tail.first), "r"(tail.last), "r"(tail.first_slot), "r"(tail.shares), "r"(tail.i0), "r"(tail.rows));
          __threadfence();
          softmax_sync();
          if (tid == 0) {
            if (join_head) st_flag(p.flags + 2 * blockIdx.x, share->up);
            if (join_tail) st_flag(p.flags + slot, share->up);
          }
        }
        const Span head = share->head;
        // Two units of few pieces are joined at once, by four warps each: nothing
        // there waits for the other warps.  (One loop: the code is there once.)
        const bool both = join_head && join_tail && head.last - head.first < kFewPieces && tail.last - tail.first < kFewPieces;
#pragma unroll 1
        for (int k = join_head ? 0 : 1; k < (join_tail ? 2 : 1); ++k) {
          if (both && k != tid >> 7) continue;
          join_unit<HD, WIN>(p, k ? tail : head, (JoinSmem *)(base + S::kring), both ? tid & 127 : tid, both ? 7 : 8, share->up, abort);
        }
      }
      if (!more) break;
      w = nx;
      ++piece;
    }
  }
  __syncwarp();  // lone-thread roles above: reconverge before the block-wide barrier
  tc::fence_before();
  __syncthreads();
  // given up: the record stands behind the launch, even if it was cleared meanwhile
  if (threadIdx.x == 0 && *abort && p.err) atomicCAS(p.err, 0, kTreeGaveUp);
  if (warp == 1) {
    tc::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(*tmem_slot), "r"(512u));
  }
}

struct TreeWorkspace {
  size_t part, state, flags, joined, bytes;
};
TreeWorkspace tree_workspace(int hd) {
  TreeWorkspace w;
  w.part = 0;
  w.state = w.part + (size_t)2 * kTreeCtas * 128 * hd * 4;
  w.flags = w.state + (size_t)2 * kTreeCtas * 128 * sizeof(float2);
  w.joined = w.flags + (size_t)2 * kTreeCtas * 8;
  w.bytes = w.joined + (size_t)kTreeCtas * 4;
  return w;
}

}  // namespace

unsigned long long new_ticket() {
  static std::atomic<unsigned long long> count{(unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count()};
  unsigned long long x = count.fetch_add(1) * 0x9E3779B97F4A7C15ull;  // mixed as in splitmix64 (Steele et al., 2014)
  x = (x ^ (x >> 30)) * 0xBF58476D1CE4E5B9ull;
  x = (x ^ (x >> 27)) * 0x94D049BB133111EBull;
  x ^= x >> 31;
  return x ? x : 1;
}

namespace {

// Blocks of a launch on the current device (all of them run together), asked
// once; 0: the kernel does not run there.
template <int HD, bool WIN>
cudaError_t tree_ctas(int *out) {
  static int ctas[64];
  static std::mutex mu;
  using S = TreeSmem<HD>;
  static_assert(S::bytes <= 232448, "shared memory of the tree attention kernel");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (!ctas[dev]) {
    int sms = 0, per_sm = 0;
    e = cudaFuncSetAttribute(tree_attn_kernel<HD, WIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::bytes);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, tree_attn_kernel<HD, WIN>, kTreeThreads, S::bytes);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorLaunchOutOfResources;
    ctas[dev] = sms < kTreeCtas ? sms : kTreeCtas;
  }
  *out = ctas[dev];
  return cudaSuccess;
}

template <int HD, bool WIN>
cudaError_t launch_tree(TreeArgs &p, cudaStream_t st) {
  const cudaError_t e = tree_ctas<HD, WIN>(&p.ctas);
  if (e != cudaSuccess) return e;
  p.inv_ctas = 1.0f / (float)p.ctas;
  // (no use asking where the rows in full tiles are more units than blocks)
  p.may_part = (long long)p.a.Hkv * p.a.n_tok * p.G / 128 <= p.ctas && p.a.Hkv <= p.ctas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.ctas);
  cfg.blockDim = dim3(kTreeThreads);
  cfg.dynamicSmemBytes = TreeSmem<HD>::bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_attn_kernel<HD, WIN>, p);
}

}  // namespace

size_t tree_attention_workspace_bytes(int, int, int, int, int hd) { return tree_workspace(hd).bytes; }

cudaError_t tree_attention(const TreeAttention &a, void *ws, int *err, cudaStream_t st) {
  if (a.n_tok == 0 || a.n_seqs == 0) return cudaSuccess;
  const TreeWorkspace w = tree_workspace(a.hd);
  TreeArgs p{};
  p.a = a;
  p.G = a.Hq / a.Hkv;
  p.scale_log2 = (float)(1.4426950408889634 * (double)a.scale);
  p.part = (float *)((unsigned char *)ws + w.part);
  p.state = (float2 *)((unsigned char *)ws + w.state);
  p.flags = (unsigned long long *)((unsigned char *)ws + w.flags);
  p.joined = (int *)((unsigned char *)ws + w.joined);
  p.ticket = new_ticket();
  p.err = err;
  if (a.window) return a.hd == 128 ? launch_tree<128, true>(p, st) : launch_tree<64, true>(p, st);
  return a.hd == 128 ? launch_tree<128, false>(p, st) : launch_tree<64, false>(p, st);
}

}  // namespace dg
