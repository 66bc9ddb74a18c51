// Equal ranges of a batch's work for the blocks of a launch, found on the device
// from the sequences' lengths: every sequence has, for each KV head, the same list of
// units, a unit has one item or more (tiles that go by while its operand stays), and
// costs its items plus kUnitCost for starting it.  A block takes a range of the
// costs' running sum; ranges may begin and end inside a unit.
//
// A list L has: L::Seq, with n (0: nothing to do), bad and visits() (units of a KV
// head, 1 or more where n > 0); L::kUnitCost; load(b); even(s) (all its units have one
// item); items(s, i) of unit i.
#pragma once
#include "common.cuh"
#include "internal.h"

namespace dg {

namespace {

constexpr unsigned kMostCost = 1u << 30;  // more than an ascending batch's cost: offsets that overlap stop here

// Cost of the units of one KV head; run by the whole warp for one sequence.
template <class L>
__device__ __forceinline__ int head_cost(const L &list, const typename L::Seq &s, int lane) {
  const int n = s.visits();
  if (list.even(s)) return n * (1 + L::kUnitCost);
  int sum = 0;
#pragma unroll 1
  for (int i = lane; i < n; i += 32) sum += list.items(s, i) + L::kUnitCost;
  return (int)min(__reduce_add_sync(0xffffffffu, (unsigned)min(sum, 1 << 26)), kMostCost);
}

// Inclusive sum over the lanes, up to kMostCost.
__device__ __forceinline__ unsigned lane_sums(unsigned v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = min(v + x, kMostCost);
  }
  return v;
}

// A block's share: `count` cost units from unit `at` of sequence b on, of the equal
// ranges of `per`.  Found by every warp for itself, 32 sequences at a time: their
// cost, then the sequence in which the range begins.  Short lists are added up by the
// sequence's lane, long ones by the warp, one after the other.
struct BlockRange {
  int b, at, count, per;
};
constexpr int kShortList = 16;
template <class L>
__device__ __forceinline__ BlockRange block_range(const L &list, int n_seqs, int heads, int ctas, int *err, int lane) {
  BlockRange r;
  r.b = r.at = r.count = r.per = 0;
  unsigned first = 0, cost = 0;
#pragma unroll 1
  for (int round = 0; round < 2; ++round) {
    unsigned total = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < n_seqs; b0 += 32) {
      if (round == 0 || n_seqs > 32) {  // (else they are still there)
        const bool there = b0 + lane < n_seqs;
        const typename L::Seq s = list.load(min(b0 + lane, n_seqs - 1));
        const int visits = there && s.n ? s.visits() : 0;
        const bool lengthy = visits > kShortList && !list.even(s);
        long long c = 0;
        if (visits && list.even(s)) {
          c = (long long)visits * (1 + L::kUnitCost);
        } else if (!lengthy) {
#pragma unroll 1
          for (int i = 0; i < visits; ++i) c += list.items(s, i) + L::kUnitCost;
        }
#pragma unroll 1
        for (unsigned many = __ballot_sync(0xffffffffu, lengthy); many; many &= many - 1) {
          const int l = __ffs(many) - 1, h = head_cost(list, list.load(b0 + l), lane);
          if (lane == l) c = h;
        }
        if (there && s.bad && round == 0 && blockIdx.x == 0 && threadIdx.x < 32 && err) atomicExch(err + 1, kBadSequence);
        cost = (unsigned)min(c * heads, (long long)kMostCost);
      }
      const unsigned incl = lane_sums(cost, lane);
      if (round) {
        const unsigned end = min(total + incl, kMostCost), begin = end - min(cost, end);
        const unsigned here = __ballot_sync(0xffffffffu, first >= begin && first < end);
        if (here) {
          const int l = __ffs(here) - 1;
          r.b = b0 + l;
          r.at = __shfl_sync(0xffffffffu, (int)(first - begin), l);
          return r;
        }
      }
      total = min(total + __shfl_sync(0xffffffffu, incl, 31), kMostCost);
    }
    if (round == 0) {
      r.per = (int)((total + ctas - 1) / ctas);
      const long long at = (long long)r.per * blockIdx.x;
      if (at >= total) return r;
      first = (unsigned)at;
      r.count = (int)min((unsigned)r.per, total - first);
    }
  }
  r.count = 0;
  return r;
}

// The pieces of a block's range: items [i0, i1) of unit u of (sequence b, KV head g).
// at: where the unit begins, relative to the range; left: what the range holds behind
// the piece.
template <class L>
struct RangeWalk {
  typename L::Seq s;
  int b, g, u, items, i0, i1, at, left;
  __device__ __forceinline__ void clip(int from, int n) {
    const int end = min(items + L::kUnitCost, from + n);
    i0 = max(0, from - L::kUnitCost);
    i1 = max(0, end - L::kUnitCost);
    left = n - (end - from);
  }
  // Run by a whole warp.  false: the range holds no item.
  __device__ __forceinline__ bool begin(const L &list, const BlockRange &range, int n_seqs, int heads, int lane) {
    b = range.b;
    s = list.load(b);
    const int head = head_cost(list, s, lane), visits = s.visits();
    g = range.at / head;
    const int rem = range.at - g * head;
    if (list.even(s)) {
      u = rem / (1 + L::kUnitCost);
      at = u * (1 + L::kUnitCost) - rem;
    } else {  // 32 units at a time
      int before = 0;
      u = visits - 1;
      at = 0;
#pragma unroll 1
      for (int k0 = 0; k0 < visits; k0 += 32) {
        const int cost = k0 + lane < visits ? list.items(s, k0 + lane) + L::kUnitCost : 0;
        const int incl = (int)lane_sums((unsigned)cost, lane);
        const unsigned here = __ballot_sync(0xffffffffu, rem < before + incl);
        if (here) {
          const int l = __ffs(here) - 1;
          u = k0 + l;
          at = __shfl_sync(0xffffffffu, before + incl - cost - rem, l);
          break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    items = list.items(s, u);
    clip(-at, range.count);
    return i0 < i1 || next(list, n_seqs, heads);
  }
  __device__ __forceinline__ bool next(const L &list, int n_seqs, int heads) {
    do {
      if (left <= 0) return false;
      at += items + L::kUnitCost;
      if (++u == s.visits()) {
        u = 0;
        if (++g == heads) {
          g = 0;
          do {
            if (++b >= n_seqs) return false;
            s = list.load(b);
          } while (s.n == 0);
        }
      }
      items = list.items(s, u);
      clip(0, left);
    } while (i0 == i1);
    return true;
  }
};

// Of a unit that spans several blocks: those of its pieces, first .. last, and the
// slot of the first (block c keeps its first piece in slot 2 c, its last in 2 c + 1).
struct UnitBlocks {
  int first, last, slot0;
  __device__ __forceinline__ int slot(int block) const { return block == first ? slot0 : 2 * block; }
};
template <class L>
__device__ __forceinline__ UnitBlocks unit_blocks(const RangeWalk<L> &w, int per) {
  const int begin = per * (int)blockIdx.x + w.at, item = begin + L::kUnitCost;
  UnitBlocks u;
  u.first = item / per;
  u.last = (item + w.items - 1) / per;
  u.slot0 = 2 * u.first + (begin > u.first * per ? 1 : 0);  // a piece of the unit before comes first there
  return u;
}

// A piece's arrival: true in the block whose piece is the unit's last to arrive.  The
// word counts arrivals; its high bits are the launch's own: up = the call's ticket,
// plus the epoch of the status word.  A launch that gives up may leave counts behind,
// and a captured call has the same ticket in every replay; but a launch that gives up
// also leaves its code in the status word, later launches give up while that is set,
// and dg_op_status, which clears it, moves the epoch on first.  0 after the last.
__device__ __forceinline__ bool arrive_last(unsigned long long *word, unsigned long long up, int pieces) {
  const unsigned long long base = up * 0x9E3779B97F4A7C15ull & ~0xfffull;  // (another epoch: other high bits)
  unsigned long long old = *(volatile unsigned long long *)word, seen;
  do {
    seen = old;
    old = atomicCAS(word, seen, (seen & ~0xfffull) == base ? seen + 1 : base + 1);
  } while (old != seen);
  const int n = (seen & ~0xfffull) == base ? (int)(seen & 0xfff) + 1 : 1;
  if (n < pieces) return false;
  *(volatile unsigned long long *)word = 0;
  return true;
}

}  // namespace

}  // namespace dg
