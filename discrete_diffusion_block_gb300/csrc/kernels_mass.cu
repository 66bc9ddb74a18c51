// Attention weight that each cached key gathers from the new tokens of its
// sequence, out of the log-sum-exp of their rows:
//   mass[j] = (mass[j] for a cached key, 0 for a new one) + sum_{t, h} 2^(x_tjh log2 e - lse_th log2 e),
//   x_tjh = scale q[t][h] . k_j,
// over the tokens t that count (the last `observe`, or all) and see key j, and the
// query heads h of its KV head.
//
// What bounds it: with single tokens the keys are read once, 2 hd bytes each; with
// chunks of rows it is the products, 2 hd flops and an exponential per pair.
//
// The scores are computed transposed, S^T = K Q^T, so that a key is a lane of the
// tensor memory and a thread adds up its key's weights over the rows without any
// exchange: a unit is 256 keys of a (sequence, KV head), two tiles of 128 with a warp
// group each, which stay in shared memory while the tiles of up to 128 rows (tokens x
// heads of the group, staged by one TMA copy) that see any of them go by.  Each row
// tile read from L2 serves both key tiles.  With one row tile, the keys stream
// and the rows stay in L2.  All blocks take equal ranges of the batch's (unit, row
// tile) pairs, found on the device as in the tree attention; a unit that spans
// several blocks leaves a partial sum per block in the workspace, and the block whose
// sum arrives last adds them up in order: no block waits, results repeat bit for bit.
//
// Roles of a block (384 threads): warp 0 copies keys out of the pre-swizzled pages,
// warp 1 the row tiles and their log-sum-exps, warp 2 issues the products from one
// thread, warps 4-7 and 8-11 take the exponentials of the first and second 128 keys.
#include <atomic>

#include "attn_tc.cuh"
#include "f32x2.cuh"
#include "internal.h"

namespace dg {

namespace {

constexpr int kMassThreads = 384;
constexpr int kMassCtas = 152;       // most blocks: one per SM
constexpr int kMassKeys = 256;       // keys of a unit
constexpr int kMassUnitCost = 1;     // cost of starting a unit, in row tiles
constexpr int kMassGaveUp = 64;      // status code of a block that gave up after an earlier kernel
constexpr float kLog2e = 1.4426950408889634f;

struct MassArgs {
  CUtensorMap q_map;  // rows [n_tok][Hq][hd], box 64 x G x T
  KeyMass a;
  int G, T, ctas;     // T: tokens of a row tile
  float scale_log2;
  float *part;                // [2 kMassCtas][kMassKeys]: block c's first piece in 2 c, its last in 2 c + 1
  unsigned long long *count;  // [kMassCtas]: pieces that have arrived of the unit that ends in block c
  unsigned long long ticket;
  int *err;
};

template <int HD>
struct MassSmem {
  static constexpr int HB = HD / 64;
  static constexpr int KR = HD == 128 ? 2 : 3, QR = HD == 128 ? 3 : 4;  // ring depths
  static constexpr int LR = QR + 2;  // log-sum-exps: those of pair i are written once the products of pair i - QR are
                                     // done, which began when the exponentials of pair i - QR - 2 had been taken
  static constexpr size_t tile = (size_t)HB * 16384;  // 128 keys or rows
  static constexpr size_t kring = 0;
  static constexpr size_t qring = kring + 2 * KR * tile;
  static constexpr size_t lse = qring + QR * tile;
  static constexpr size_t bars = lse + LR * 512;
  static constexpr int n_bars = 2 * KR + 2 * QR + 4 + 1;  // full and empty of K, Q, S; drained
  static constexpr size_t slot = bars + n_bars * 8;
  static constexpr size_t bytes = slot + 32;
};

struct MassSeq {
  int row0, n, pre, tf, row_tiles, units;  // tf: the first token that counts
  bool bad;
};

__device__ __forceinline__ MassSeq load_seq(const MassArgs &p, int b) {
  MassSeq s;
  const int o0 = p.a.offsets[b], o1 = p.a.offsets[b + 1];
  s.row0 = o0;
  s.pre = p.a.prefix_lens[b];
  const long long n = (long long)o1 - o0, keys = (long long)s.pre + n;
  const long long room = min((long long)p.a.max_pages * p.a.pg, (long long)0x7fffff00);
  s.bad = n != 0 && (o0 < 0 || n < 0 || o1 > p.a.n_tok || s.pre < 0 || keys > room);
  s.n = s.bad ? 0 : (int)n;
  s.tf = p.a.observe ? max(0, s.n - p.a.observe) : 0;
  s.row_tiles = ceil_div(s.n - s.tf, p.T);
  s.units = s.n ? (int)((keys + kMassKeys - 1) / kMassKeys) : 0;
  return s;
}

// Tokens [t0, t1) that count and see a key of [j0, j1) (j1 - 1 a slot of the sequence).
struct Tokens {
  int t0, t1;
};
__device__ __forceinline__ Tokens seen_by(const MassArgs &p, const MassSeq &s, int j0, int j1) {
  Tokens t;
  t.t0 = max(s.tf, j0 - s.pre);
  t.t1 = j0 < p.a.sinks ? s.n : (int)min((long long)s.n, (long long)j1 - 1 + p.a.window - s.pre);
  return t;
}

// The row tiles of a unit: [first, first + count).  A unit with new keys that no
// token sees takes a tile too: its new keys are set to 0.
struct Rows {
  int first, count;
};
__device__ __forceinline__ Rows unit_rows(const MassArgs &p, const MassSeq &s, int u) {
  const int j0 = u * kMassKeys, j1 = min(j0 + kMassKeys, s.pre + s.n);
  const Tokens t = seen_by(p, s, j0, j1);
  Rows r;
  r.first = r.count = 0;
  if (t.t0 < t.t1) {
    r.first = (t.t0 - s.tf) / p.T;
    r.count = ceil_div(t.t1 - s.tf, p.T) - r.first;
  } else if (j1 > s.pre) {
    r.count = 1;
  }
  return r;
}

// The next unit from u on that a token sees or that holds new keys: between the first
// tokens and the first window there is none.
__device__ __forceinline__ int next_unit(const MassArgs &p, const MassSeq &s, int u, Rows &r) {
  r = unit_rows(p, s, u);
  if (r.count == 0 && u < s.units) {
    u = max(u, min(max(0, s.pre + s.tf - p.a.window + 1), s.pre) / kMassKeys);
    r = unit_rows(p, s, u);
  }
  return u;
}

// Cost of the units of one KV head.
__device__ __forceinline__ int head_cost(const MassArgs &p, const MassSeq &s) {
  int sum = 0;
  Rows r;
#pragma unroll 1
  for (int u = next_unit(p, s, 0, r); u < s.units; u = next_unit(p, s, u + 1, r)) sum += r.count + kMassUnitCost;
  return sum;
}

// The pieces of a block's range: row tiles [q0, q1) of unit (b, g, u).
struct MassWalk {
  MassSeq s;
  Rows r;
  int b, g, u, q0, q1, at, left;
  __device__ __forceinline__ void clip(int from, int n) {
    const int end = min(r.count + kMassUnitCost, from + n);
    q0 = max(0, from - kMassUnitCost);
    q1 = max(0, end - kMassUnitCost);
    left = n - (end - from);
  }
  __device__ __forceinline__ bool begin(const MassArgs &p, int b_, int from, int n) {
    b = b_;
    s = load_seq(p, b);
    const int head = head_cost(p, s);
    g = from / head;
    at = g * head - from;
    u = next_unit(p, s, 0, r);
#pragma unroll 1
    while (at + r.count + kMassUnitCost <= 0) {  // (the head's last unit ends behind `from`)
      at += r.count + kMassUnitCost;
      u = next_unit(p, s, u + 1, r);
    }
    clip(-at, n);
    return q0 < q1 || next(p);
  }
  __device__ __forceinline__ bool next(const MassArgs &p) {
    do {
      if (left <= 0) return false;
      at += r.count + kMassUnitCost;
      u = next_unit(p, s, u + 1, r);
      if (u >= s.units) {
        if (++g == p.a.Hkv) {
          g = 0;
          do {
            if (++b >= p.a.n_seqs) return false;
            s = load_seq(p, b);
          } while (s.n == 0);
        }
        u = next_unit(p, s, 0, r);
      }
      clip(0, left);
    } while (q0 == q1);
    return true;
  }
};

// A block's share: `count` cost units from unit `at` of sequence b on, of the equal
// ranges of `per`.  Found by every warp for itself.
struct MassRange {
  int b, at, count, per;
};
__device__ __forceinline__ MassRange block_range(const MassArgs &p, int lane) {
  const int run = ceil_div(p.a.n_seqs, 32), lo = min(p.a.n_seqs, lane * run), hi = min(p.a.n_seqs, lo + run);
  constexpr unsigned kMost = 1 << 30;  // more than an ascending batch's sum
  unsigned mine = 0;
#pragma unroll 1
  for (int b = lo; b < hi; ++b) {
    const MassSeq s = load_seq(p, b);
    if (s.n) mine = min(mine + (unsigned)(p.a.Hkv * head_cost(p, s)), kMost);
    if (s.bad && blockIdx.x == 0 && threadIdx.x < 32 && p.err) atomicExch(p.err + 1, kBadSequence);
  }
  unsigned incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl = min(incl + v, kMost);
  }
  const int total = (int)__shfl_sync(0xffffffffu, incl, 31);
  MassRange r;
  r.per = (int)(((unsigned)total + (unsigned)p.ctas - 1) / (unsigned)p.ctas);
  const long long first = (long long)r.per * blockIdx.x;
  r.count = (int)min((long long)r.per, total - first);
  r.b = -1;
  r.at = 0;
  const int start = (int)min(first, (long long)total);
  int at = (int)__shfl_up_sync(0xffffffffu, incl, 1);
  if (lane == 0) at = 0;
  const bool here = start >= at && start < (int)incl;
  if (here) {
#pragma unroll 1
    for (int b = lo; b < hi; ++b) {
      const MassSeq s = load_seq(p, b);
      const int n = s.n ? p.a.Hkv * head_cost(p, s) : 0;
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

// A piece's arrival: true in the block whose piece is the unit's last to arrive.
// The word counts arrivals of this launch (its high bits are the launch's own, see
// the tree attention's flags), and is 0 again after the last.
__device__ __forceinline__ bool arrive_last(unsigned long long *word, unsigned long long up, int pieces) {
  const unsigned long long base = up & ~0xfffull;
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

__device__ __forceinline__ bool mass_wait(uint64_t *b, uint32_t parity, int *err, int code, volatile int *abort) {
  return tc::mbar_try_wait(b, parity) || tc::mbar_wait(b, parity, err, code, abort);
}

__device__ __forceinline__ void mass_sync() { asm volatile("barrier.sync 6, 256;\n" ::: "memory"); }

template <int HD>
__global__ void __launch_bounds__(kMassThreads, 1) key_mass_kernel(const __grid_constant__ MassArgs p) {
  using S = MassSmem<HD>;
  constexpr int HB = S::HB, KR = S::KR, QR = S::QR;
  extern __shared__ __align__(1024) unsigned char base[];
  uint64_t *k_full = (uint64_t *)(base + S::bars), *k_empty = k_full + KR;
  uint64_t *q_full = k_empty + KR, *q_empty = q_full + QR;
  uint64_t *s_full = q_empty + QR, *s_empty = s_full + 2, *drained = s_empty + 2;
  uint32_t *tmem_slot = (uint32_t *)(base + S::slot);
  volatile int *abort = (volatile int *)(tmem_slot + 1), *last = abort + 1;
  float *lse2 = (float *)(base + S::lse);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (tc::smem_u32(base) & 1023u) {  // the operand tiles' swizzle needs it: the same in every block
    if (threadIdx.x == 0 && p.err) atomicExch(p.err, kShapeErrorBase + 6);
    return;
  }
  if (threadIdx.x == 0) {
    *abort = 0;
    for (int i = 0; i < KR; ++i) {
      tc::mbar_init(k_full + i, 1);
      tc::mbar_init(k_empty + i, 1);
    }
    for (int i = 0; i < QR; ++i) {
      tc::mbar_init(q_full + i, 1);
      tc::mbar_init(q_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(s_full + i, 1);
      tc::mbar_init(s_empty + i, 8);  // one arrival per warp
    }
    tc::mbar_init(drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  }
  const MassRange range = block_range(p, lane);  // the same in every warp
  MassWalk w;
  if (range.count <= 0 || !w.begin(p, range.b, range.at, range.count)) return;
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(tc::smem_u32(tmem_slot)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  unsigned long long status = 0;
  if (warp == 4) {
    if (p.err) asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];\n" : "=l"(status) : "l"(p.err - 1) : "memory");
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (status >> 32) *abort = 1;  // an earlier kernel gave up
  const uint32_t tmem = *tmem_slot;  // S^T of key tile k, buffer b: columns 128 (2 b + k)

  if (warp == 0) {
    // ---- keys: lane (half, hd block) copies 64 keys of 64 elements -----------------
    int slot = 0, phase = 0, issued = 0;
    bool ok = true, more = true;
    while (ok && more) {
      if (lane == 0) {
        if (issued >= KR) ok = mass_wait(k_empty + slot, phase ^ 1, p.err, 65, abort);
        if (*abort) ok = false;
        if (ok) tc::mbar_expect_tx(k_full + slot, (uint32_t)(2 * S::tile));
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      if (lane < 4 * HB) {
        const int half = lane / HB, blk = lane % HB, j0 = w.u * kMassKeys + 64 * half, end = w.s.pre + w.s.n;
        unsigned char *d = base + S::kring + (size_t)slot * 2 * S::tile + (half >> 1) * S::tile + (size_t)blk * 16384 + (half & 1) * kAttnSlotHalfBytes;
        const bf16 *src = nullptr;
        if (j0 < end) {
          const Tokens t = seen_by(p, w.s, j0, min(j0 + 64, end));
          if (t.t0 < t.t1) {  // pages that hold no such key are not touched
            const int page = p.a.page_tables[(size_t)w.b * p.a.max_pages + j0 / p.a.pg];
            if (page >= 0 && page < p.a.n_pages)
              src = p.a.k_pool + ((size_t)page * p.a.Hkv + w.g) * p.a.pg * HD + (size_t)blk * p.a.pg * 64 + (size_t)(j0 % p.a.pg) * 64;
          }
        }
        tc::bulk_load(d, src ? (const void *)src : (const void *)g_zero_half, kAttnSlotHalfBytes, k_full + slot);
      }
      ++issued;
      if (++slot == KR) {
        slot = 0;
        phase ^= 1;
      }
      more = w.next(p);
    }
    if (!ok && lane == 0) {  // gave up: wait (bounded) for the copies in flight
      for (int i = issued - 1; i >= 0 && i >= issued - KR; --i) {
        const long long t0 = clock64();
        while (!tc::mbar_try_wait(k_full + i % KR, (i / KR) & 1) && clock64() - t0 < tc::kWaitCycles) {
        }
      }
    }
  } else if (warp == 1) {
    // ---- row tiles and their log-sum-exps ------------------------------------------
    int slot = 0, phase = 0, issued = 0, entry = 0;
    bool ok = true, more = true;
    while (ok && more) {
      for (int q = w.q0; ok && q < w.q1; ++q) {
        const int t0 = w.s.tf + (w.r.first + q) * p.T, cols = min(p.T, w.s.n - t0) * p.G;
        // column c: token t0 + c / G, head g G + c % G; rows without a key (-inf) weigh nothing
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = lane + 32 * k, t = c / p.G;
          v[k] = 0.0f;
          if (c < cols) {
            v[k] = p.a.lse[(size_t)(w.s.row0 + t0 + t) * p.a.Hq + w.g * p.G + c - t * p.G] * kLog2e;
            if (v[k] == __int_as_float(0xff800000)) v[k] = __int_as_float(0x7f800000);
          }
        }
        if (lane == 0) {
          if (issued >= QR) ok = mass_wait(q_empty + slot, phase ^ 1, p.err, 66, abort);
          if (*abort) ok = false;
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) lse2[128 * entry + lane + 32 * k] = v[k];
        __syncwarp();
        if (lane == 0) {
          const uint32_t box = 128u * p.T * p.G;
          tc::mbar_expect_tx(q_full + slot, HB * box);
#pragma unroll
          for (int blk = 0; blk < HB; ++blk)
            tc::tma_load_3d(base + S::qring + (size_t)slot * S::tile + (size_t)blk * 16384, &p.q_map, 64 * blk, w.g * p.G, w.s.row0 + t0,
                            q_full + slot);
        }
        ++issued;
        if (++slot == QR) {
          slot = 0;
          phase ^= 1;
        }
        if (++entry == S::LR) entry = 0;
      }
      more = ok && w.next(p);
    }
    if (!ok && lane == 0) {
      for (int i = issued - 1; i >= 0 && i >= issued - QR; --i) {
        const long long t0 = clock64();
        while (!tc::mbar_try_wait(q_full + i % QR, (i / QR) & 1) && clock64() - t0 < tc::kWaitCycles) {
        }
      }
    }
  } else if (warp == 2) {
    // ---- S^T = K Q^T -----------------------------------------------------------------
    if (lane == 0) {
      bool ok = true, more = true;
      int ks = 0, kphase = 0, qs = 0, qphase = 0, i = 0;
      while (ok && more) {
        ok = mass_wait(k_full + ks, kphase, p.err, 67, abort);
        for (int q = w.q0; ok && q < w.q1; ++q, ++i) {
          const int buf = i & 1, t0 = w.s.tf + (w.r.first + q) * p.T, cols = min(p.T, w.s.n - t0) * p.G;
          if (i >= 2) ok = mass_wait(s_empty + buf, ((i >> 1) - 1) & 1, p.err, 68, abort);
          ok = ok && mass_wait(q_full + qs, qphase, p.err, 69, abort);
          if (!ok) break;
          tc::fence_after();
          const uint32_t idesc = tc::idesc_bf16(128, (cols + 15) & ~15);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
              const uint64_t adesc = tc::sw128_desc(tc::smem_u32(base + S::kring + (size_t)(2 * ks + k) * S::tile + (size_t)(kk >> 2) * 16384)) + 2 * (kk & 3);
              const uint64_t bdesc = tc::sw128_desc(tc::smem_u32(base + S::qring + (size_t)qs * S::tile + (size_t)(kk >> 2) * 16384)) + 2 * (kk & 3);
              tc::mma_bf16(tmem + 128 * (2 * buf + k), adesc, bdesc, idesc, kk ? 1u : 0u);
            }
          }
          tc::mma_commit(s_full + buf);
          tc::mma_commit(q_empty + qs);
          if (++qs == QR) {
            qs = 0;
            qphase ^= 1;
          }
        }
        if (!ok) break;
        tc::mma_commit(k_empty + ks);
        if (++ks == KR) {
          ks = 0;
          kphase ^= 1;
        }
        more = w.next(p);
      }
      if (!ok) {  // gave up: wait (bounded) for the products in flight
        tc::mma_commit(drained);
        const long long t0 = clock64();
        while (!tc::mbar_try_wait(drained, 0) && clock64() - t0 < tc::kWaitCycles) {
        }
      }
    }
  } else if (warp >= 4) {
    // ---- weights: thread = key ---------------------------------------------------------
    const int k = (warp - 4) >> 2, tid = threadIdx.x - 128;  // tid: the key's place in the unit
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const unsigned long long up = p.ticket + (uint32_t)status;  // (thread 0 of these warps)
    // Where the key's weight lies: < 0 where none is written (behind the sequence,
    // not seen by any row and not new, on a bad page), and what it was.
    auto place = [&](const MassWalk &u, float &old) {
      const int j = u.u * kMassKeys + tid;
      long long at = -1;
      old = 0.0f;
      if (j < u.s.pre + u.s.n) {
        const Tokens t = seen_by(p, u.s, j, j + 1);
        if (j >= u.s.pre || t.t0 < t.t1) {
          const int page = p.a.page_tables[(size_t)u.b * p.a.max_pages + j / p.a.pg];
          if (page >= 0 && page < p.a.n_pages) {
            at = ((long long)page * p.a.Hkv + u.g) * p.a.pg + j % p.a.pg;
            if (j < u.s.pre) old = p.a.mass[at];
          } else if (p.err) {
            atomicExch(p.err + 1, kBadPage);
          }
        }
      }
      return at;
    };
    int i = 0, piece = 0, entry = 0;
    float old;
    long long at = place(w, old);
    bool ok = true;
    while (true) {
      MassWalk nx = w;
      const bool more = nx.next(p);
      float next_old = 0.0f;
      long long next_at = -1;
      if (more) next_at = place(nx, next_old);
      const int j = w.u * kMassKeys + tid;
      float sum = 0.0f;
      for (int q = w.q0; q < w.q1; ++q, ++i) {
        const int buf = i & 1, t0 = w.s.tf + (w.r.first + q) * p.T, cols = min(p.T, w.s.n - t0) * p.G;
        // the key's columns [c0, c1): tokens from its own on, up to the window's end
        const long long far = (long long)j + p.a.window - w.s.pre - t0;
        const int c0 = min(max(j - w.s.pre - t0, 0), 128) * p.G;
        const int c1 = j < p.a.sinks ? cols : (int)max(0ll, min((long long)cols, far * p.G));
        if (!mass_wait(s_full + buf, (i >> 1) & 1, p.err, 70, abort)) ok = false;
        __syncwarp();
        tc::fence_after();
        const float *ls = lse2 + 128 * entry;
        const f32x2 scale2 = pair(p.scale_log2, p.scale_log2);
        f32x2 s0 = pair(0.0f, 0.0f), s1 = s0;
#pragma unroll 1
        for (int c = 0; c < cols; c += 32) {
          uint32_t x[32];
          tc::tmem_ld32(tmem + 128 * (2 * buf + k) + lane_off + c, x);
          float4 l[8];
#pragma unroll
          for (int m = 0; m < 8; ++m) l[m] = *(const float4 *)(ls + c + 4 * m);
          tc::tmem_ld_wait(x);
          if (c + 32 >= cols) {  // the tile's last columns: the buffer is free for the next but one
            tc::fence_before();
            __syncwarp();
            if (lane == 0) attn_arrive(s_empty + buf);
          }
          const bool all = __all_sync(0xffffffffu, c0 <= c && c1 >= c + 32);
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            const float2 d = split(fma2(pair(__uint_as_float(x[4 * m]), __uint_as_float(x[4 * m + 1])), scale2, pair(-l[m].x, -l[m].y)));
            const float2 e = split(fma2(pair(__uint_as_float(x[4 * m + 2]), __uint_as_float(x[4 * m + 3])), scale2, pair(-l[m].z, -l[m].w)));
            float a0 = ex2(d.x), a1 = ex2(d.y), a2 = ex2(e.x), a3 = ex2(e.y);
            if (!all) {
              const int cc = c + 4 * m;
              a0 = cc >= c0 && cc < c1 ? a0 : 0.0f;
              a1 = cc + 1 >= c0 && cc + 1 < c1 ? a1 : 0.0f;
              a2 = cc + 2 >= c0 && cc + 2 < c1 ? a2 : 0.0f;
              a3 = cc + 3 >= c0 && cc + 3 < c1 ? a3 : 0.0f;
            }
            s0 = add2(s0, pair(a0, a1));
            s1 = add2(s1, pair(a2, a3));
          }
        }
        const float2 r = split(add2(s0, s1));
        sum += r.x + r.y;
        if (++entry == S::LR) entry = 0;
      }
      if (w.q0 == 0 && w.q1 == w.r.count) {
        if (at >= 0 && ok) p.a.mass[at] = old + sum;
      } else {
        // a piece: cost units begin .. of the unit, relative to the first block's range
        const int slot = 2 * blockIdx.x + (piece ? 1 : 0);
        p.part[(size_t)slot * kMassKeys + tid] = sum;
        const int begin = range.per * (int)blockIdx.x + w.at, tiles = begin + kMassUnitCost;
        const int b0 = tiles / range.per, b1 = (tiles + w.r.count - 1) / range.per;
        const int slot0 = 2 * b0 + (begin > b0 * range.per ? 1 : 0);  // a piece of the unit before comes first there
        __threadfence();
        mass_sync();
        if (tid == 0) *last = !*abort && arrive_last(p.count + b1, up, b1 - b0 + 1);
        mass_sync();
        if (*last && at >= 0) {
          __threadfence();
          float total = __ldcg(p.part + (size_t)slot0 * kMassKeys + tid);
          for (int b = b0 + 1; b <= b1; ++b) total += __ldcg(p.part + (size_t)2 * b * kMassKeys + tid);
          p.a.mass[at] = old + total;
        }
      }
      if (!more) break;
      w = nx;
      at = next_at;
      old = next_old;
      ++piece;
    }
  }
  __syncwarp();  // lone-thread roles above: reconverge before the block-wide barrier
  tc::fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort && p.err) atomicCAS(p.err, 0, kMassGaveUp);
  if (warp == 2) {
    tc::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512u));
  }
}

struct MassWorkspace {
  static constexpr size_t part = 0;
  static constexpr size_t count = part + (size_t)2 * kMassCtas * kMassKeys * 4;
  static constexpr size_t bytes = count + (size_t)kMassCtas * 8;
};

// Blocks of a launch on the current device, asked once.
template <int HD>
cudaError_t mass_ctas(int *out) {
  static std::atomic<int> ctas[64];
  static_assert(MassSmem<HD>::bytes <= 232448, "shared memory of the key mass kernel");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int n = ctas[dev].load();
  if (!n) {
    e = cudaFuncSetAttribute(key_mass_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MassSmem<HD>::bytes);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    n = n < kMassCtas ? n : kMassCtas;
    ctas[dev].store(n);
  }
  *out = n;
  return cudaSuccess;
}

template <int HD>
cudaError_t launch_mass(MassArgs &p, cudaStream_t st) {
  const cudaError_t e = mass_ctas<HD>(&p.ctas);
  if (e != cudaSuccess) return e;
  key_mass_kernel<HD><<<p.ctas, kMassThreads, MassSmem<HD>::bytes, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t key_mass_workspace_bytes() { return MassWorkspace::bytes; }

cudaError_t key_mass(const KeyMass &a, void *ws, int *err, cudaStream_t st) {
  if (a.n_tok == 0 || a.n_seqs == 0) return cudaSuccess;
  MassArgs p{};
  p.a = a;
  p.G = a.Hq / a.Hkv;
  p.T = 128 / p.G;
  p.scale_log2 = (float)(1.4426950408889634 * (double)a.scale);
  p.part = (float *)((unsigned char *)ws + MassWorkspace::part);
  p.count = (unsigned long long *)((unsigned char *)ws + MassWorkspace::count);
  p.ticket = new_ticket();
  p.err = err;
  const cudaError_t e = rows_map(&p.q_map, a.q, a.q_stride, a.n_tok, a.Hq, a.hd, p.G, p.T);
  if (e != cudaSuccess) return e;
  return a.hd == 128 ? launch_mass<128>(p, st) : launch_mass<64>(p, st);
}

}  // namespace dg
