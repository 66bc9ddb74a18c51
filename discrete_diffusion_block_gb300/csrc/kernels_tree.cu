// Attention of drafted tokens over the paged KV cache, for a batch of uneven
// sequences: token t of sequence b (row offsets[b] + t) sees the sequence's
// prefix_lens[b] cached keys and those of its drafted keys whose bit is set in
// its mask words (without masks: the drafted keys up to itself).
//   out[t][h] = sum_j p_j v_j,  p = softmax_j(scale q[t][h] . k_j)
// over the keys it sees; a row that sees none is zero.
//
// What bounds it: every key and value is read once for the n G rows of its
// sequence and KV head (G = Hq / Hkv), 4 n G flops per element of K and V, so
// up to ~275 rows per KV head the cache's bytes are the floor.  The rows of a
// (sequence, KV head) are packed into tiles of 128 (the MMA's M); one tile and
// its sequence's keys, in tiles of 128, are a unit.  Lengths live on the
// device: every block adds up the units' key tiles, all blocks take equal
// ranges of that sum (a range may end inside a unit, and hold several small
// ones), and the memory pipes of all SMs stay equally busy however uneven the
// batch is.  A unit that lies in one range is written out by its block; the
// fp32 partial sums and softmax states of a unit that spans several go to the
// workspace, and tree_merge_kernel joins them in the order of the keys (the
// sums do not depend on which block ends first, so results repeat bit for bit).
//
// Roles of a block (384 threads, as in the canvas attention): warps 0 and 6
// stream K and V tiles through rings of bulk copies out of the pre-swizzled
// pages, across the ends of units; warps 1 and 11 issue S = Q K^T and O += P V
// from one thread each; warps 2-5 and 7-10 do the softmax, two warps per
// quarter of the tile's rows (thread = row, half of a tile's keys each), and
// stage the next unit's rows as soon as the last S of a unit is done.  Quarters
// without rows (a few drafted tokens fill one) skip the arithmetic.
//
// Roundings: P is rounded to bf16 for the second product, the row sum adds the
// rounded values, so that a row whose weight is on one key returns that value
// unchanged; scores, sums, accumulators and partial sums are fp32.
#include "attn_tc.cuh"
#include "internal.h"

namespace dg {

namespace {

constexpr int kTreeThreads = 384;
constexpr int kTreePvWarp = 11;
constexpr int kTreeCtas = 152;      // one block per SM
constexpr int kTreeFlags = 8;       // K tiles whose bad-page flags are kept: more than are ever in flight

// What block c's first unit needs from tree_merge_kernel: set when the unit
// began in an earlier block and ends in this one.
struct TreeMerge {
  int on, first_cta, first_slot;  // its pieces: slot first_slot of block first_cta, then slot 2 c' of the blocks up to c
  int row0, n_rows, r0, g, pad;   // packed rows of its sequence: row r0 + i is token row0 + (r0 + i) / G
};

struct TreeArgs {
  TreeAttention a;
  int G, min_tiles;
  float scale_log2;
  float *part;       // [2 kTreeCtas] slots of [hd / 4][128 rows] float4
  float2 *state;     // [2 kTreeCtas][128]: (m, l) of each row
  TreeMerge *merge;  // [kTreeCtas]
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
  static constexpr size_t xch = vring + KR * tile;         // [2 halves][128 rows] fp32; the block's scan before
  static constexpr size_t flags = xch + 2 * 128 * 4;       // [kTreeFlags] bad halves of a K tile (2 bits)
  static constexpr size_t bars = flags + kTreeFlags * 4;
  // q_full, k_full[KR], k_empty[KR], v_full[KR], v_empty[KR], s_full[2],
  // s_empty[2], p_full[2], p_empty[2], o_full, o_empty, drained[2]
  static constexpr int n_bars = 1 + 4 * KR + 8 + 4;
  static constexpr size_t bytes = bars + n_bars * 8 + 16 + 1024;
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

__device__ __forceinline__ long long seq_tiles(const TreeArgs &p, const Seq &s) {
  return (long long)p.a.Hkv * s.row_tiles * s.key_tiles;
}

// The pieces of a block's range: the key tiles [kt0, kt1) of unit (b, g, rt).
struct Walk {
  Seq s;
  int b, g, rt, kt0, kt1;
  long long left;
  __device__ __forceinline__ void begin(const TreeArgs &p, int b_, long long at, long long n) {
    b = b_;
    s = load_seq(p, b);
    left = n;
    const long long u = at / s.key_tiles;
    kt0 = (int)(at - u * s.key_tiles);
    g = (int)(u / s.row_tiles);
    rt = (int)(u - (long long)g * s.row_tiles);
    kt1 = (int)min((long long)s.key_tiles, kt0 + left);
  }
  __device__ __forceinline__ bool next(const TreeArgs &p) {
    left -= kt1 - kt0;
    if (left <= 0) return false;
    kt0 = 0;
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
    kt1 = (int)min((long long)s.key_tiles, left);
    return true;
  }
};

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

template <int HD>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_attn_kernel(const __grid_constant__ TreeArgs p) {
  using S = TreeSmem<HD>;
  constexpr int HB = S::HB, KR = S::KR;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *base = (unsigned char *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
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

  // ---- this block's range of the batch's key tiles ---------------------------
  // Each thread adds up a run of sequences; a scan over the threads finds the
  // sequence in which the range begins.
  long long *wsum = (long long *)(base + S::xch);       // [12] warp totals
  long long *where = wsum + 12;                          // [2]: sequence, tile in it
  int *err_seen = (int *)(where + 2);
  const int run = ceil_div(p.a.n_seqs, kTreeThreads);
  const int b_lo = threadIdx.x * run, b_hi = min(p.a.n_seqs, b_lo + run);
  long long mine = 0;
  if (threadIdx.x == 0) *err_seen = ld_err_word(p.err);
  for (int b = b_lo; b < b_hi; ++b) {
    const Seq s = load_seq(p, b);
    mine += seq_tiles(p, s);
    if (s.bad && blockIdx.x == 0 && p.err) atomicExch(p.err + 1, kBadSequence);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  long long total = 0, before = 0;
  for (int w = 0; w < kTreeThreads / 32; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
  const long long per = max((total + gridDim.x - 1) / (long long)gridDim.x, (long long)p.min_tiles);
  const long long start = per * blockIdx.x, count = min(per, total - start);
  if (count <= 0 || *err_seen) {  // the same in every thread
    if (threadIdx.x == 0) p.merge[blockIdx.x].on = 0;
    return;
  }
  long long at = before + incl - mine;
  if (start >= at && start < at + mine) {
    for (int b = b_lo; b < b_hi; ++b) {
      const long long n = seq_tiles(p, load_seq(p, b));
      if (start < at + n) {
        where[0] = b;
        where[1] = start - at;
        break;
      }
      at += n;
    }
  }
  if (threadIdx.x == 0) {
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
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     tc::smem_u32(tmem_slot)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  // S double buffer: columns [0, 128) [128, 256); O: [256, 256 + HD); P double
  // buffer (bf16 pairs): [384, 448) [448, 512)
  const uint32_t t_s = tmem, t_o = tmem + 256, t_p = tmem + 384;
  Walk w;
  w.begin(p, (int)where[0], where[1], count);
  __syncthreads();  // `where` is read before the softmax exchange reuses its place

  // The first unit, when it began in an earlier block and ends here, is joined
  // by tree_merge_kernel.
  if (threadIdx.x == 0) {
    TreeMerge m = {};
    m.on = w.kt0 > 0 && w.kt1 == w.s.key_tiles;
    if (m.on) {
      const long long t0 = start - w.kt0;  // where the unit begins
      m.first_cta = (int)(t0 / per);
      m.first_slot = 2 * m.first_cta + (t0 > m.first_cta * per ? 1 : 0);
      m.row0 = w.s.row0;
      m.r0 = 128 * w.rt;
      m.n_rows = min(128, w.s.n * p.G - m.r0);
      m.g = w.g;
    }
    p.merge[blockIdx.x] = m;
  }

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
    do {
      const int n_keys = w.s.pre + w.s.n;
      const int *table = p.a.page_tables + (size_t)w.b * p.a.max_pages;
      int my_page = -1;
      for (int kt = w.kt0; ok && kt < w.kt1; ++kt) {
        // physical pages of the next 16 tiles' 64-key halves, one a lane; -1:
        // past the last key, -2: a page outside the pools
        const int j = (kt - w.kt0) & 15;
        if (j == 0) {
          const int key = 128 * kt + 64 * lane;
          my_page = -1;
          if (kt + (lane >> 1) < w.kt1 && key < n_keys) {
            my_page = table[key / p.a.pg];
            if (my_page < 0 || my_page >= p.a.n_pages) {
              if (p.err) atomicExch(p.err + 1, kBadPage);
              my_page = -2;
            }
          }
        }
        const int pgs[2] = {__shfl_sync(0xffffffffu, my_page, 2 * j), __shfl_sync(0xffffffffu, my_page, 2 * j + 1)};
        if (lane == 0) {
          if (issued >= KR) ok = tc::mbar_wait(empty + slot, phase ^ 1, p.err, is_k ? 51 : 50, abort);
          if (*abort) ok = false;
          if (ok) {
            if (is_k) flags[issued & (kTreeFlags - 1)] = (pgs[0] == -2 ? 1 : 0) | (pgs[1] == -2 ? 2 : 0);
            unsigned char *dst = ring + (size_t)slot * S::tile;
            uint64_t *bar = full + slot;
            tc::mbar_expect_tx(bar, (uint32_t)S::tile);
            const int key0 = 128 * kt, at0 = key0 % p.a.pg;
            const bool whole = pgs[0] >= 0 && pgs[1] == pgs[0] && at0 + 128 <= p.a.pg && (is_k || key0 + 128 <= n_keys);
            for (int h = 0; h < (whole ? 1 : 2); ++h) {
              // rows copied from the page; the rest of the half is zero.  K: the
              // page's slots past the last key too (their scores are masked);
              // V: the sequence's own rows only (0 times anything must be 0).
              const int key = key0 + 64 * h;
              const int rows = whole ? 128 : pgs[h] < 0 ? 0 : is_k ? 64 : min(64, n_keys - key);
              const bf16 *src = pool + ((size_t)max(pgs[h], 0) * p.a.Hkv + w.g) * p.a.pg * HD + (size_t)(key % p.a.pg) * 64;
              for (int b = 0; b < HB; ++b) {
                unsigned char *d = dst + (size_t)b * 16384 + h * kAttnSlotHalfBytes;
                if (rows > 0) tc::bulk_load(d, src + (size_t)b * p.a.pg * 64, 128u * rows, bar);
                if (rows < 64) tc::bulk_load(d + 128 * rows, g_zero_half, 128u * (64 - rows), bar);
              }
            }
            ++issued;
            if (++slot == KR) {
              slot = 0;
              phase ^= 1;
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
    } while (ok && w.next(p));
    if (!ok && lane == 0) {  // gave up: wait (bounded) for the copies in flight
      for (int i = issued - 1; i >= 0 && i >= issued - KR; --i) {
        const long long t0 = clock64();
        while (!tc::mbar_try_wait(full + i % KR, (i / KR) & 1) && clock64() - t0 < tc::kWaitCycles) {
        }
      }
    }
  } else if (warp == 1 || warp == kTreePvWarp) {
    if (lane == 0) {
      bool ok = true;
      int i = 0, slot = 0, phase = 0, piece = 0;
      if (warp == 1) {  // ---- S = Q K^T
        const uint32_t idesc = tc::idesc_bf16(128, 128);
        do {
          ok = tc::mbar_wait(q_full, piece & 1, p.err, 52, abort);
          for (int kt = w.kt0; ok && kt < w.kt1; ++kt, ++i) {
            const int buf = i & 1;
            if (i >= 2) ok = tc::mbar_wait(s_empty + buf, ((i >> 1) - 1) & 1, p.err, 53, abort);
            ok = ok && tc::mbar_wait(k_full + slot, phase, p.err, 54, abort);
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
          if (piece) ok = tc::mbar_wait(o_empty, (piece - 1) & 1, p.err, 55, abort);
          for (int kt = w.kt0; ok && kt < w.kt1; ++kt, ++i) {
            const int buf = i & 1;
            ok = tc::mbar_wait(p_full + buf, (i >> 1) & 1, p.err, 56, abort) &&
                 tc::mbar_wait(v_full + slot, phase, p.err, 57, abort);
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
    float *xch = (float *)(base + S::xch);  // [2 halves][128 rows]
    auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;\n" ::"r"(1 + q4) : "memory"); };
    // The piece's query rows into the operand tile (row r: token r / G, head g G + r % G).
    auto stage_q = [&](const Walk &u) {
      const int rows = min(128, u.s.n * p.G - 128 * u.rt);
      for (int idx = tid; idx < rows * (HD / 8); idx += 256) {
        const int r = idx / (HD / 8), c = idx & (HD / 8 - 1);
        const int rg = 128 * u.rt + r, t = rg / p.G, h = u.g * p.G + rg - t * p.G;
        const uint4 v = *(const uint4 *)(p.a.q + (size_t)(u.s.row0 + t) * p.a.q_stride + (size_t)h * HD + 8 * c);
        *(uint4 *)(base + S::q + (size_t)(c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      __syncwarp();
      if (lane == 0) attn_arrive(q_full);
    };
    stage_q(w);
    int i = 0, piece = 0;
    bool more;
    do {
      const int rows = min(128, w.s.n * p.G - 128 * w.rt);
      const bool active = 32 * q4 < rows;  // the same in both warps of the quarter
      const int rg = 128 * w.rt + row, t = row < rows ? rg / p.G : 0, h = w.g * p.G + rg - t * p.G;
      float m = NEG, l = 0.0f;  // l: this half's share of the row sum
      for (int kt = w.kt0; kt < w.kt1; ++kt, ++i) {
        const int buf = i & 1;
        tc::mbar_wait(s_full + buf, (i >> 1) & 1, p.err, 58, abort);
        if (!active) {
          // nothing to compute: the arrivals alone, P's after the buffer's last use
          if (lane == 0) attn_arrive(s_empty + buf);
          if (i >= 2) tc::mbar_wait(p_empty + buf, ((i >> 1) - 1) & 1, p.err, 59, abort);
          __syncwarp();
          if (lane == 0) attn_arrive(p_full + buf);
          continue;
        }
        tc::fence_after();
        const int key_base = 128 * kt + 64 * half;
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
        if (key_base + 64 > w.s.pre || bad) {
          unsigned long long see = (bad >> half) & 1 ? 0ull : row_bits(p, w.s, t, key_base - w.s.pre);
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
          for (int j = 0; j < 32; j += 4) {
            a0 = fmaxf(a0, __uint_as_float(x[c][j]));
            a1 = fmaxf(a1, __uint_as_float(x[c][j + 1]));
            a2 = fmaxf(a2, __uint_as_float(x[c][j + 2]));
            a3 = fmaxf(a3, __uint_as_float(x[c][j + 3]));
          }
        const float hmax = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3));
        xch[half * 128 + row] = hmax;
        pair_sync();
        const float tmax = fmaxf(hmax, xch[(half ^ 1) * 128 + row]) * p.scale_log2;
        pair_sync();  // both read before the next tile's maxima overwrite the slots
        const float m_new = fmaxf(m, tmax);
        const bool grow = m_new > m + kRescaleLog2;  // false while both are -inf; the same in both halves
        // P buffer i & 1 is free once P V of tile i - 2 is done
        if (i >= 2) tc::mbar_wait(p_empty + buf, ((i >> 1) - 1) & 1, p.err, 60, abort);
        const float m_old = m;
        if (grow) m = m_new;
        const float nmu = m == NEG ? 0.0f : -m;
        float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
        const uint32_t prow = t_p + 64 * buf + 32 * half + lane_off;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float p0 = ex2(fmaf(__uint_as_float(x[c][j]), p.scale_log2, nmu));
            const float p1 = ex2(fmaf(__uint_as_float(x[c][j + 1]), p.scale_log2, nmu));
            const uint32_t k2 = pack_bf16(p0, p1);
            pk[j >> 1] = k2;
            const float r = __uint_as_float(k2 << 16) + __uint_as_float(k2 & 0xffff0000u);  // as rounded
            if ((j & 6) == 0) s0 += r;
            else if ((j & 6) == 2) s1 += r;
            else if ((j & 6) == 4) s2 += r;
            else s3 += r;
          }
          tmem_st16(prow + 16 * c, pk);
        }
        // rows whose maximum grew: O (and l) to the new reference, O <- O 2^(m_old - m);
        // each half rescales its half of the O columns
        float f = 1.0f;
        if (__any_sync(0xffffffffu, grow) && kt > w.kt0) {
          // O must hold P V of every earlier tile of the piece: wait for tile i - 1's
          tc::mbar_wait(p_empty + (buf ^ 1), ((i - 1) >> 1) & 1, p.err, 61, abort);
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
        l = l * f + ((s0 + s1) + (s2 + s3));
        asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");  // P (and O) written before the release
        tc::fence_before();
        __syncwarp();
        if (lane == 0) attn_arrive(p_full + buf);
      }
      // every S of this piece is done (its last s_full): the next piece's rows
      Walk nx = w;
      more = nx.next(p);  // the same in all softmax warps (never cut short: they meet at named barriers)
      if (more) stage_q(nx);
      tc::mbar_wait(o_full, piece & 1, p.err, 62, abort);  // inactive warps too: o_empty counts one arrival of each a piece
      if (active) {  // the row sum of both halves
        xch[half * 128 + row] = l;
        pair_sync();
        const float lt = half ? xch[row] + l : l + xch[128 + row];  // keys 0-63 first
        pair_sync();
        tc::fence_after();
        const bool full_unit = w.kt0 == 0 && w.kt1 == w.s.key_tiles;
        const float inv = lt > 0.0f ? 1.0f / lt : 0.0f;
        const int slot = 2 * blockIdx.x + (piece ? 1 : 0);
        bf16 *dst = p.a.out + (size_t)(w.s.row0 + t) * p.a.out_stride + (size_t)h * HD;
        float4 *part = (float4 *)p.part + (size_t)slot * 128 * (HD / 4) + row;
#pragma unroll 1
        for (int c = half * (HD / 64); c < (half + 1) * (HD / 64); ++c) {
          uint32_t v[32];
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
        if (!full_unit && half == 0 && row < rows) p.state[(size_t)slot * 128 + row] = make_float2(m, lt);
        tc::fence_before();
      }
      __syncwarp();
      if (lane == 0) attn_arrive(o_empty);
      w = nx;
      ++piece;
    } while (more);
  }
  __syncwarp();  // lone-thread roles above: reconverge before the block-wide barrier
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512u));
  }
}

// Joins the pieces of the units that span several blocks: weights 2^(m_s - m*),
// pieces in the order of the keys.  Block (c, y): the unit that ends in block
// c's first piece, rows y R .. y R + R - 1, one float4 column a thread.
template <int HD>
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeArgs p) {
  constexpr int R = 1024 / HD;  // rows per block: 256 threads, HD / 4 columns each
  const TreeMerge m = p.merge[blockIdx.x];
  const int i = R * blockIdx.y + (threadIdx.x & (R - 1)), col = threadIdx.x / R;
  if (!m.on || i >= m.n_rows) return;
  const int n = (int)blockIdx.x - m.first_cta + 1;  // pieces
  auto slot = [&](int s) { return s == 0 ? m.first_slot : 2 * (m.first_cta + s); };
  const float NEG = __int_as_float(0xff800000);
  float mx = NEG;
#pragma unroll 8
  for (int s = 0; s < n; ++s) mx = fmaxf(mx, p.state[(size_t)slot(s) * 128 + i].x);
  float L = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int s = 0; s < n; ++s) {
    const float2 ml = p.state[(size_t)slot(s) * 128 + i];
    const float4 o = ((const float4 *)p.part)[((size_t)slot(s) * (HD / 4) + col) * 128 + i];
    const float f = ml.x == NEG ? 0.0f : ex2(ml.x - mx);
    L += f * ml.y;
    acc.x += f * o.x;
    acc.y += f * o.y;
    acc.z += f * o.z;
    acc.w += f * o.w;
  }
  const float inv = L > 0.0f ? 1.0f / L : 0.0f;
  const int rg = m.r0 + i, t = rg / p.G, h = m.g * p.G + rg - t * p.G;
  *(uint2 *)(p.a.out + (size_t)(m.row0 + t) * p.a.out_stride + (size_t)h * HD + 4 * col) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

struct TreeWorkspace {
  size_t part, state, merge, bytes;
};
TreeWorkspace tree_workspace(int hd) {
  TreeWorkspace w;
  w.part = 0;
  w.state = w.part + (size_t)2 * kTreeCtas * 128 * hd * 4;
  w.merge = w.state + (size_t)2 * kTreeCtas * 128 * sizeof(float2);
  w.bytes = w.merge + (size_t)kTreeCtas * sizeof(TreeMerge);
  return w;
}

template <int HD>
cudaError_t launch_tree(const TreeArgs &p, cudaStream_t st) {
  using S = TreeSmem<HD>;
  static_assert(S::bytes <= 232448, "shared memory of the tree attention kernel");
  static unsigned long long attr_set = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((attr_set >> dev) & 1ull)) {
    e = cudaFuncSetAttribute(tree_attn_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::bytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set |= 1ull << dev;
  }
  tree_attn_kernel<HD><<<kTreeCtas, kTreeThreads, S::bytes, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // no unit has more rows than the whole batch
  const int rows = (int)min(128ll, (long long)p.a.n_tok * p.G);
  tree_merge_kernel<HD><<<dim3(kTreeCtas, ceil_div(rows, 1024 / HD)), 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t tree_attention_workspace_bytes(int, int, int, int, int hd) { return tree_workspace(hd).bytes; }

cudaError_t tree_attention(const TreeAttention &a, void *ws, int *err, cudaStream_t st) {
  if (a.n_tok == 0 || a.n_seqs == 0) return cudaSuccess;
  const TreeWorkspace w = tree_workspace(a.hd);
  TreeArgs p;
  p.a = a;
  p.G = a.Hq / a.Hkv;
  p.min_tiles = 1;
  p.scale_log2 = (float)(1.4426950408889634 * (double)a.scale);
  p.part = (float *)((unsigned char *)ws + w.part);
  p.state = (float2 *)((unsigned char *)ws + w.state);
  p.merge = (TreeMerge *)((unsigned char *)ws + w.merge);
  p.err = err;
  return a.hd == 128 ? launch_tree<128>(p, st) : launch_tree<64>(p, st);
}

}  // namespace dg
