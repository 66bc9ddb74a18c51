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
// exchange.  A row's -lse / scale comes in as 16 more columns of its operand (three
// bf16 numbers whose sum is the fp32 one; the keys have ones there): added up by the
// tensor core it costs an eighth of the products, read from shared memory by every
// thread it cost as much of that memory's bandwidth as the products themselves
// (8192 rows: 141 us).  A unit is 1, 2 or 4 tiles of 128 keys of a (sequence, KV head):
// they stay in shared memory while the tiles of up to 128 rows (tokens x heads of the
// group, staged by one TMA copy) that see any of them go by.  A unit has 4 key tiles, which
// share each row tile read from L2 and what every role does per unit (with single tokens that
// took longer than the keys' stream: 48 sequences over up to 16k keys 207 us with 1, 142 with
// 2, 125 with 4, at 6.1 TB/s); where there is little to do, what gives each block one unit.
// All blocks take equal ranges of the batch's (unit, row tile) pairs (ranges.cuh); a unit that
// spans several blocks leaves a partial sum per block in the workspace, and the block whose
// sum arrives last adds them up in order: no block waits, results repeat bit for bit.
//
// Roles of a block (640 threads): warp 0 copies keys out of the pre-swizzled pages,
// warp 1 the row tiles and their log-sum-exps; warps 2 and 3 issue the products of
// every other key tile from one thread each, and give a key tile back with its last ones
// (all at the unit's end: 151 us); warps 4-19 take the exponentials, four warps a key tile,
// four key tiles at a time.
//
// Measured (16 query and 8 KV heads of 128): one token over 8k keys 8.3 us, latency; 8192
// rows of a prompt 110 to 115 us, by machine, 63 to 66% of the measured product rate (of a
// row tile's 9 x 64 cycles on the tensor core a ninth are the log-sum-exps'; its exponentials
// take 512 cycles of all special function units).
#include <atomic>

#include "attn_tc.cuh"
#include "f32x2.cuh"
#include "internal.h"
#include "ranges.cuh"

namespace dg {

namespace {

constexpr int kMassThreads = 640;
constexpr int kMassCtas = 152;       // most blocks: one per SM
constexpr int kMassTiles = 4;        // most key tiles of a unit
constexpr int kMassGaveUp = 64;      // status code of a block that gave up after an earlier kernel

struct MassArgs {
  CUtensorMap q_map, few_map;  // rows [n_tok][Hq][hd], boxes 64 x G x T and 64 x G x few
  KeyMass a;
  int G, T, few, ctas;  // T: tokens of a row tile
  int pg_shift;         // log2 of the page size, -1 where it is no power of two
  uint32_t t_magic;     // 2^32 / T, rounded up (0: divide)
  float scale_log2, inv_scale;
  float *part;                // [2 kMassCtas][kMassTiles * 128]: block c's first piece in 2 c, its last in 2 c + 1
  unsigned long long *count;  // [kMassTiles][kMassCtas]: pieces that have arrived of tile k of the unit that ends in block c
  unsigned long long ticket;
  int *err;
};

template <int HD>
struct MassSmem {
  static constexpr int HB = HD / 64;
  static constexpr int KR = HD == 128 ? 4 : 8, QR = HD == 128 ? 2 : 4;  // ring depths, in tiles
  static constexpr size_t tile = (size_t)HB * 16384;                    // 128 keys or rows
  static constexpr size_t kring = 0;
  static constexpr size_t qring = kring + KR * tile;
  static constexpr size_t ones = qring + QR * tile;  // 16 columns of 128 keys: 1 in the first three
  static constexpr size_t lse = ones + 4096;         // [QR] 16 columns of 128 rows
  static constexpr size_t bars = lse + QR * 4096;
  static constexpr int n_bars = 2 * KR + 2 * QR + 8 + 2;  // full and empty of K, Q, S (one buffer a group); drained
  static constexpr size_t slot = bars + n_bars * 8;
  static constexpr size_t bytes = slot + 8 + 4 * kMassTiles;
};

// n = 0: nothing to do, or rows or slots outside the call's arrays.  Of its units
// those below `sink` and from `low` on hold a key which some token sees, or a new key
// (it is set to 0 otherwise).
struct MassSeq {
  int row0, n, pre, tf, row_tiles, sink, low, units;  // tf: the first token that counts
  bool bad;
  __device__ __forceinline__ int visits() const { return sink + units - low; }
  __device__ __forceinline__ int unit(int i) const { return i < sink ? i : i - sink + low; }  // the i-th visited
};

// Tokens [t0, t1) that count and see a key of [j0, j1) (j1 - 1 a slot of the sequence).
struct Tokens {
  int t0, t1;
};
__device__ __forceinline__ Tokens seen_by(const MassArgs &p, const MassSeq &s, int j0, int j1) {
  Tokens t;
  const int last = j1 - 1 - s.pre;  // (last + window where it is below n)
  t.t0 = max(s.tf, j0 - s.pre);
  t.t1 = j0 < p.a.sinks || last >= s.n - p.a.window ? s.n : last + p.a.window;
  return t;
}

// Units of `keys` keys (a power of two), their items the row tiles that see any.
struct MassList {
  typedef MassSeq Seq;
  static constexpr int kUnitCost = 1;
  const MassArgs &p;
  int keys;
  // t / T: t ceil(2^32 / T) / 2^32 is above t / T by less than t / 2^32, and so exact
  // below 2^25 tokens (T <= 128).  Divisions took most of the start of a batch of prompts.
  __device__ __forceinline__ int row_tile(int t) const { return p.t_magic ? (int)__umulhi((uint32_t)t, p.t_magic) : t / p.T; }
  __device__ __forceinline__ Seq load(int b) const {
    Seq s;
    const int o0 = p.a.offsets[b], o1 = p.a.offsets[b + 1];
    s.row0 = o0;
    s.pre = p.a.prefix_lens[b];
    const long long n = (long long)o1 - o0, end = (long long)s.pre + n;
    const long long room = min((long long)p.a.max_pages * p.a.pg, (long long)0x7fffff00);
    s.bad = n != 0 && (o0 < 0 || n < 0 || o1 > p.a.n_tok || s.pre < 0 || end > room);
    s.n = s.bad ? 0 : (int)n;
    s.tf = p.a.observe ? max(0, s.n - p.a.observe) : 0;
    s.row_tiles = row_tile(s.n - s.tf + p.T - 1);
    s.sink = s.low = s.units = 0;
    if (s.n) {
      const int shift = 31 - __clz(keys);
      s.units = (int)(((unsigned)s.pre + s.n + keys - 1) >> shift);
      s.low = min(max(0, s.pre + s.tf - p.a.window + 1), s.pre) >> shift;
      s.sink = min((int)(((unsigned)p.a.sinks + keys - 1) >> shift), s.low);
    }
    return s;
  }
  __device__ __forceinline__ bool even(const Seq &s) const { return s.row_tiles <= 1; }
  // The row tiles of the i-th unit: [first, first + count), one at least.
  __device__ __forceinline__ int rows(const Seq &s, int i, int &first) const {
    first = 0;
    if (s.row_tiles <= 1) return 1;
    const int j0 = s.unit(i) * keys;
    const Tokens t = seen_by(p, s, j0, j0 + min(keys, s.pre + s.n - j0));  // (slots go up to 2^31: j0 + keys may pass it)
    if (t.t0 >= t.t1) return 1;
    first = row_tile(t.t0 - s.tf);
    return row_tile(t.t1 - s.tf + p.T - 1) - first;
  }
  __device__ __forceinline__ int items(const Seq &s, int i) const {
    int first;
    return rows(s, i, first);
  }
};

// The units' key tiles: as many as give every block one unit where there is that
// little to do, or 4.
__device__ __forceinline__ int unit_tiles(const MassArgs &p, int lane) {
  const MassList list{p, 128};
  unsigned total = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.a.n_seqs; b0 += 32) {
    const MassSeq s = list.load(min(b0 + lane, p.a.n_seqs - 1));
    const long long c = b0 + lane < p.a.n_seqs && s.n ? (long long)s.visits() * s.row_tiles * p.a.Hkv : 0;
    total = min(total + __shfl_sync(0xffffffffu, lane_sums((unsigned)min(c, (long long)kMostCost), lane), 31), kMostCost);
  }
  const unsigned ctas = (unsigned)p.ctas;
  return total <= ctas ? 1 : total <= 2 * ctas ? 2 : 4;
}

// The walk over a block's pieces, with the unit's first key and first row tile.
struct MassWalk : RangeWalk<MassList> {
  int key0, tile0;
  __device__ __forceinline__ void locate(const MassList &list) {
    key0 = s.unit(u) * list.keys;
    list.rows(s, u, tile0);
  }
  __device__ __forceinline__ bool begin(const MassList &list, const BlockRange &range, int lane) {
    const bool some = RangeWalk<MassList>::begin(list, range, list.p.a.n_seqs, list.p.a.Hkv, lane);
    if (some) locate(list);
    return some;
  }
  __device__ __forceinline__ bool next(const MassList &list) {
    const bool more = RangeWalk<MassList>::next(list, list.p.a.n_seqs, list.p.a.Hkv);
    if (more) locate(list);
    return more;
  }
  // Row tile q of the piece: its first token, its columns (rows).
  __device__ __forceinline__ int token(const MassArgs &p, int q) const { return s.tf + (tile0 + q) * p.T; }
  __device__ __forceinline__ int columns(const MassArgs &p, int t0) const { return min(p.T, s.n - t0) * p.G; }
  // The tokens that count and see a key of the unit's tile k (none: t0 >= t1).
  __device__ __forceinline__ Tokens tile_tokens(const MassList &list, int k) const {
    const int left = s.pre + s.n - key0 - 128 * k;  // of the sequence, from the tile on
    Tokens t;
    t.t0 = t.t1 = 0;
    if (128 * k < list.keys && left > 0) t = seen_by(list.p, s, key0 + 128 * k, key0 + 128 * k + min(128, left));
    return t;
  }
};

// The entry of the page table for slot j of sequence b; slot: j's place in the page.
__device__ __forceinline__ int page_entry(const MassArgs &p, int b, int j) {
  return table_entry(p.a.page_tables, (size_t)b * p.a.max_pages + (p.pg_shift >= 0 ? j >> p.pg_shift : j / p.a.pg));
}
__device__ __forceinline__ int page_slot(const MassArgs &p, int j) {
  return p.pg_shift >= 0 ? j & (p.a.pg - 1) : j % p.a.pg;
}

// A bounded wait that costs one test when the phase is over already; the loop is not
// inlined: the roles' code has to stay short.
__device__ __noinline__ bool mass_wait_on(uint64_t *b, uint32_t parity, int *err, int code, volatile int *abort) {
  return tc::mbar_wait(b, parity, err, code, abort);
}
__device__ __forceinline__ bool mass_wait(uint64_t *b, uint32_t parity, int *err, int code, volatile int *abort) {
  return tc::mbar_try_wait(b, parity) || mass_wait_on(b, parity, err, code, abort);
}

// tc::mma_bf16 with the low halves of the operands' descriptors: the high ones are
// those of every K-major tile.
__device__ __forceinline__ void mma_low(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accum) {
  const uint64_t high = tc::sw128_desc(0) & 0xffffffff00000000ull;
  tc::mma_bf16(d_tmem, high | a, high | b, idesc, accum);
}

// Shared-memory descriptor of 16 columns without swizzle: 8 x 8 element blocks of
// 128 bytes, the next 8 columns 128 bytes on, the next 8 rows 256.
__device__ __forceinline__ uint64_t plain_desc(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(128 >> 4) << 16;
  d |= (uint64_t)(256 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}

// The four warps of a group meet.
__device__ __forceinline__ void group_sync(int group) { asm volatile("barrier.sync %0, 128;\n" ::"r"(1 + group) : "memory"); }

template <int HD>
__global__ void __launch_bounds__(kMassThreads, 1) key_mass_kernel(const __grid_constant__ MassArgs p) {
  using S = MassSmem<HD>;
  constexpr int HB = S::HB, KR = S::KR, QR = S::QR;
  extern __shared__ __align__(1024) unsigned char base[];
  uint64_t *k_full = (uint64_t *)(base + S::bars), *k_empty = k_full + KR;
  uint64_t *q_full = k_empty + KR, *q_empty = q_full + QR;
  uint64_t *s_full = q_empty + QR, *s_empty = s_full + 4, *drained = s_empty + 4;
  uint32_t *tmem_slot = (uint32_t *)(base + S::slot);
  volatile int *abort = (volatile int *)(tmem_slot + 1), *last = abort + 1;  // last: [kMassTiles]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (tc::smem_u32(base) & 1023u) {  // the operand tiles' swizzle needs it: the same in every block
    if (threadIdx.x == 0 && p.err) atomicExch(p.err, kShapeErrorBase + 6);
    return;
  }
  if (threadIdx.x == 0) {
    *abort = 0;
    for (int i = 0; i < KR; ++i) {
      tc::mbar_init(k_full + i, 1);
      tc::mbar_init(k_empty + i, 2);  // both issuing warps wait for all key tiles: none is replaced before both have
    }
    for (int i = 0; i < QR; ++i) {
      tc::mbar_init(q_full + i, 2);  // the copies, and the log-sum-exps
      tc::mbar_init(q_empty + i, 2);  // the products of both warps
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(s_full + i, 1);
      tc::mbar_init(s_empty + i, 4);  // one arrival per warp of the group
    }
    tc::mbar_init(drained, 1);
    tc::mbar_init(drained + 1, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  }
  // The operands' further columns: 16-byte chunk c of row r at chunk position
  // 16 (r / 8) + 8 c + r % 8.
  for (int i = threadIdx.x; i < (1 + QR) * 256; i += kMassThreads)
    *(uint4 *)(base + S::ones + 16 * i) = i < 256 && !(i & 8) ? make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  const int tiles = unit_tiles(p, lane);  // the same in every warp, as what follows
  const MassList list{p, 128 * tiles};
  const BlockRange range = block_range(list, p.a.n_seqs, p.a.Hkv, p.ctas, p.err, lane);
  MassWalk w;
  if (range.count <= 0 || !w.begin(list, range, lane)) return;
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(tc::smem_u32(tmem_slot)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  unsigned long long status = 0;
  if (warp >= 4 && !(warp & 3))
    if (p.err) asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];\n" : "=l"(status) : "l"(p.err - 1) : "memory");
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (status >> 32) *abort = 1;  // an earlier kernel gave up
  const uint32_t tmem = *tmem_slot;  // S^T of group g: columns 128 g

  // Key tiles are numbered through the block's pieces: tile o = tiles x piece + k is
  // taken by group o & 3, its products issued by warp 2 + (o & 1).  Steps (row tile,
  // key tile) in which no row sees a key are left out, everywhere alike.  A row tile
  // that the next piece begins with again stays in its slot.
  if (warp == 0) {
    // ---- keys: lane (tile, half, hd block) copies 64 keys of 64 elements -------------
    int slot = 0, phase = 0, issued = 0;
    bool ok = true, more = true;
    const int k_lane = lane / (2 * HB), half = lane / HB & 1, blk = lane % HB;
    // the half's entry of the page table; kNotRead: not seen by any row (its page is not touched)
    auto entry_of = [&](const MassWalk &x) {
      const int left = x.s.pre + x.s.n - x.key0 - 128 * k_lane - 64 * half;  // of the sequence, from the half on
      if (k_lane >= tiles || left <= 0) return kNotRead;
      const int j0 = x.key0 + 128 * k_lane + 64 * half;
      const Tokens t = seen_by(p, x.s, j0, j0 + min(64, left));
      return t.t0 < t.t1 ? page_entry(p, x.b, j0) : kNotRead;
    };
    int page = entry_of(w);
    while (ok && more) {
      const void *src = g_zero_half;
      if (page >= 0 && page < p.a.n_pages)
        src = p.a.k_pool + ((size_t)page * p.a.Hkv + w.g) * p.a.pg * HD + (size_t)blk * p.a.pg * 64 +
              (size_t)page_slot(p, w.key0 + 128 * k_lane + 64 * half) * 64;
      const Tokens t = w.tile_tokens(list, lane);
      unsigned used = __ballot_sync(0xffffffffu, t.t0 < t.t1);
      more = w.next(list);
      if (more) page = entry_of(w);
      for (; used; used &= used - 1) {
        if (lane == 0) {
          if (issued >= KR) ok = mass_wait(k_empty + slot, phase ^ 1, p.err, 65, abort);
          if (*abort) ok = false;
          if (ok) tc::mbar_expect_tx(k_full + slot, (uint32_t)S::tile);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (k_lane == __ffs(used) - 1)
          tc::bulk_load(base + S::kring + (size_t)slot * S::tile + (size_t)blk * 16384 + half * kAttnSlotHalfBytes, src, kAttnSlotHalfBytes,
                        k_full + slot);
        __syncwarp();
        ++issued;
        if (++slot == KR) {
          slot = 0;
          phase ^= 1;
        }
      }
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
    int slot = 0, phase = 0, issued = 0, q = w.i0, t0 = w.token(p, q), cols = w.columns(p, t0);
    bool ok = true, more = true;
    // row c of the tile: token t0 + c / G, head g G + c % G
    int off[4];
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = lane + 32 * k, t = c / p.G;
      off[k] = t * p.a.Hq + c - t * p.G;
    }
    auto load = [&]() {
      const float *src = p.a.lse + (size_t)(w.s.row0 + t0) * p.a.Hq + w.g * p.G;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = lane + 32 * k < cols ? src[off[k]] : 0.0f;
    };
    load();
    while (more) {
      if (lane == 0) {
        if (issued >= QR) ok = mass_wait(q_empty + slot, phase ^ 1, p.err, 66, abort);
        if (*abort) ok = false;
        if (ok) {
          const bool few = cols <= p.few * p.G;
          const CUtensorMap *map = few ? &p.few_map : &p.q_map;
          tc::mbar_expect_tx(q_full + slot, HB * 128u * (few ? p.few : p.T) * p.G);
#pragma unroll
          for (int blk = 0; blk < HB; ++blk)
            tc::tma_load_3d(base + S::qring + (size_t)slot * S::tile + (size_t)blk * 16384, map, 64 * blk, w.g * p.G, w.s.row0 + t0, q_full + slot);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = lane + 32 * k;
        float x = v[k] * -p.inv_scale;
        if (x == __int_as_float(0x7f800000)) x = -x;  // rows without a key (lse -inf) weigh nothing
        const float a = __bfloat162float(__float2bfloat16_rn(x)), rest = isfinite(a) ? x - a : 0.0f;
        const float b = __bfloat162float(__float2bfloat16_rn(rest));
        *(uint2 *)(base + S::lse + 4096 * slot + 256 * (c >> 3) + 16 * (c & 7)) = make_uint2(pack_bf16(a, b), pack_bf16(rest - b, 0.0f));
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      __syncwarp();
      if (lane == 0) attn_arrive(q_full + slot);
      ++issued;
      if (++slot == QR) {
        slot = 0;
        phase ^= 1;
      }
      // the next row tile that is another one
      const int b = w.b, g = w.g, tile = w.tile0 + q;
      do {
        if (++q >= w.i1) {
          more = w.next(list);
          q = w.i0;
        }
      } while (more && w.b == b && w.g == g && w.tile0 + q == tile);
      if (more) {
        t0 = w.token(p, q);
        cols = w.columns(p, t0);
        load();
      }
    }
    if (!ok && lane == 0) {
      for (int i = issued - 1; i >= 0 && i >= issued - QR; --i) {
        const long long t0 = clock64();
        while (!tc::mbar_try_wait(q_full + i % QR, (i / QR) & 1) && clock64() - t0 < tc::kWaitCycles) {
        }
      }
    }
  } else if (warp < 4) {
    // ---- S^T = K Q^T -----------------------------------------------------------------
    bool ok = true, more = true, fresh = true;
    const int half = warp - 2;
    int ks = 0, kphase = 0, qs = 0, qphase = 0, order = 0, step0 = 0, step1 = 0;  // steps of groups half, half + 2
    const uint32_t kdesc = (uint32_t)tc::sw128_desc(tc::smem_u32(base + S::kring)), qdesc = (uint32_t)tc::sw128_desc(tc::smem_u32(base + S::qring));
    while (ok && more) {
      const Tokens mine = w.tile_tokens(list, lane);  // of tile `lane`
      const unsigned used = __ballot_sync(0xffffffffu, mine.t0 < mine.t1);
      const int q0 = w.i0, q1 = w.i1, n = w.s.n, b = w.b, h = w.g, last_tile = w.tile0 + q1 - 1;
      int t0 = w.token(p, q0);
      more = w.next(list);
      const bool stays = more && w.b == b && w.g == h && w.tile0 + w.i0 == last_tile;  // the next piece begins with the row tile
      const int n_used = __popc(used);
      int ring = 0;  // key tiles of the unit that have arrived, from slot ks on
      auto arrived = [&]() {
        const int slot = ks + ring;
        ++ring;
        return mass_wait(k_full + (slot < KR ? slot : slot - KR), slot < KR ? kphase : kphase ^ 1, p.err, 67, abort);
      };
      const unsigned turn = 0x55555555u << ((order + half) & 1);  // this warp's tiles
#pragma unroll 1
      for (int q = q0; ok && q < q1; ++q, t0 += p.T) {
        const int cols = min(p.T, n - t0) * p.G;
        const unsigned live = __ballot_sync(0xffffffffu, max(mine.t0, t0) < min(mine.t1, t0 + p.T)) & turn;
        const bool end = q + 1 == q1;  // the piece's last row tile: the key tiles go back one by one
        // (all threads agree on `ok`: one is elected below)
        if (fresh) ok = __all_sync(0xffffffffu, mass_wait(q_full + qs, qphase, p.err, 69, abort));
        const uint32_t idesc = tc::idesc_bf16(128, (cols + 15) & ~15);
        for (unsigned left = end ? used : live; ok && left; left &= left - 1) {
          const int k = __ffs(left) - 1, at = __popc(used & ((1u << k) - 1));
          while (ok && ring <= at) ok = arrived();
          int slot = ks + at;
          if (slot >= KR) slot -= KR;
          if (live >> k & 1) {
            const int g = (order + k) & 3, step = g >= 2 ? step1++ : step0++;
            if (ok && step) ok = mass_wait(s_empty + g, (step - 1) & 1, p.err, 68, abort);
            __syncwarp();
            if (tc::elect_one() && ok) {
              tc::fence_after();
              const uint32_t a = kdesc + slot * (uint32_t)(S::tile >> 4), b = qdesc + qs * (uint32_t)(S::tile >> 4);
#pragma unroll
              for (int kk = 0; kk < HD / 16; ++kk)
                mma_low(tmem + 128 * g, a + (kk >> 2) * 1024 + 2 * (kk & 3), b + (kk >> 2) * 1024 + 2 * (kk & 3), idesc, kk ? 1u : 0u);
              tc::mma_bf16(tmem + 128 * g, plain_desc(tc::smem_u32(base + S::ones)), plain_desc(tc::smem_u32(base + S::lse + 4096 * qs)), idesc, 1u);
              tc::mma_commit(s_full + g);
            }
          }
          __syncwarp();
          if (end && tc::elect_one() && ok) {
            if (((order + k) & 1) == half) tc::mma_commit(k_empty + slot);
            else attn_arrive(k_empty + slot);
          }
          ok = __all_sync(0xffffffffu, ok);
        }
        fresh = q + 1 < q1 || !stays;
        if (ok && fresh) {
          if (tc::elect_one()) tc::mma_commit(q_empty + qs);
          if (++qs == QR) {
            qs = 0;
            qphase ^= 1;
          }
        }
      }
      ks += n_used;
      if (ks >= KR) {
        ks -= KR;
        kphase ^= 1;
      }
      order += tiles;
    }
    if (tc::elect_one() && !ok) {  // gave up: wait (bounded) for the products in flight
      tc::mma_commit(drained + half);
      const long long t0 = clock64();
      while (!tc::mbar_try_wait(drained + half, 0) && clock64() - t0 < tc::kWaitCycles) {
      }
    }
  } else if (warp >= 4) {
    // ---- weights: thread = key of tile k of the unit ------------------------------------
    const int g = (warp - 4) >> 2, row = threadIdx.x & 127;
    const uint32_t col = tmem + 128 * g + ((uint32_t)(32 * (warp & 3)) << 16);
    const f32x2 scale2 = pair(p.scale_log2, p.scale_log2);
    int order = 0, piece = 0, step = 0;
    bool ok = true, more = true;
    // The key's entry of the page table: kNotRead where no weight is written (another
    // group's, behind the sequence, neither new nor seen by any row).
    auto entry = [&]() {
      const int k = (g - order) & 3, j = w.key0 + 128 * k + row;
      if (k >= tiles || j >= w.s.pre + w.s.n) return kNotRead;
      const Tokens t = seen_by(p, w.s, j, j + 1);
      return j >= w.s.pre || t.t0 < t.t1 ? page_entry(p, w.b, j) : kNotRead;
    };
    int page = entry();
    while (more) {
      const int k = (g - order) & 3;
      const bool mine = k < tiles;
      // where the weight lies (< 0: none is written), and what it was
      const int j = w.key0 + 128 * k + row;
      long long at = -1;
      float old = 0.0f, sum = 0.0f;
      if (page >= 0 && page < p.a.n_pages) {
        at = ((long long)page * p.a.Hkv + w.g) * p.a.pg + page_slot(p, j);
        if (j < w.s.pre) old = p.a.mass[at];
      } else if (page != kNotRead && p.err) {
        atomicExch(p.err + 1, kBadPage);
      }
      // the piece, and the next one: its entry of the page table is on its way meanwhile
      const int pre = w.s.pre, n = w.s.n, q0 = w.i0, q1 = w.i1;
      const bool whole = q0 == 0 && q1 == w.items;
      UnitBlocks blocks{};
      if (!whole) blocks = unit_blocks(w, range.per);
      int t0 = w.token(p, q0);
      const Tokens seen = w.tile_tokens(list, k);
      more = w.next(list);
      order += tiles;
      if (more) page = entry();
#pragma unroll 1
      for (int q = q0; q < q1; ++q, t0 += p.T) {
        if (max(seen.t0, t0) < min(seen.t1, t0 + p.T)) {
          const int span = min(p.T, n - t0), cols = span * p.G;
          // the key's columns [c0, c1): tokens from its own on, up to the window's end
          const int away = j - pre - t0;
          const int c0 = min(max(away, 0), 128) * p.G;
          const int c1 = j < p.a.sinks || away >= span - p.a.window ? cols : max(0, away + p.a.window) * p.G;
          if (!mass_wait(s_full + g, step & 1, p.err, 70, abort)) ok = false;
          ++step;
          __syncwarp();
          tc::fence_after();
          f32x2 s0 = pair(0.0f, 0.0f), s1 = s0;
          // 2^(scale (x - lse / scale)) of four columns, added up
          auto add4 = [&](const uint32_t *y, int cc, bool all) {
            const float2 d = split(mul2(pair(__uint_as_float(y[0]), __uint_as_float(y[1])), scale2));
            const float2 e = split(mul2(pair(__uint_as_float(y[2]), __uint_as_float(y[3])), scale2));
            float a0 = ex2(d.x), a1 = ex2(d.y), a2 = ex2(e.x), a3 = ex2(e.y);
            if (!all) {
              a0 = cc >= c0 && cc < c1 ? a0 : 0.0f;
              a1 = cc + 1 >= c0 && cc + 1 < c1 ? a1 : 0.0f;
              a2 = cc + 2 >= c0 && cc + 2 < c1 ? a2 : 0.0f;
              a3 = cc + 3 >= c0 && cc + 3 < c1 ? a3 : 0.0f;
            }
            s0 = add2(s0, pair(a0, a1));
            s1 = add2(s1, pair(a2, a3));
          };
          auto release = [&]() {  // the buffer is free for the group's next step
            tc::fence_before();
            __syncwarp();
            if (lane == 0) attn_arrive(s_empty + g);
          };
          // (few instructions, run over and over: a loop that is unrolled for all
          // columns and both forms waits for its instructions)
          if (__all_sync(0xffffffffu, c0 == 0 && c1 == 128)) {
            uint32_t x[2][16];
            tmem_ld16(col, x[0]);
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
              tmem_ld_wait16(x[0]);
              tmem_ld16(col + c + 16, x[1]);
#pragma unroll
              for (int i = 0; i < 4; ++i) add4(x[0] + 4 * i, 0, true);
              tmem_ld_wait16(x[1]);
              if (c < 96) tmem_ld16(col + c + 32, x[0]);
              else release();
#pragma unroll
              for (int i = 0; i < 4; ++i) add4(x[1] + 4 * i, 0, true);
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < cols; c += 16) {
              uint32_t x[16];
              tmem_ld16(col + c, x);
              tmem_ld_wait16(x);
              if (c + 16 >= cols) release();
#pragma unroll
              for (int i = 0; i < 4; ++i) add4(x + 4 * i, c + 4 * i, false);
            }
          }
          const float2 r = split(add2(s0, s1));
          sum += r.x + r.y;
        }
      }
      if (whole) {
        if (at >= 0 && ok) p.a.mass[at] = old + sum;
      } else if (mine) {
        const int to = 2 * blockIdx.x + (piece ? 1 : 0);
        p.part[((size_t)to * kMassTiles + k) * 128 + row] = sum;
        __threadfence();
        group_sync(g);
        if (row == 0) last[g] = !*abort && arrive_last(p.count + (size_t)k * kMassCtas + blocks.last, p.ticket + (uint32_t)status,
                                                           blocks.last - blocks.first + 1);
        group_sync(g);
        if (last[g] && at >= 0) {
          __threadfence();
          const float *src = p.part + (size_t)k * 128 + row;
          float total = 0.0f;
          for (int c = blocks.first; c <= blocks.last; ++c) total += __ldcg(src + (size_t)blocks.slot(c) * kMassTiles * 128);
          p.a.mass[at] = old + total;
        }
      }
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
  static constexpr size_t count = part + (size_t)2 * kMassCtas * kMassTiles * 128 * 4;
  static constexpr size_t bytes = count + (size_t)kMassTiles * kMassCtas * 8;
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
  p.inv_scale = (float)(1.0 / (double)a.scale);
  p.part = (float *)((unsigned char *)ws + MassWorkspace::part);
  p.count = (unsigned long long *)((unsigned char *)ws + MassWorkspace::count);
  p.ticket = new_ticket();
  p.err = err;
  p.few = max(1, 16 / p.G);
  p.pg_shift = (a.pg & (a.pg - 1)) ? -1 : __builtin_ctz(a.pg);
  p.t_magic = p.T > 1 && a.n_tok < (1 << 25) - 256 ? (uint32_t)(((1ull << 32) + p.T - 1) / p.T) : 0;
  cudaError_t e = rows_map(&p.q_map, a.q, a.q_stride, a.n_tok, a.Hq, a.hd, p.G, p.T);
  if (e == cudaSuccess) e = rows_map(&p.few_map, a.q, a.q_stride, a.n_tok, a.Hq, a.hd, p.G, p.few);
  if (e != cudaSuccess) return e;
  return a.hd == 128 ? launch_mass<128>(p, st) : launch_mass<64>(p, st);
}

}  // namespace dg
