// Per-head RMS norm with the position rotation, and the append of rotated
// keys (and values) to the paged KV cache.
//
// Per head row x of hd values (report §1, context encoding; the rotation is
// the rotate-half form of the decoder's QKV epilogue):
//   y = x * rsqrt(mean(x^2) + eps) * gain            (no gain: y = x)
//   (y_j, y_{j+rd/2}) <- (y_j c - y_{j+rd/2} s, y_{j+rd/2} c + y_j s),  j < rd/2,
// c, s = cos, sin of position * base^(-2j/rd); values past rd keep y.
// fp32 throughout, one rounding to bf16 at the store.
//
// Angles: the host rounds each frequency in turns, base^(-2j/rd) / (2 pi), to
// a 64-bit fraction; position * fraction modulo 2^64 is the angle in turns
// without any loss at far positions (an fp32 product would be off by 0.06 rad
// at position 10^6).  Its top 32 bits split exactly into a quadrant and a
// remainder in [-pi/4, pi/4], whose sine and cosine are Taylor sums.
//
// Bound by the bytes of the rows: 16384 tokens of 16 + 8 heads of 128 (201 MB in
// and out) take 34.7 us, 5.8 TB/s; a plain addition that reads and writes as
// much takes 33.2.
//
// Layout: a head is handled by hd / 16 lanes.  Lane i < rd / 16 holds the
// 8-element chunks i and i + rd / 16, whose elements rotate with one another, the
// lanes behind it the chunks 2 i and 2 i + 1: the rotation needs no exchange
// between lanes, and loads and stores are 16 bytes wide.  A warp takes a token
// at a time, and of its heads as many as the lanes hold, twice over: the token's
// sines and cosines are computed once, multiplied with the gains, into the warp's
// own shared memory, from where every head takes them.  The rows of the next
// groups of heads, the next token's too, are on their way to shared memory
// meanwhile (each lane copies and reads its own chunks), so no warp waits for
// another.  A block of some tokens that loaded, met at a barrier and stored took
// 40.8 us, although as many bytes were on their way: its phases did not overlap.
#include <math.h>

#include "f32x2.cuh"
#include "internal.h"

namespace dg {

namespace {

// Warps of a block and resident blocks, and the groups of heads a warp has on
// their way: 16384 tokens of 16 + 8 heads of 128 take 34.7 us and 17,667 tokens
// appended to 8 heads 26.4 us with (2 blocks, 3 stages), 35.1 and 26.9 with
// (2, 4), 34.6 and 28.5 with (3, 3), 41.1 and 33.8 with (3, 6).
constexpr int kRopeWarps = 8, kRopeBlocks = 2, kStages = 3;
constexpr int kMaxHalfRope = 128;

// Frequencies of the rotation in turns, as 64-bit fractions.
struct RopeFreq {
  unsigned long long turn[kMaxHalfRope];
};

// A lane's two chunks of a head as loaded, and its way through shared memory:
// piece n of lane l at stage[32 n + l], which the lane itself copies and reads.
template <typename T>
struct Chunks {
  static constexpr int kPieces = sizeof(T);  // of 16 bytes
  uint4 a[kPieces / 2], b[kPieces / 2];
  static __device__ __forceinline__ void request(uint4 *stage, const T *head, int c0, int c1) {
#pragma unroll
    for (int i = 0; i < kPieces / 2; ++i) {
      copy16(stage + 32 * i, (const uint4 *)(head + 8 * c0) + i);
      copy16(stage + 32 * (kPieces / 2 + i), (const uint4 *)(head + 8 * c1) + i);
    }
  }
  __device__ __forceinline__ void read(const uint4 *stage) {
#pragma unroll
    for (int i = 0; i < kPieces / 2; ++i) {
      a[i] = stage[32 * i];
      b[i] = stage[32 * (kPieces / 2 + i)];
    }
  }
  static __device__ __forceinline__ void copy16(uint4 *to, const uint4 *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
  }
};

// Eight values of a chunk as four pairs.
__device__ __forceinline__ void unpack8(const uint4 (&w)[1], f32x2 *x) {
  const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pair(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}
__device__ __forceinline__ void unpack8(const uint4 (&w)[2], f32x2 *x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[2 * i] = pair(__uint_as_float(w[i].x), __uint_as_float(w[i].y));
    x[2 * i + 1] = pair(__uint_as_float(w[i].z), __uint_as_float(w[i].w));
  }
}
__device__ __forceinline__ uint4 pack8(const f32x2 *x) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __float22bfloat162_rn(split(x[i]));
    u[i] = *(const uint32_t *)&v;
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Chunk indices of lane i of a head.
__device__ __forceinline__ void lane_chunks(int i, int rd16, int *c0, int *c1) {
  *c0 = i < rd16 ? i : 2 * i;
  *c1 = i < rd16 ? i + rd16 : 2 * i + 1;
}

// 1 / RMS of the head held by a group of HD / 16 lanes.
template <int HD>
__device__ __forceinline__ float head_scale(const f32x2 *a, const f32x2 *b, float eps) {
  f32x2 s = mul2(a[0], a[0]), t = mul2(b[0], b[0]);
#pragma unroll
  for (int e = 1; e < 4; ++e) {
    s = fma2(a[e], a[e], s);
    t = fma2(b[e], b[e], t);
  }
  const float2 u = split(s), v = split(t);
  float r = (u.x + u.y) + (v.x + v.y);
#pragma unroll
  for (int o = HD / 32; o; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  return rsqrtf(r * (1.0f / HD) + eps);
}

// Sine and cosine of the angle pos * turn (pos as a signed number).  |r| <=
// pi / 4: sin r to r^9 / 9!, cos r to r^10 / 10!, each within 2^-25 before
// rounding.
__device__ __forceinline__ float2 turn_angle(unsigned long long turn, int pos) {
  const uint32_t t = (uint32_t)(((unsigned long long)(long long)pos * turn) >> 32);
  const uint32_t q = (t + 0x20000000u) >> 30;  // nearest quarter turn
  const float r = (float)(int)(t - (q << 30)) * (float)(6.283185307179586 / 4294967296.0);
  const float z = r * r;
  float s = 1.0f / 362880.0f;
  s = fmaf(s, z, -1.0f / 5040.0f);
  s = fmaf(s, z, 1.0f / 120.0f);
  s = fmaf(s, z, -1.0f / 6.0f);
  s = fmaf(s * z, r, r);
  float c = -1.0f / 3628800.0f;
  c = fmaf(c, z, 1.0f / 40320.0f);
  c = fmaf(c, z, -1.0f / 720.0f);
  c = fmaf(c, z, 1.0f / 24.0f);
  c = fmaf(c, z, -0.5f);
  c = fmaf(c, z, 1.0f);
  const float u = (q & 1) ? c : s, v = (q & 1) ? s : c;  // sine and cosine up to signs
  return make_float2((q & 2) ? -u : u, ((q + 1) & 2) ? -v : v);
}

// A token's factors for one side: a' = a ga c - b gb s, b' = b gb c + a ga s
// (without rotation a ga, b gb), as float4 [ga c, -gb s, gb c, ga s][2][lanes]:
// lane i's eight values of each, four to a float4, lanes adjacent: 2 HD floats.

// Factors of the pairs j and j + 1 (j even; elements j, j + 1 of the lanes'
// first chunks and their partners).
template <int HD>
__device__ __forceinline__ void put_factors(float *to, int j, int rd16, const float *gain, float2 sc0, float2 sc1) {
  constexpr int L = HD / 16;
  const int i = j >> 3, e = j & 7;
  int c0, c1;
  lane_chunks(i, rd16, &c0, &c1);
  float2 ga = make_float2(1.0f, 1.0f), gb = ga;
  if (gain) {
    ga = *(const float2 *)(gain + 8 * c0 + e);
    gb = *(const float2 *)(gain + 8 * c1 + e);
  }
  float2 *at = (float2 *)(to + ((e >> 2) * L + i) * 4 + (e & 3));
  at[0 * 4 * L] = make_float2(ga.x * sc0.y, ga.y * sc1.y);
  at[1 * 4 * L] = make_float2(-gb.x * sc0.x, -gb.y * sc1.x);
  at[2 * 4 * L] = make_float2(gb.x * sc0.y, gb.y * sc1.y);
  at[3 * 4 * L] = make_float2(ga.x * sc0.x, ga.y * sc1.x);
}

// Norm (any: some head of the launch has one; normed: this side's) and rotation
// of a lane's chunks of U heads with their token's factors (a head's first
// chunk: x[u][0..3], its second: x[u][4..7]); live: the heads to take, the same
// in the whole warp.
template <int HD, int U>
__device__ __forceinline__ void turn_heads(f32x2 (&x)[U][8], int live, bool any, bool normed, float eps, bool turns,
                                           const float *factors, int i) {
  constexpr int L = HD / 16;
  if (any) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u >= live) break;
      const float s = head_scale<HD>(x[u], x[u] + 4, eps), r = normed ? s : 1.0f;
      const f32x2 rr = pair(r, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[u][e] = mul2(x[u][e], rr);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const ulonglong2 *at = (const ulonglong2 *)factors + (e >> 1) * L + i;
    const ulonglong2 ac = at[0], bc = at[4 * L];
    ulonglong2 bs, as;
    if (turns) {
      bs = at[2 * L];
      as = at[6 * L];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u >= live) break;
      f32x2 *a = x[u] + e, *b = x[u] + 4 + e;
      const f32x2 x0 = a[0], x1 = a[1], y0 = b[0], y1 = b[1];
      a[0] = mul2(x0, ac.x);
      a[1] = mul2(x1, ac.y);
      b[0] = mul2(y0, bc.x);
      b[1] = mul2(y1, bc.y);
      if (turns) {
        a[0] = fma2(y0, bs.x, a[0]);
        a[1] = fma2(y1, bs.y, a[1]);
        b[0] = fma2(x0, as.x, b[0]);
        b[1] = fma2(x1, as.y, b[1]);
      }
    }
  }
}

// How a launch is laid out: a token's heads are groups of U 32 / (hd / 16)
// heads, those of the first side and then those of the second; a warp's item is
// a token, or one of its `parts` of `each` groups.
struct RopePlan {
  int parts, each, groups, first;  // groups: of both sides; first: of the first side
};

struct QkArgs {
  const void *q, *k;
  long long q_stride, k_stride;
  const int *positions;
  int n_tok, Hq, Hkv, rd16;
  const float *q_gain, *k_gain;
  float eps;
  bf16 *q_out, *k_out;
  long long q_out_stride, k_out_stride;
  RopePlan plan;
};

// Where a warp is: group g of [g0, g1) of token t; end: it has no more.
struct At {
  uint32_t item, t;
  int g, g0, g1;
  __device__ __forceinline__ At(const RopePlan &p, uint32_t it, int n_tok) { set(p, it, n_tok); }
  __device__ __forceinline__ void set(const RopePlan &p, uint32_t it, int n_tok) {
    item = t = it;
    g0 = 0;
    if (p.parts > 1) {
      t = it / p.parts;
      g0 = (int)(it - t * p.parts) * p.each;
    }
    g = g0;
    g1 = t < (uint32_t)n_tok ? min(g0 + p.each, p.groups) : 0;
  }
  __device__ __forceinline__ bool end() const { return g >= g1; }
};

// Shared memory of a warp in 16-byte pieces: the rows of kStages groups on their
// way, then the token's factors.
template <typename T, int HD, int U, int SIDES>
struct RopeSmem {
  static constexpr int stage = 32 * U * Chunks<T>::kPieces;
  static constexpr int warp = kStages * stage + SIDES * (2 * HD * 4 / 16);
};

template <typename T, int HD>
__global__ void __launch_bounds__(32 * kRopeWarps, kRopeBlocks) qk_norm_rope_kernel(const __grid_constant__ QkArgs p,
                                                                            const __grid_constant__ RopeFreq f) {
  constexpr int L = HD / 16, F = 2 * HD, U = sizeof(T) == 2 ? 2 : 1, step = 32 / L;
  using S = RopeSmem<T, HD, U, 2>;
  extern __shared__ uint4 s_rope[];
  __shared__ __align__(16) unsigned long long s_turn[kMaxHalfRope];
  const int lane = threadIdx.x & 31, i = lane & (L - 1), n_warps = blockDim.x >> 5;
  uint4 *stages = s_rope + (threadIdx.x >> 5) * S::warp + lane;
  float *factors = (float *)(s_rope + (threadIdx.x >> 5) * S::warp + kStages * S::stage);  // [q, k][F]
  int c0, c1;
  lane_chunks(i, p.rd16, &c0, &c1);
  const bool turns = i < p.rd16, any = p.q_gain || p.k_gain;
  const uint32_t stride = gridDim.x * n_warps;
  At at(p.plan, blockIdx.x * n_warps + (threadIdx.x >> 5), p.n_tok), ahead = at;
  // a lane's heads of a group: h, h + step, ..
  auto head_of = [&](const At &at) { return U * step * (at.g < p.plan.first ? at.g : at.g - p.plan.first) + lane / L; };
  // requests the rows of the group `ahead`, and goes on to the next
  auto request = [&](int stage) {
    if (!ahead.end()) {
      const bool is_q = ahead.g < p.plan.first;
      const int h = head_of(ahead), n = (is_q ? p.Hq : p.Hkv) - h;
      const T *src = (is_q ? (const T *)p.q + ahead.t * p.q_stride : (const T *)p.k + ahead.t * p.k_stride) +
                     (long long)h * HD;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u * step < n) Chunks<T>::request(stages + stage * S::stage + 32 * u * Chunks<T>::kPieces, src + u * step * HD, c0, c1);
      if (++ahead.g == ahead.g1) ahead.set(p.plan, ahead.item + stride, p.n_tok);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) request(k);
  int stage = 0, pos = p.rd16 && !at.end() ? p.positions[at.t] : 0;
  for (int j = threadIdx.x; j < 8 * p.rd16; j += blockDim.x) s_turn[j] = f.turn[j];
  __syncthreads();
  while (!at.end()) {
    // the token's factors, while its rows are in flight
#pragma unroll
    for (int j = 2 * lane; j < HD / 2; j += 64) {
      float2 sc0 = make_float2(0.0f, 1.0f), sc1 = sc0;
      if (j < 8 * p.rd16) {
        const ulonglong2 turn = *(const ulonglong2 *)(s_turn + j);
        sc0 = turn_angle(turn.x, pos);
        sc1 = turn_angle(turn.y, pos);
      }
      if (at.g0 < p.plan.first) put_factors<HD>(factors, j, p.rd16, p.q_gain, sc0, sc1);
      if (at.g1 > p.plan.first) put_factors<HD>(factors + F, j, p.rd16, p.k_gain, sc0, sc1);
    }
    __syncwarp();
    At next = at;
    next.set(p.plan, at.item + stride, p.n_tok);
    if (p.rd16 && !next.end()) pos = p.positions[next.t];
    for (; !at.end(); ++at.g) {
      const bool is_q = at.g < p.plan.first;
      const int h = head_of(at), n = (is_q ? p.Hq : p.Hkv) - h;
      const int live = n + lane / L > step ? U : 1;  // whether any lane has a second head
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 2) : "memory");
      f32x2 x[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        Chunks<T> raw;
        raw.read(stages + stage * S::stage + 32 * u * Chunks<T>::kPieces);
        unpack8(raw.a, x[u]);
        unpack8(raw.b, x[u] + 4);
      }
      request(stage ? stage - 1 : kStages - 1);  // the stage that was read last
      stage = stage == kStages - 1 ? 0 : stage + 1;
      turn_heads<HD, U>(x, live, any, is_q ? p.q_gain != nullptr : p.k_gain != nullptr, p.eps, turns, factors + (is_q ? 0 : F), i);
      bf16 *dst = (is_q ? p.q_out + at.t * p.q_out_stride : p.k_out + at.t * p.k_out_stride) + (long long)h * HD;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u * step < n) {
          *(uint4 *)(dst + u * step * HD + 8 * c0) = pack8(x[u]);
          *(uint4 *)(dst + u * step * HD + 8 * c1) = pack8(x[u] + 4);
        }
      }
    }
    __syncwarp();  // the factors have been read
    at = next;
  }
}

struct AppendArgs {
  const bf16 *k, *v;
  long long k_stride, v_stride;
  const int *positions, *prefix, *offsets, *tables;
  int max_pages, n_seqs, n_tok, Hkv, rd16;
  const float *k_gain;
  float eps;
  bf16 *k_pool, *v_pool;
  int n_pages, pg;
  int *err;
  RopePlan plan;
};

// Sequence of packed row t (the same in the whole warp): the last b with
// offsets[b] <= t; n_seqs when the row lies behind the last sequence, -1 before
// the first.  The lanes look at 32 evenly spread offsets at a time.
__device__ __forceinline__ int row_sequence(const int *offsets, int n_seqs, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = n_seqs + 1;  // the count of offsets <= t is in [lo, lo + n]
  while (n > 0) {
    const int gap = (n + 31) / 32, at = lo + min(n, (lane + 1) * gap) - 1;
    const int hits = __popc(__ballot_sync(0xffffffffu, offsets[at] <= t));  // ascending: the first `hits` lanes
    const int past = min(n, hits * gap);
    lo += past;
    n = hits == 32 ? 0 : min(n - past, gap) - 1;
  }
  return lo - 1;
}

// Where a token's rows go: page (< 0: nowhere) and slot in it; pos: its logical slot.
struct Place {
  int page, slot, pos;
};

// Laid out as qk_norm_rope_kernel, but that the groups run through the heads of
// the keys and on into those of the values (few heads fill one group): keys normed
// and rotated, values copied, both into the token's page slot.
template <int HD>
__global__ void __launch_bounds__(32 * kRopeWarps, kRopeBlocks) rope_kv_append_kernel(const __grid_constant__ AppendArgs p,
                                                                              const __grid_constant__ RopeFreq f) {
  constexpr int L = HD / 16, U = 2, step = 32 / L;
  using S = RopeSmem<bf16, HD, U, 1>;
  extern __shared__ uint4 s_rope[];
  __shared__ __align__(16) unsigned long long s_turn[kMaxHalfRope];
  const int lane = threadIdx.x & 31, i = lane & (L - 1), n_warps = blockDim.x >> 5;
  uint4 *stages = s_rope + (threadIdx.x >> 5) * S::warp + lane;
  float *factors = (float *)(s_rope + (threadIdx.x >> 5) * S::warp + kStages * S::stage);
  int c0, c1;
  lane_chunks(i, p.rd16, &c0, &c1);
  const bool turns = i < p.rd16;
  const uint32_t stride = gridDim.x * n_warps;
  At at(p.plan, blockIdx.x * n_warps + (threadIdx.x >> 5), p.n_tok), ahead = at;
  // a lane's heads of a group: h, h + step, .. of the keys' heads and then the values'
  auto head_of = [&](const At &at) { return U * step * at.g + lane / L; };
  auto request = [&](int stage) {
    if (!ahead.end()) {
      const int h = head_of(ahead);
      const bf16 *k = p.k + ahead.t * p.k_stride, *v = p.v + ahead.t * p.v_stride - (long long)p.Hkv * HD;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int hu = h + u * step;
        if (hu < 2 * p.Hkv)
          Chunks<bf16>::request(stages + stage * S::stage + 64 * u, (hu < p.Hkv ? k : v) + (long long)hu * HD, c0, c1);
      }
      if (++ahead.g == ahead.g1) ahead.set(p.plan, ahead.item + stride, p.n_tok);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
  // where token t's rows go; the same in the whole warp
  auto place_of = [&](int t) {
    const int b = row_sequence(p.offsets, p.n_seqs, t);
    Place to{-1, 0, 0};
    if (b < 0 || b >= p.n_seqs) return to;  // rows of no sequence take no part
    const long long slot = (long long)p.prefix[b] + t - p.offsets[b];
    if (slot >= 0 && slot < min((long long)p.max_pages * p.pg, 0x7fffffffll)) {
      const int logical = (int)slot / p.pg;
      to.page = p.tables[(long long)b * p.max_pages + logical];
      to.slot = (int)slot - logical * p.pg;
      to.pos = (int)slot;
    }
    if (to.page < 0 || to.page >= p.n_pages) {  // not written, reported by dg_op_status
      to.page = -1;
      if (lane == 0 && p.err) atomicExch(p.err + 1, kBadPage);
    }
    return to;
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) request(k);
  Place to{-1, 0, 0};
  int stage = 0, pos = 0;
  if (!at.end()) {
    to = place_of((int)at.t);
    pos = p.positions ? p.positions[at.t] : to.pos;
  }
  for (int j = threadIdx.x; j < 8 * p.rd16; j += blockDim.x) s_turn[j] = f.turn[j];
  __syncthreads();
  while (!at.end()) {
    if (U * step * at.g0 < p.Hkv) {  // the token's factors, while its rows are in flight
#pragma unroll
      for (int j = 2 * lane; j < HD / 2; j += 64) {
        float2 sc0 = make_float2(0.0f, 1.0f), sc1 = sc0;
        if (j < 8 * p.rd16) {
          const ulonglong2 turn = *(const ulonglong2 *)(s_turn + j);
          sc0 = turn_angle(turn.x, pos);
          sc1 = turn_angle(turn.y, pos);
        }
        put_factors<HD>(factors, j, p.rd16, p.k_gain, sc0, sc1);
      }
    }
    __syncwarp();
    At next = at;
    next.set(p.plan, at.item + stride, p.n_tok);
    Place next_to{-1, 0, 0};
    if (!next.end()) {
      next_to = place_of((int)next.t);
      pos = p.positions ? p.positions[next.t] : next_to.pos;
    }
    for (; !at.end(); ++at.g) {
      const int h = head_of(at), keys = p.Hkv - U * step * at.g;  // keys: the group's, if more than 0
      asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 2) : "memory");
      Chunks<bf16> y[U];
#pragma unroll
      for (int u = 0; u < U; ++u) y[u].read(stages + stage * S::stage + 64 * u);
      if (keys > 0) {
        f32x2 x[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          unpack8(y[u].a, x[u]);
          unpack8(y[u].b, x[u] + 4);
        }
        turn_heads<HD, U>(x, keys > step ? U : 1, p.k_gain != nullptr, true, p.eps, turns, factors, i);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (h + u * step < p.Hkv) {
            y[u].a[0] = pack8(x[u]);
            y[u].b[0] = pack8(x[u] + 4);
          }
        }
      }
      request(stage ? stage - 1 : kStages - 1);  // the stage that was read last
      stage = stage == kStages - 1 ? 0 : stage + 1;
      if (to.page >= 0) {
        const long long head = (long long)p.pg * HD;
        const int s7 = to.slot & 7;
        const long long at0 = (long long)to.page * p.Hkv * head + (long long)to.slot * 64;
        const long long d0 = (long long)(c0 >> 3) * p.pg * 64 + (((c0 & 7) ^ s7) << 3);
        const long long d1 = (long long)(c1 >> 3) * p.pg * 64 + (((c1 & 7) ^ s7) << 3);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int hu = h + u * step;
          if (hu < 2 * p.Hkv) {
            bf16 *dst = (hu < p.Hkv ? p.k_pool : p.v_pool) + at0 + (hu < p.Hkv ? hu : hu - p.Hkv) * head;
            *(uint4 *)(dst + d0) = y[u].a[0];
            *(uint4 *)(dst + d1) = y[u].b[0];
          }
        }
      }
    }
    __syncwarp();  // the factors have been read
    at = next;
    to = next_to;
  }
}

// The frequencies of a call; those of the thread's last call are kept (64
// calls of pow take longer than the launch).
const RopeFreq &rope_frequencies(int rope_dim, float base) {
  static thread_local RopeFreq f;
  static thread_local int last_dim = -1;
  static thread_local float last_base = 0.0f;
  if (rope_dim == last_dim && base == last_base) return f;
  for (int j = 0; j < kMaxHalfRope; ++j) {
    f.turn[j] = 0;
    if (2 * j >= rope_dim) continue;
    const double turns = pow((double)base, -2.0 * j / rope_dim) * 0.15915494309189535;  // / (2 pi), below 1
    f.turn[j] = (unsigned long long)(turns * 18446744073709551616.0);
  }
  last_dim = rope_dim;
  last_base = base;
  return f;
}

struct RopeLaunch {
  RopePlan plan;
  int grid, threads;
};

// first, second: heads of the two sides; group: heads of a group.
RopeLaunch rope_plan(int n_tok, int first, int second, int group) {
  RopeLaunch r;
  RopePlan &p = r.plan;
  p.first = (first + group - 1) / group;
  p.groups = p.first + (second + group - 1) / group;
  // parts of a token, each with factors of its own, only while whole tokens
  // would leave warps without work
  constexpr int most = 152 * kRopeBlocks * kRopeWarps;
  int want = most / n_tok;
  if (want > p.groups) want = p.groups;
  if (want < 1) want = 1;
  p.each = (p.groups + want - 1) / want;
  p.parts = (p.groups + p.each - 1) / p.each;
  const long long items = (long long)n_tok * p.parts;
  const int warps = (int)(items < 152 * kRopeWarps ? (items + 151) / 152 : kRopeWarps);
  // every warp the same count of items
  const long long rounds = (items + most - 1) / most;
  r.threads = 32 * warps;
  r.grid = (int)((items + rounds * warps - 1) / (rounds * warps));
  return r;
}

// A kernel's blocks may ask for more than the 48 KiB that need no leave: it is
// taken for the most a block asks for, whatever this call does (another thread
// may be about to launch a larger one).
template <typename K>
cudaError_t rope_smem(K kern, size_t bytes, size_t per_warp) {
  if (bytes <= (40 << 10)) return cudaSuccess;
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kRopeWarps * per_warp));
}

template <typename T, int HD>
cudaError_t launch_qk(QkArgs p, const RopeFreq &f, cudaStream_t st) {
  constexpr int U = sizeof(T) == 2 ? 2 : 1;
  const RopeLaunch l = rope_plan(p.n_tok, p.Hq, p.Hkv, 32 / (HD / 16) * U);
  p.plan = l.plan;
  constexpr size_t per_warp = RopeSmem<T, HD, U, 2>::warp * 16;
  const size_t smem = l.threads / 32 * per_warp;
  const cudaError_t e = rope_smem(qk_norm_rope_kernel<T, HD>, smem, per_warp);
  if (e != cudaSuccess) return e;
  qk_norm_rope_kernel<T, HD><<<l.grid, l.threads, smem, st>>>(p, f);
  return cudaGetLastError();
}

template <int HD>
cudaError_t launch_append(AppendArgs p, const RopeFreq &f, cudaStream_t st) {
  const RopeLaunch l = rope_plan(p.n_tok, 2 * p.Hkv, 0, 32 / (HD / 16) * 2);
  p.plan = l.plan;
  constexpr size_t per_warp = RopeSmem<bf16, HD, 2, 1>::warp * 16;
  const size_t smem = l.threads / 32 * per_warp;
  const cudaError_t e = rope_smem(rope_kv_append_kernel<HD>, smem, per_warp);
  if (e != cudaSuccess) return e;
  rope_kv_append_kernel<HD><<<l.grid, l.threads, smem, st>>>(p, f);
  return cudaGetLastError();
}

}  // namespace

cudaError_t qk_norm_rope(const QkNormRope &a, cudaStream_t st) {
  if (a.n_tok == 0 || a.Hq + a.Hkv == 0) return cudaSuccess;
  const QkArgs p{a.q, a.k, a.q_stride, a.k_stride, a.positions, a.n_tok, a.Hq, a.Hkv, a.rope_dim / 16,
                 a.q_gain, a.k_gain, a.eps, a.q_out, a.k_out, a.q_out_stride, a.k_out_stride, {}};
  const RopeFreq &f = rope_frequencies(a.rope_dim, a.rope_base);
  if (a.in_f32)
    return a.hd == 64 ? launch_qk<float, 64>(p, f, st) : a.hd == 128 ? launch_qk<float, 128>(p, f, st) : launch_qk<float, 256>(p, f, st);
  return a.hd == 64 ? launch_qk<bf16, 64>(p, f, st) : a.hd == 128 ? launch_qk<bf16, 128>(p, f, st) : launch_qk<bf16, 256>(p, f, st);
}

cudaError_t rope_kv_append(const RopeKvAppend &a, int *err, cudaStream_t st) {
  if (a.n_tok == 0 || a.n_seqs == 0) return cudaSuccess;
  const AppendArgs p{a.k, a.v, a.k_stride, a.v_stride, a.positions, a.prefix_lens, a.offsets, a.page_tables,
                     a.max_pages, a.n_seqs, a.n_tok, a.Hkv, a.rope_dim / 16, a.k_gain, a.eps, a.k_pool, a.v_pool,
                     a.n_pages, a.pg, err, {}};
  const RopeFreq &f = rope_frequencies(a.rope_dim, a.rope_base);
  return a.hd == 64 ? launch_append<64>(p, f, st) : a.hd == 128 ? launch_append<128>(p, f, st) : launch_append<256>(p, f, st);
}

}  // namespace dg
