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
// Bound by the bytes of the rows.  Layout: a head is handled by hd / 16 lanes.
// Lane i < rd / 16 holds the 8-element chunks i and i + rd / 16, whose elements
// rotate with one another, the lanes behind it the chunks 2 i and 2 i + 1: the
// rotation needs no exchange between lanes, and loads and stores are 16 bytes
// wide.  A block takes a few tokens at a time, all their heads at once: while
// the rows are in flight its threads compute the tokens' sines and cosines
// once each, multiplied with the gains, into shared memory, from where every
// head of a token takes them.
#include <math.h>

#include "f32x2.cuh"
#include "internal.h"

namespace dg {

namespace {

constexpr int kRopeThreads = 512;   // most threads of a block
constexpr int kMaxHalfRope = 128;
constexpr int kRopeSmem = 64 << 10;  // most shared memory of a block's factors

// Frequencies of the rotation in turns, as 64-bit fractions.
struct RopeFreq {
  unsigned long long turn[kMaxHalfRope];
};

// A lane's two chunks of a head as loaded.
template <typename T>
struct Chunks {
  uint4 a[sizeof(T) / 2], b[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ void load_chunks(Chunks<T> &x, const T *head, int c0, int c1) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
    x.a[i] = ((const uint4 *)(head + 8 * c0))[i];
    x.b[i] = ((const uint4 *)(head + 8 * c1))[i];
  }
}

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

// Factors of pair j (element j of the lanes' first chunks and its partner).
template <int HD>
__device__ __forceinline__ void put_factors(float *to, int j, int rd16, const float *gain, float2 sc) {
  constexpr int L = HD / 16;
  const int i = j >> 3, e = j & 7;
  int c0, c1;
  lane_chunks(i, rd16, &c0, &c1);
  const float ga = gain ? gain[8 * c0 + e] : 1.0f, gb = gain ? gain[8 * c1 + e] : 1.0f;
  float *at = to + ((e >> 2) * L + i) * 4 + (e & 3);
  at[0 * 8 * L] = ga * sc.y;
  at[1 * 8 * L] = -gb * sc.x;
  at[2 * 8 * L] = gb * sc.y;
  at[3 * 8 * L] = ga * sc.x;
}

// Norm (any: some head of the launch has one; normed: this one) and rotation of
// a lane's chunks with its token's factors.
template <int HD>
__device__ __forceinline__ void turn_head(f32x2 *a, f32x2 *b, bool any, bool normed, float eps, bool turns, const float *factors, int i) {
  constexpr int L = HD / 16;
  if (any) {
    const float r = head_scale<HD>(a, b, eps);
    const f32x2 rr = pair(r, r);
    if (normed) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = mul2(a[e], rr);
        b[e] = mul2(b[e], rr);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const ulonglong2 *at = (const ulonglong2 *)factors + (e >> 1) * L + i;
    const ulonglong2 ac = at[0], bc = at[4 * L];
    const f32x2 x0 = a[e], x1 = a[e + 1], y0 = b[e], y1 = b[e + 1];
    a[e] = mul2(x0, ac.x);
    a[e + 1] = mul2(x1, ac.y);
    b[e] = mul2(y0, bc.x);
    b[e + 1] = mul2(y1, bc.y);
    if (turns) {
      const ulonglong2 bs = at[2 * L], as = at[6 * L];
      a[e] = fma2(y0, bs.x, a[e]);
      a[e + 1] = fma2(y1, bs.y, a[e + 1]);
      b[e] = fma2(x0, as.x, b[e]);
      b[e + 1] = fma2(x1, as.y, b[e + 1]);
    }
  }
}

// How a launch is laid out: a block's threads are `abreast` tokens x heads x
// lanes (heads in `rounds` turns when they exceed a block), and each takes up
// to `deep` tokens at a time.
struct RopePlan {
  int abreast, deep, heads, rounds, threads, grid;
  size_t smem;
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

// Tokens a thread has in flight (of bf16 rows; half as many of fp32 rows or of
// keys with values) and the resident blocks the registers are held down for:
// 16384 tokens of 16 + 8 heads of 128 take 40.8 us with (2, 2), 46.3 with
// (4, 2), 50.4 with (2, 1): latency, not bytes, rules below half occupancy.
constexpr int kDeep = 2, kRopeBlocks = 2;

template <typename T, int HD>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) qk_norm_rope_kernel(const __grid_constant__ QkArgs p,
                                                                    const __grid_constant__ RopeFreq f) {
  constexpr int L = HD / 16, F = 2 * HD, kU = sizeof(T) == 2 ? kDeep : kDeep / 2;
  extern __shared__ float4 s_factors4[];
  float *s_factors = (float *)s_factors4;  // [token][q, k][F]
  __shared__ unsigned long long s_turn[kMaxHalfRope];
  for (int j = threadIdx.x; j < 8 * p.rd16; j += blockDim.x) s_turn[j] = f.turn[j];
  __syncthreads();
  const int i = threadIdx.x & (L - 1), H = p.Hq + p.Hkv;
  const int tt = (threadIdx.x / L) / p.plan.heads, h_mine = threadIdx.x / L - tt * p.plan.heads;
  int c0, c1;
  lane_chunks(i, p.rd16, &c0, &c1);
  const bool turns = i < p.rd16;
  const int block_toks = p.plan.abreast * min(kU, p.plan.deep);
  for (long long t0 = (long long)blockIdx.x * block_toks; t0 < p.n_tok; t0 += (long long)gridDim.x * block_toks) {
    const int n_here = (int)min((long long)block_toks, p.n_tok - t0);
    for (int round = 0; round < p.plan.rounds; ++round) {
      const int h = round * p.plan.heads + h_mine;
      const bool is_q = h < p.Hq, live = tt < p.plan.abreast && h < H;
      const T *src = (is_q ? (const T *)p.q + t0 * p.q_stride + (long long)h * HD
                           : (const T *)p.k + t0 * p.k_stride + (long long)(h - p.Hq) * HD);
      const long long stride = is_q ? p.q_stride : p.k_stride;
      Chunks<T> x[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int t = tt + u * p.plan.abreast;
        if (live && t < n_here) load_chunks(x[u], src + t * stride, c0, c1);
      }
      if (round == 0) {  // the factors, while the rows are in flight
        __syncthreads();  // the last tokens' have been read
        for (int it = threadIdx.x; it < n_here * (HD / 2); it += blockDim.x) {
          const int t = it / (HD / 2), j = it & (HD / 2 - 1);
          float2 sc = make_float2(0.0f, 1.0f);
          if (j < 8 * p.rd16) sc = turn_angle(s_turn[j], p.positions[t0 + t]);
          if (p.Hq) put_factors<HD>(s_factors + (2 * t) * F, j, p.rd16, p.q_gain, sc);
          if (p.Hkv) put_factors<HD>(s_factors + (2 * t + 1) * F, j, p.rd16, p.k_gain, sc);
        }
        __syncthreads();
      }
      bf16 *dst = is_q ? p.q_out + t0 * p.q_out_stride + (long long)h * HD
                       : p.k_out + t0 * p.k_out_stride + (long long)(h - p.Hq) * HD;
      const long long dst_stride = is_q ? p.q_out_stride : p.k_out_stride;
      const bool normed = is_q ? p.q_gain != nullptr : p.k_gain != nullptr;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int t = tt + u * p.plan.abreast;
        if (u * p.plan.abreast >= n_here) break;  // the same in the whole block
        f32x2 a[4], b[4];
        unpack8(x[u].a, a);
        unpack8(x[u].b, b);
        turn_head<HD>(a, b, p.q_gain || p.k_gain, normed, p.eps, turns, s_factors + (2 * min(t, n_here - 1) + !is_q) * F, i);
        if (live && t < n_here) {
          *(uint4 *)(dst + t * dst_stride + 8 * c0) = pack8(a);
          *(uint4 *)(dst + t * dst_stride + 8 * c1) = pack8(b);
        }
      }
    }
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

// Laid out as qk_norm_rope_kernel: keys normed and rotated, values copied, both
// into the token's page slot.
template <int HD>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) rope_kv_append_kernel(const __grid_constant__ AppendArgs p,
                                                                      const __grid_constant__ RopeFreq f) {
  constexpr int L = HD / 16, F = 2 * HD, kU = kDeep / 2;
  extern __shared__ float4 s_factors4[];
  float *s_factors = (float *)s_factors4;  // [token][F]
  __shared__ unsigned long long s_turn[kMaxHalfRope];
  __shared__ Place s_place[kRopeThreads / 4 * kU];
  for (int j = threadIdx.x; j < 8 * p.rd16; j += blockDim.x) s_turn[j] = f.turn[j];
  __syncthreads();
  const int i = threadIdx.x & (L - 1);
  const int tt = (threadIdx.x / L) / p.plan.heads, h_mine = threadIdx.x / L - tt * p.plan.heads;
  int c0, c1;
  lane_chunks(i, p.rd16, &c0, &c1);
  const bool turns = i < p.rd16;
  const int block_toks = p.plan.abreast * min(kU, p.plan.deep);
  for (long long t0 = (long long)blockIdx.x * block_toks; t0 < p.n_tok; t0 += (long long)gridDim.x * block_toks) {
    const int n_here = (int)min((long long)block_toks, p.n_tok - t0);
    for (int round = 0; round < p.plan.rounds; ++round) {
      const int h = round * p.plan.heads + h_mine;
      const bool live = tt < p.plan.abreast && h < p.Hkv;
      const bf16 *ks = p.k + t0 * p.k_stride + (long long)h * HD, *vs = p.v + t0 * p.v_stride + (long long)h * HD;
      Chunks<bf16> x[kU], y[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int t = tt + u * p.plan.abreast;
        if (live && t < n_here) {
          load_chunks(x[u], ks + t * p.k_stride, c0, c1);
          load_chunks(y[u], vs + t * p.v_stride, c0, c1);
        }
      }
      if (round == 0) {  // slots and factors, while the rows are in flight
        __syncthreads();  // the last tokens' have been read
        for (int t = threadIdx.x >> 5; t < n_here; t += blockDim.x >> 5) {
          const int row = (int)t0 + t, b = row_sequence(p.offsets, p.n_seqs, row);
          Place at{-1, 0, 0};
          if (b < p.n_seqs) {  // rows behind the last sequence are left alone
            const long long slot = b < 0 ? -1 : (long long)p.prefix[b] + row - p.offsets[b];
            if (slot >= 0 && slot < min((long long)p.max_pages * p.pg, 0x7fffffffll)) {
              const int logical = (int)slot / p.pg;
              at.page = p.tables[(long long)b * p.max_pages + logical];
              at.slot = (int)slot - logical * p.pg;
              at.pos = (int)slot;
            }
            if (at.page < 0 || at.page >= p.n_pages) {  // not written, reported by dg_op_status
              at.page = -1;
              if ((threadIdx.x & 31) == 0 && p.err) atomicExch(p.err + 1, kBadPage);
            }
          }
          if ((threadIdx.x & 31) == 0) s_place[t] = at;
        }
        if (!p.positions) __syncthreads();  // the angles go by the slots
        for (int it = threadIdx.x; it < n_here * (HD / 2); it += blockDim.x) {
          const int t = it / (HD / 2), j = it & (HD / 2 - 1);
          float2 sc = make_float2(0.0f, 1.0f);
          if (j < 8 * p.rd16) sc = turn_angle(s_turn[j], p.positions ? p.positions[t0 + t] : s_place[t].pos);
          put_factors<HD>(s_factors + t * F, j, p.rd16, p.k_gain, sc);
        }
        __syncthreads();
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int t = tt + u * p.plan.abreast;
        if (u * p.plan.abreast >= n_here) break;  // the same in the whole block
        f32x2 a[4], b[4];
        unpack8(x[u].a, a);
        unpack8(x[u].b, b);
        const int ts = min(t, n_here - 1);
        turn_head<HD>(a, b, p.k_gain != nullptr, p.k_gain != nullptr, p.eps, turns, s_factors + ts * F, i);
        const Place at = s_place[ts];
        if (live && t < n_here && at.page >= 0) {
          const long long blk = ((long long)at.page * p.Hkv + h) * p.pg * HD + (long long)at.slot * 64;
          const long long a0 = blk + (long long)(c0 >> 3) * p.pg * 64 + (((c0 & 7) ^ (at.slot & 7)) << 3);
          const long long a1 = blk + (long long)(c1 >> 3) * p.pg * 64 + (((c1 & 7) ^ (at.slot & 7)) << 3);
          *(uint4 *)(p.k_pool + a0) = pack8(a);
          *(uint4 *)(p.k_pool + a1) = pack8(b);
          *(uint4 *)(p.v_pool + a0) = y[u].a[0];
          *(uint4 *)(p.v_pool + a1) = y[u].b[0];
        }
      }
    }
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

// heads: of all sides; sides: factor sets per token; in_flight: tokens a thread
// loads at once.
RopePlan rope_plan(int n_tok, int heads, int hd, int sides, int in_flight) {
  RopePlan r;
  const int lanes = hd / 16;
  r.heads = heads * lanes <= kRopeThreads ? heads : kRopeThreads / lanes;
  r.rounds = (heads + r.heads - 1) / r.heads;
  r.abreast = 256 / (r.heads * lanes);
  if (r.abreast < 1) r.abreast = 1;
  r.deep = in_flight;
  const size_t per_tok = (size_t)sides * 2 * hd * sizeof(float);
  while (r.abreast > 1 && r.abreast * r.deep * per_tok > kRopeSmem) --r.abreast;
  // fewer tokens a block while the blocks do not fill the machine
  while (r.deep > 1 && (long long)r.abreast * r.deep * 152 * 4 > n_tok) r.deep /= 2;
  while (r.abreast > 1 && (long long)r.abreast * 152 * 2 > n_tok) r.abreast /= 2;
  r.threads = (r.abreast * r.heads * lanes + 31) / 32 * 32;
  const int toks = r.abreast * r.deep, blocks = (n_tok + toks - 1) / toks;
  r.grid = blocks < 152 * 32 ? blocks : 152 * 32;
  r.smem = toks * per_tok;
  return r;
}

template <typename T, int HD>
cudaError_t launch_qk(QkArgs p, const RopeFreq &f, cudaStream_t st) {
  p.plan = rope_plan(p.n_tok, p.Hq + p.Hkv, HD, 2, sizeof(T) == 2 ? kDeep : kDeep / 2);
  auto kern = qk_norm_rope_kernel<T, HD>;
  if (p.plan.smem > (48 << 10) - 2048) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRopeSmem);
    if (e != cudaSuccess) return e;
  }
  kern<<<p.plan.grid, p.plan.threads, p.plan.smem, st>>>(p, f);
  return cudaGetLastError();
}

template <int HD>
cudaError_t launch_append(AppendArgs p, const RopeFreq &f, cudaStream_t st) {
  p.plan = rope_plan(p.n_tok, p.Hkv, HD, 1, kDeep / 2);
  auto kern = rope_kv_append_kernel<HD>;
  if (p.plan.smem > (48 << 10) - 8192) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRopeSmem);
    if (e != cudaSuccess) return e;
  }
  kern<<<p.plan.grid, p.plan.threads, p.plan.smem, st>>>(p, f);
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
