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
// at position 10^6), and its top 32 bits go to sincospif.
//
// Layout: a head is handled by hd / 16 lanes.  Lane i < rd / 16 holds the
// 8-element chunks i and i + rd / 16, whose elements rotate with one another,
// the lanes behind it the chunks 2 i and 2 i + 1: the rotation needs no
// exchange between lanes, and loads and stores are 16 bytes wide.
#include <math.h>

#include "internal.h"

namespace dg {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kMaxHalfRope = 128;

// Frequencies of the rotation in turns, as 64-bit fractions.
struct RopeFreq {
  unsigned long long turn[kMaxHalfRope];
};

struct HeadVec {
  float a[8], b[8];  // the lane's two chunks
};

__device__ __forceinline__ void unpack8(uint4 w, float *x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float *x) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *(const uint32_t *)&v;
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ void load8(const bf16 *p, float *x) { unpack8(*(const uint4 *)p, x); }
__device__ __forceinline__ void load8(const float *p, float *x) {
  const float4 u = *(const float4 *)p, v = *(const float4 *)(p + 4);
  x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
  x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
}

// Chunk indices of lane i of a head.
__device__ __forceinline__ void lane_chunks(int i, int rd16, int *c0, int *c1) {
  *c0 = i < rd16 ? i : 2 * i;
  *c1 = i < rd16 ? i + rd16 : 2 * i + 1;
}

// Norm of the head whose values the `lanes` lanes of a group hold.
__device__ __forceinline__ void head_norm(HeadVec &x, const float *gain, int c0, int c1, int hd, float eps, int lanes) {
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s += x.a[e] * x.a[e] + x.b[e] * x.b[e];
  for (int o = lanes >> 1; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const float r = rsqrtf(s / (float)hd + eps);
  float ga[8], gb[8];
  load8(gain + 8 * c0, ga);
  load8(gain + 8 * c1, gb);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x.a[e] = x.a[e] * r * ga[e];
    x.b[e] = x.b[e] * r * gb[e];
  }
}

__device__ __forceinline__ void lane_angles(const RopeFreq &f, int i, int pos, float *cs, float *sn) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const unsigned long long t = (unsigned long long)(long long)pos * f.turn[8 * i + e];
    sincospif((float)(int)(t >> 32) * 4.656612873077393e-10f, sn + e, cs + e);  // 2^-31: half turns
  }
}

__device__ __forceinline__ void rotate(HeadVec &x, const float *cs, const float *sn) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = x.a[e], b = x.b[e];
    x.a[e] = a * cs[e] - b * sn[e];
    x.b[e] = b * cs[e] + a * sn[e];
  }
}

struct QkArgs {
  const void *q, *k;
  long long q_stride, k_stride;
  const int *positions;
  int n_tok, Hq, Hkv, hd, rd16;
  const float *q_gain, *k_gain;
  float eps;
  bf16 *q_out, *k_out;
  long long q_out_stride, k_out_stride;
};

// One group of hd / 16 lanes per (token, head).
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const QkArgs p, const RopeFreq f) {
  const int lanes = p.hd / 16, i = threadIdx.x & (lanes - 1);
  const int H = p.Hq + p.Hkv;
  const long long n = (long long)p.n_tok * H;
  const int per_block = kRopeThreads / lanes;
  int c0, c1;
  lane_chunks(i, p.rd16, &c0, &c1);
  for (long long base = (long long)blockIdx.x * per_block; base < n; base += (long long)gridDim.x * per_block) {
    const long long item = base + threadIdx.x / lanes;
    const bool ok = item < n;  // the whole warp stays for the norm's exchange
    const int t = ok ? (int)(item / H) : 0, h = ok ? (int)(item - (long long)t * H) : 0;
    const bool is_q = h < p.Hq;
    const T *src = is_q ? (const T *)p.q + t * p.q_stride + (long long)h * p.hd
                        : (const T *)p.k + t * p.k_stride + (long long)(h - p.Hq) * p.hd;
    bf16 *dst = is_q ? p.q_out + t * p.q_out_stride + (long long)h * p.hd
                     : p.k_out + t * p.k_out_stride + (long long)(h - p.Hq) * p.hd;
    const float *gain = is_q ? p.q_gain : p.k_gain;
    HeadVec x = {};
    if (ok) {
      load8(src + 8 * c0, x.a);
      load8(src + 8 * c1, x.b);
    }
    HeadVec y = x;
    const float *g = gain ? gain : (p.q_gain ? p.q_gain : p.k_gain);
    if (g) head_norm(y, g, c0, c1, p.hd, p.eps, lanes);
    if (gain) x = y;
    if (i < p.rd16 && ok) {
      float cs[8], sn[8];
      lane_angles(f, i, p.positions[t], cs, sn);
      rotate(x, cs, sn);
    }
    if (ok) {
      *(uint4 *)(dst + 8 * c0) = pack8(x.a);
      *(uint4 *)(dst + 8 * c1) = pack8(x.b);
    }
  }
}

struct AppendArgs {
  const bf16 *k, *v;
  long long k_stride, v_stride;
  const int *positions, *prefix, *offsets, *tables;
  int max_pages, n_seqs, n_tok, Hkv, hd, rd16;
  const float *k_gain;
  float eps;
  bf16 *k_pool, *v_pool;
  int n_pages, pg;
  int *err;
};

// Sequence of packed row t: the last b with offsets[b] <= t; n_seqs when the
// row lies behind the last sequence, -1 before the first.
__device__ __forceinline__ int row_sequence(const int *offsets, int n_seqs, int t) {
  if (t >= offsets[n_seqs]) return n_seqs;
  int lo = -1, hi = n_seqs;  // offsets[lo] <= t < offsets[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// One group of hd / 16 lanes per (token, KV head): the key normed and
// rotated, the value copied, both into the token's page slot.
__global__ void __launch_bounds__(kRopeThreads) rope_kv_append_kernel(const AppendArgs p, const RopeFreq f) {
  const int lanes = p.hd / 16, i = threadIdx.x & (lanes - 1);
  const long long n = (long long)p.n_tok * p.Hkv;
  const int per_block = kRopeThreads / lanes;
  int c0, c1;
  lane_chunks(i, p.rd16, &c0, &c1);
  for (long long base = (long long)blockIdx.x * per_block; base < n; base += (long long)gridDim.x * per_block) {
    const long long item = base + threadIdx.x / lanes;
    bool ok = item < n;
    const int t = ok ? (int)(item / p.Hkv) : 0, h = ok ? (int)(item - (long long)t * p.Hkv) : 0;
    long long slot = 0, blk = 0;
    if (ok) {
      const int b = row_sequence(p.offsets, p.n_seqs, t);
      ok = b < p.n_seqs;  // rows behind the last sequence are left alone
      if (ok) {
        int page = -1;
        slot = b < 0 ? -1 : (long long)p.prefix[b] + (t - p.offsets[b]);
        if (slot >= 0 && slot < (long long)p.max_pages * p.pg) page = p.tables[(long long)b * p.max_pages + slot / p.pg];
        if (page < 0 || page >= p.n_pages) {  // not written, reported by dg_op_status
          if (i == 0 && p.err) atomicExch(p.err + 1, kBadPage);
          ok = false;
        } else {
          blk = ((long long)page * p.Hkv + h) * p.pg * p.hd;
        }
      }
    }
    HeadVec x = {};
    uint4 va = {}, vb = {};
    if (ok) {
      const bf16 *ks = p.k + t * p.k_stride + (long long)h * p.hd, *vs = p.v + t * p.v_stride + (long long)h * p.hd;
      load8(ks + 8 * c0, x.a);
      load8(ks + 8 * c1, x.b);
      va = *(const uint4 *)(vs + 8 * c0);
      vb = *(const uint4 *)(vs + 8 * c1);
    }
    if (p.k_gain) head_norm(x, p.k_gain, c0, c1, p.hd, p.eps, lanes);
    if (!ok) continue;
    if (i < p.rd16) {
      float cs[8], sn[8];
      lane_angles(f, i, p.positions ? p.positions[t] : (int)slot, cs, sn);
      rotate(x, cs, sn);
    }
    const int s = (int)(slot % p.pg);
    auto at = [&](int c) { return blk + (long long)(c >> 3) * p.pg * 64 + (long long)s * 64 + (((c & 7) ^ (s & 7)) << 3); };
    *(uint4 *)(p.k_pool + at(c0)) = pack8(x.a);
    *(uint4 *)(p.k_pool + at(c1)) = pack8(x.b);
    *(uint4 *)(p.v_pool + at(c0)) = va;
    *(uint4 *)(p.v_pool + at(c1)) = vb;
  }
}

void rope_frequencies(RopeFreq *f, int rope_dim, float base) {
  for (int j = 0; j < kMaxHalfRope; ++j) {
    f->turn[j] = 0;
    if (2 * j >= rope_dim) continue;
    const double turns = pow((double)base, -2.0 * j / rope_dim) * 0.15915494309189535;  // / (2 pi)
    const double frac = turns - floor(turns);
    f->turn[j] = (unsigned long long)(frac * 18446744073709551616.0);
  }
}

}  // namespace

cudaError_t qk_norm_rope(const QkNormRope &a, cudaStream_t st) {
  const long long n = (long long)a.n_tok * (a.Hq + a.Hkv);
  if (n == 0) return cudaSuccess;
  RopeFreq f;
  rope_frequencies(&f, a.rope_dim, a.rope_base);
  QkArgs p{a.q, a.k, a.q_stride, a.k_stride, a.positions, a.n_tok, a.Hq, a.Hkv, a.hd, a.rope_dim / 16,
           a.q_gain, a.k_gain, a.eps, a.q_out, a.k_out, a.q_out_stride, a.k_out_stride};
  const long long per_block = kRopeThreads / (a.hd / 16);
  const long long blocks = (n + per_block - 1) / per_block;
  const int grid = (int)(blocks < 152 * 64 ? blocks : 152 * 64);
  if (a.in_f32)
    qk_norm_rope_kernel<float><<<grid, kRopeThreads, 0, st>>>(p, f);
  else
    qk_norm_rope_kernel<bf16><<<grid, kRopeThreads, 0, st>>>(p, f);
  return cudaGetLastError();
}

cudaError_t rope_kv_append(const RopeKvAppend &a, int *err, cudaStream_t st) {
  const long long n = (long long)a.n_tok * a.Hkv;
  if (n == 0) return cudaSuccess;
  RopeFreq f;
  rope_frequencies(&f, a.rope_dim, a.rope_base);
  AppendArgs p{a.k, a.v, a.k_stride, a.v_stride, a.positions, a.prefix_lens, a.offsets, a.page_tables,
               a.max_pages, a.n_seqs, a.n_tok, a.Hkv, a.hd, a.rope_dim / 16, a.k_gain, a.eps, a.k_pool, a.v_pool,
               a.n_pages, a.pg, err};
  const long long per_block = kRopeThreads / (a.hd / 16);
  const long long blocks = (n + per_block - 1) / per_block;
  const int grid = (int)(blocks < 152 * 64 ? blocks : 152 * 64);
  rope_kv_append_kernel<<<grid, kRopeThreads, 0, st>>>(p, f);
  return cudaGetLastError();
}

}  // namespace dg
