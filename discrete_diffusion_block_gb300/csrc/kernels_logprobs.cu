// Log probabilities of given tokens under rows of logits, with each row's
// entropy and its most likely tokens.  With y = logit / tau, m = max y,
// S = sum e^(y - m), A = sum e^(y - m) (y - m):
//   log p(v) = (y_v - m) - log S,  lse = m + log S,  entropy = log S - A / S.
//
// Bound by the logits' bytes, each read once.  A row is split over the blocks
// of a cluster when there are fewer rows than blocks fit the machine, and
// their states joined through distributed shared memory (one launch, no
// workspace).  A thread takes a batch of kVecs 16-byte vectors at a time, the
// next batch already in flight, and moves its running maximum once per batch;
// sums are kept in units of log2, fp32.
//
// The most likely tokens: each warp keeps a list of its 32 best entries, one a
// lane, in descending order of a 64-bit key (order-preserving bits of the
// value, then the complement of the index: equal values go to the lower
// index).  A list starts empty, so nearly every entry of a warp's first
// batches would enter it; the k-th largest of the block's thread maxima of the
// first batch is a lower bound of the block's k-th best entry, and entries
// below it are dropped at one compare per batch: of a row of 262144 random
// logits about k * 262144 / 8192 reach a list, however many warps share it.
#include "gemm_tc.cuh"
#include "internal.h"

namespace dg {

namespace {

constexpr int kLpThreads = 512, kLpWarps = kLpThreads / 32;
constexpr int kVecs = 4;            // 16-byte vectors of a thread's batch
constexpr int kMaxLpCluster = 16;   // blocks of a row (a non-portable cluster size)
constexpr float kLn2f = 0.693147180559945309f;

// m: largest raw logit; s = sum 2^d, a = sum 2^d d with d = (x - m) c.
struct RowSum {
  float m, s, a;
};

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// (s, a) moved to a reference maximum that is larger by -d / c.
__device__ __forceinline__ void rebase(RowSum &r, float m, float c) {
  if (r.m > -INFINITY) {
    const float d = (r.m - m) * c, f = ex2_approx(d);
    r.a = f > 0.0f ? f * (r.a + d * r.s) : 0.0f;
    r.s *= f;
  }
  r.m = m;
}

__device__ __forceinline__ RowSum merge(RowSum x, RowSum y, float c) {
  const float m = fmaxf(x.m, y.m);
  rebase(x, m, c);
  rebase(y, m, c);
  return RowSum{m, x.s + y.s, x.a + y.a};
}

// Order-preserving bits of a value; NaN counts as -inf, -0 as 0.  0 is below all.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = v != v ? 0xff800000u : __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t b) {
  return __uint_as_float((b & 0x80000000u) ? b & 0x7fffffffu : ~b);
}

template <typename K>
__device__ __forceinline__ K larger(K a, K b) { return a > b ? a : b; }
template <typename K>
__device__ __forceinline__ K smaller(K a, K b) { return a < b ? a : b; }

// The 32 largest of two descending lists, one entry a lane, descending.
template <typename K>
__device__ __forceinline__ K merge_lists(K x, K y) {
  const int lane = threadIdx.x & 31;
  x = larger(x, __shfl_sync(0xffffffffu, y, 31 - lane));  // bitonic
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const K z = __shfl_xor_sync(0xffffffffu, x, o);
    x = (lane & o) ? smaller(x, z) : larger(x, z);
  }
  return x;
}

// 32 entries, one a lane, into descending order.
template <typename K>
__device__ __forceinline__ K sort_lanes(K x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
    for (int o = n >> 1; o; o >>= 1) {
      const K z = __shfl_xor_sync(0xffffffffu, x, o);
      const bool first = !(lane & o), down = !(lane & n);
      x = (first == down) ? larger(x, z) : smaller(x, z);
    }
  return x;
}

// The block's warps' lists (one per warp, kLpWarps of them) joined in shared
// memory, pairwise; list[0] holds the result after the call.
template <typename K>
__device__ __forceinline__ void join_lists(K (*list)[32], K mine) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  list[warp][lane] = mine;
#pragma unroll
  for (int n = kLpWarps / 2; n; n >>= 1) {
    __syncthreads();
    if (warp < n) {
      mine = merge_lists(mine, list[warp + n][lane]);
      list[warp][lane] = mine;
    }
  }
  __syncthreads();
}

// Elements of a thread's batch, held as loaded.
template <typename T>
struct Batch;
template <>
struct Batch<float> {
  static constexpr int E = 4;  // elements of a vector
  uint4 r[kVecs];
  __device__ __forceinline__ float at(int j) const { return __uint_as_float((&r[j >> 2].x)[j & 3]); }
  __device__ __forceinline__ float max() const {
    float m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = at(j);
#pragma unroll
    for (int j = 4; j < 4 * kVecs; ++j) m[j & 3] = fmaxf(m[j & 3], at(j));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
  }
  static __device__ __forceinline__ uint32_t absent() { return 0xff800000u; }
};
template <>
struct Batch<bf16> {
  static constexpr int E = 8;
  uint4 r[kVecs];
  __device__ __forceinline__ float at(int j) const {
    const uint32_t w = (&r[j >> 3].x)[(j >> 1) & 3];
    return __uint_as_float((j & 1) ? w & 0xffff0000u : w << 16);
  }
  __device__ __forceinline__ float max() const {
    __nv_bfloat162 m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = *(const __nv_bfloat162 *)(&r[0].x + j);
#pragma unroll
    for (int j = 4; j < 4 * kVecs; ++j) m[j & 3] = __hmax2(m[j & 3], *(const __nv_bfloat162 *)(&r[j >> 2].x + (j & 3)));
    const __nv_bfloat162 a = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
    return fmaxf(__low2float(a), __high2float(a));
  }
  static __device__ __forceinline__ uint32_t absent() { return 0xff80ff80u; }
};

template <typename T>
__device__ __forceinline__ uint32_t elem_bits(const T *p);
template <>
__device__ __forceinline__ uint32_t elem_bits<float>(const float *p) { return __float_as_uint(*p); }
template <>
__device__ __forceinline__ uint32_t elem_bits<bf16>(const bf16 *p) { return *(const uint16_t *)p; }

struct LpArgs {
  TokenLogprobs a;
  float c;       // log2(e) / tau
  int cluster;   // blocks per row
  int *err;
};

template <typename T>
__global__ void __launch_bounds__(kLpThreads, 2) token_logprobs_kernel(const __grid_constant__ LpArgs p) {
  constexpr int E = Batch<T>::E, N = E * kVecs;
  __shared__ unsigned long long s_top[kLpWarps][32];
  __shared__ uint32_t s_bound[kLpWarps][32];
  __shared__ RowSum s_sum[kLpWarps];
  // every block of the launch sees the same cluster size
  if (p.cluster > 1 && cluster_ctas() != (uint32_t)p.cluster) {
    if (threadIdx.x == 0 && p.err) atomicExch(p.err, kShapeErrorBase + 4);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x / p.cluster, rank = blockIdx.x - row * p.cluster;
  const int V = p.a.V, k = p.a.top_k;
  const T *x = (const T *)p.a.logits + (size_t)row * p.a.row_stride;
  // 16-byte vectors from the boundary at or before the row on; vector j holds
  // the entries j E - lead ..; entries outside the row are not read
  const int lead = (int)(((uintptr_t)x & 15) / sizeof(T));
  const long long n_vec = ((long long)V + lead + E - 1) / E;
  const long long per = (n_vec + p.cluster - 1) / p.cluster;
  const long long v_begin = per * rank, v_end = min(n_vec, v_begin + per);
  auto load = [&](Batch<T> &b, long long v0) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const long long v = v0 + u * kLpThreads + threadIdx.x, i0 = v * E - lead;
      if (v < v_end && i0 >= 0 && i0 + E <= V) {
        b.r[u] = __ldcs((const uint4 *)(x + i0));
      } else {
        uint32_t w[4] = {Batch<T>::absent(), Batch<T>::absent(), Batch<T>::absent(), Batch<T>::absent()};
        if (v < v_end) {
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (i0 + e >= 0 && i0 + e < V) {
              const uint32_t bits = elem_bits(x + i0 + e);
              if (sizeof(T) == 4) w[e & 3] = bits;
              else w[e >> 1] = (e & 1) ? (w[e >> 1] & 0xffffu) | (bits << 16) : (w[e >> 1] & 0xffff0000u) | bits;
            }
        }
        b.r[u] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  };

  RowSum r{-INFINITY, 0.0f, 0.0f};
  unsigned long long best = 0, kth = 0;  // the warp's list; its k-th entry
  uint32_t bound = 0;                    // entries below it are not among the block's k best
  Batch<T> cur, nxt;
  constexpr long long kStep = (long long)kLpThreads * kVecs;
  long long refresh = v_begin + kStep;  // the batch after which the bound is renewed
  load(cur, v_begin);
  for (long long v0 = v_begin; v0 < v_end; v0 += kStep) {
    if (v0 + kStep < v_end) load(nxt, v0 + kStep);
    const float mb = cur.max();
    if (mb > r.m) rebase(r, mb, p.c);
    const float m = r.m > -INFINITY ? r.m : 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float d = (cur.at(j) - m) * p.c, e = ex2_approx(d);
      r.s += e;  // NaN here marks the row
      r.a += e * fmaxf(d, -1000.0f);
    }
    if (k) {
      const uint32_t ob = order_bits(mb);
      if (v0 == v_begin) {  // the block's bound; a thread without entries has none
        join_lists(s_bound, sort_lanes(v0 + threadIdx.x < v_end ? ob : 0u));
        bound = s_bound[0][k - 1];
      }
      // later batches hold higher indices, so an equal value does not enter a full list
      if (__any_sync(0xffffffffu, ob >= bound && (ob > (uint32_t)(kth >> 32) || kth == 0))) {
        // the lane's candidates (NaN among them: the exact test drops it)
        const uint32_t low = larger(bound, (uint32_t)(kth >> 32));
        const float lim = low ? order_value(low) : -INFINITY;
        uint32_t mask = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) mask |= cur.at(j) < lim ? 0u : 1u << j;
        while (__any_sync(0xffffffffu, mask != 0)) {
          const int j = __ffs(mask) - 1;
          float v = 0.0f;
#pragma unroll
          for (int q = 0; q < N; ++q)
            if (q == j) v = cur.at(q);
          const long long at_v = v0 + (j / E) * kLpThreads + threadIdx.x, i = at_v * E - lead + j % E;
          const uint32_t o = order_bits(v);
          const unsigned long long key = ((unsigned long long)o << 32) | (uint32_t)~(uint32_t)i;
          unsigned todo = __ballot_sync(0xffffffffu, mask && at_v < v_end && i >= 0 && i < V && o >= bound && key > kth);
          mask &= mask - 1;
          while (todo) {
            const unsigned long long n = __shfl_sync(0xffffffffu, key, __ffs(todo) - 1);
            const int at = __popc(__ballot_sync(0xffffffffu, best > n));  // entries before it
            const unsigned long long up = __shfl_up_sync(0xffffffffu, best, 1);
            if (lane == at) best = n;
            else if (lane > at) best = up;
            kth = __shfl_sync(0xffffffffu, best, k - 1);
            todo &= todo - 1;
            todo &= __ballot_sync(0xffffffffu, key > kth);
          }
        }
      }
      // after 2, 4, 8 ... batches: the k-th entry of all the block's lists so far
      if (v0 == refresh) {
        refresh = v_begin + 2 * (refresh + kStep - v_begin) - kStep;
        if (v0 + kStep < v_end) {
          join_lists(s_bound, (uint32_t)(best >> 32));
          bound = larger(bound, s_bound[0][k - 1]);
        }
      }
    }
    cur = nxt;
  }

  // ---- the block's state, then the row's ------------------------------------------
  for (int o = 16; o; o >>= 1) {
    RowSum q;
    q.m = __shfl_xor_sync(0xffffffffu, r.m, o);
    q.s = __shfl_xor_sync(0xffffffffu, r.s, o);
    q.a = __shfl_xor_sync(0xffffffffu, r.a, o);
    r = merge(r, q, p.c);
  }
  if (lane == 0) s_sum[warp] = r;
  if (k) join_lists(s_top, best);
  else __syncthreads();
  if (warp == 0) {
    r = s_sum[0];
    for (int w = 1; w < kLpWarps; ++w) r = merge(r, s_sum[w], p.c);
  }
  if (p.cluster > 1) {
    __syncthreads();
    if (threadIdx.x == 0) s_sum[0] = r;
    __syncwarp();
    tc::cluster_sync();
    if (rank == 0) {  // warp w takes block w's state
      RowSum q{-INFINITY, 0.0f, 0.0f};
      unsigned long long l = 0;
      if (warp < p.cluster) {
        const uint32_t at = tc::cluster_addr(tc::smem_u32(&s_sum[0]), (uint32_t)warp);
        asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(q.m) : "r"(at) : "memory");
        asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(q.s) : "r"(at + 4) : "memory");
        asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(q.a) : "r"(at + 8) : "memory");
        asm volatile("ld.shared::cluster.u64 %0, [%1];\n"
                     : "=l"(l)
                     : "r"(tc::cluster_addr(tc::smem_u32(&s_top[0][lane]), (uint32_t)warp))
                     : "memory");
      }
      __syncthreads();  // this block's own state is read before it is overwritten
      if (lane == 0) s_sum[warp] = q;
      if (k) join_lists(s_top, l);
      else __syncthreads();
      if (warp == 0) {
        r = s_sum[0];
        for (int w = 1; w < p.cluster; ++w) r = merge(r, s_sum[w], p.c);
      }
    }
    __syncwarp();
    tc::cluster_sync();  // the peers' states have been read
  }
  if (rank != 0 || warp != 0) return;
  const float nan = __int_as_float(0x7fc00000);
  const float top = r.m * p.a.inv_tau;
  const bool bad = !(r.s >= 0.0f) || top == INFINITY;  // a NaN entry, or +inf
  const float logs = bad ? nan : (r.s > 0.0f ? logf(r.s) : 0.0f);
  auto logprob = [&](float raw) {
    if (bad) return nan;
    return raw == -INFINITY ? raw : (raw * p.a.inv_tau - top) - logs;
  };
  if (lane == 0) {
    if (p.a.lse) p.a.lse[row] = top + logs;
    if (p.a.entropy) p.a.entropy[row] = bad ? nan : (r.s > 0.0f ? logs - kLn2f * (r.a / r.s) : 0.0f);
  }
  if (lane < k) {
    const unsigned long long key = s_top[0][lane];
    p.a.top_ids[(size_t)row * k + lane] = (int)~(uint32_t)key;
    if (p.a.top_logprobs) p.a.top_logprobs[(size_t)row * k + lane] = logprob(order_value((uint32_t)(key >> 32)));
  }
  for (int j = lane; j < p.a.n_given; j += 32) {
    const size_t at = (size_t)row * p.a.n_given + j;
    const int id = p.a.tokens[at];
    float lp = 0.0f;  // -1: no token here
    if (id >= 0 && id < V) {
      const uint32_t b = elem_bits(x + id);
      lp = logprob(__uint_as_float(sizeof(T) == 4 ? b : b << 16));
    } else if (id != -1) {
      lp = nan;
      if (p.err) atomicExch(p.err + 1, kBadToken);
    }
    p.a.logprobs[at] = lp;
  }
}

template <typename T>
cudaError_t launch(const LpArgs &p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.a.rows * p.cluster);
  cfg.blockDim = dim3(kLpThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  if (p.cluster > 1) {
    if (p.cluster > 8) {
      static unsigned long long attr_set = 0;
      int dev = 0;
      cudaError_t e = cudaGetDevice(&dev);
      if (e != cudaSuccess) return e;
      if (dev >= 64 || !((attr_set >> dev) & 1ull)) {
        e = cudaFuncSetAttribute(token_logprobs_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_set |= 1ull << dev;
      }
    }
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T>, p);
}

}  // namespace

cudaError_t token_logprobs(const TokenLogprobs &a, int *err, cudaStream_t st) {
  if (a.rows == 0) return cudaSuccess;
  LpArgs p;
  p.a = a;
  p.c = (float)(1.4426950408889634 * (double)a.inv_tau);
  p.err = err;
  // blocks per row: two for every SM in all, no fewer than 8192 entries each
  int c = 1;
  while (c < kMaxLpCluster && (long long)a.rows * c * 2 <= 2 * 152 && a.V / (2 * c) >= 8192) c *= 2;
  p.cluster = c;
  return a.is_bf16 ? launch<bf16>(p, st) : launch<float>(p, st);
}

}  // namespace dg
