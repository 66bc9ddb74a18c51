// Log probabilities of given tokens under rows of logits, with each row's
// entropy and its most likely tokens.  With y = logit / tau, m = max y,
// S = sum e^(y - m), A = sum e^(y - m) (y - m):
//   log p(v) = (y_v - m) - log S,  lse = m + log S,  entropy = log S - A / S.
//
// Bound by the logits' bytes, each read once: 1024 rows of 262144 fp32 take 162 us,
// 6.6 TB/s.  (It was 186 us with per-vector checks and every distance clamped: the
// instructions of an entry, not loads in flight; batches on their way through
// shared memory, more of them, were slower.)  A row is split over the blocks of a
// cluster when there are few rows, and their states joined through distributed
// shared memory (one launch, no workspace).  A thread takes a batch of kVecs
// 16-byte vectors at a time, the next batch already in flight, and moves its
// running maximum once per batch; sums are kept in units of log2, fp32.
//
// The most likely tokens: each warp keeps a list of its 32 best entries, one a
// lane, in descending order of a 64-bit key (order-preserving bits of the
// value, then the complement of the index: equal values go to the lower
// index).  A list starts empty, so nearly every entry of a warp's first
// batches would enter it.  The k-th largest of the running maxima of 64 groups
// of threads is a lower bound of the block's k-th best entry, close to it (the
// groups' maxima are mostly the best entries themselves), and cheap: entries
// below are dropped at one compare per batch, with the bound renewed after 1, 4,
// 16 ... batches (after 1, 2, 4, 8 ..., 1024 rows of 262144 take 166 us; after 1, 8,
// 64 ..., 301 rows of 50001 with k = 32 take 23.6 us instead of 17.7), and about
// k + 1.5 k log2(batches) of a block's random logits reach a list.  At the end the
// lists' entries above the bound, at most a few times k, are gathered and each
// finds its place by counting the larger ones.
#include <atomic>
#include <type_traits>

#include "f32x2.cuh"
#include "gemm_tc.cuh"
#include "internal.h"

namespace dg {

namespace {

constexpr int kLpThreads = 512, kLpWarps = kLpThreads / 32;
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

// Order-preserving bits of a value; NaN counts as -inf, -0 as 0.  0 is below all.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = v != v ? 0xff800000u : __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t b) {
  return __uint_as_float((b & 0x80000000u) ? b & 0x7fffffffu : ~b);
}

constexpr int kGroups = 64;  // no fewer than the largest k

// The k-th largest of the maxima of up to 64 groups of threads, from each thread's
// (order bits; 0: none); run by the whole block, on two buffers in turn.  Groups
// are of 2^lg <= 8 threads.  Eight threads count the larger ones of a group (ties
// in group order), an eighth each.
struct __align__(16) GroupMax {
  uint32_t max[kGroups], bound;
};
__device__ __forceinline__ uint32_t group_bound(uint32_t mine, int k, int lg, GroupMax *s) {
  const int group = threadIdx.x >> 3, part = threadIdx.x & 7;
  if (lg == 3) {
#pragma unroll
    for (int o = 4; o; o >>= 1) mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, o));
    if (part == 0) s->max[group] = mine;
    __syncthreads();
  } else {
    for (int o = (1 << lg) >> 1; o; o >>= 1) mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, o));
    if ((threadIdx.x & ((1 << lg) - 1)) == 0 && threadIdx.x < kGroups << lg) s->max[threadIdx.x >> lg] = mine;
    __syncthreads();
    mine = s->max[group];
  }
  const uint4 v = *(const uint4 *)(s->max + 8 * part), w = *(const uint4 *)(s->max + 8 * part + 4);
  const uint32_t m[8] = {v.x, v.y, v.z, v.w, w.x, w.y, w.z, w.w};
  const int before = group - 8 * part;  // entries of this eighth that lie before the group
  int above = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) above += m[e] > mine || (m[e] == mine && e < before);
#pragma unroll
  for (int o = 4; o; o >>= 1) above += __shfl_xor_sync(0xffffffffu, above, o);
  if (part == 0 && above == k - 1) s->bound = mine;
  __syncthreads();
  return s->bound;
}

// Entries collected in shared memory, and the k best of them in order.
struct Picks {
  int n;
  unsigned long long key[kLpThreads];
  unsigned long long top[32];
};
__device__ __forceinline__ void collect(Picks *s, unsigned long long key, bool in) {
  const int lane = threadIdx.x & 31;
  const unsigned m = __ballot_sync(0xffffffffu, in);
  int at = 0;
  if (lane == 0 && m) at = atomicAdd(&s->n, __popc(m));
  at = __shfl_sync(0xffffffffu, at, 0) + __popc(m & ((1u << lane) - 1));
  if (in) s->key[at] = key;
}
// After a barrier: entry t finds its place; top[] is complete after the next one.
__device__ __forceinline__ void place(Picks *s, int k) {
  const int n = s->n, t = threadIdx.x;
  if (t >= n) return;
  const unsigned long long mine = s->key[t];
  int above = 0;
  for (int q = 0; q < n; ++q) above += s->key[q] > mine;
  if (above < k) s->top[above] = mine;
}

// Largest of the lanes' raw logits (NaN not among them).
__device__ __forceinline__ float lanes_max(float m) {
  return order_value(__reduce_max_sync(0xffffffffu, order_bits(m)));
}
// The lanes' sums, of `n` lanes each (a power of two), moved to maximum m and added.
__device__ __forceinline__ void lanes_sum(RowSum &r, float m, float c, int n) {
  rebase(r, m, c);
  for (int o = n / 2; o; o >>= 1) {
    r.s += __shfl_xor_sync(0xffffffffu, r.s, o);
    r.a += __shfl_xor_sync(0xffffffffu, r.a, o);
  }
}

// Elements of a thread's batch, held as loaded.
template <typename T>
struct Batch;
template <>
struct Batch<float> {
  static constexpr int E = 4, kVecs = 4;  // elements of a vector, vectors of a batch
  uint4 r[kVecs];
  __device__ __forceinline__ float at(int j) const { return __uint_as_float((&r[j >> 2].x)[j & 3]); }
  __device__ __forceinline__ float max() const {
    float m[2] = {at(0), at(1)};
#pragma unroll
    for (int j = 2; j < 4 * kVecs - 2; j += 4) {
      m[0] = fmaxf(fmaxf(m[0], at(j)), at(j + 1));
      m[1] = fmaxf(fmaxf(m[1], at(j + 2)), at(j + 3));
    }
    return fmaxf(fmaxf(fmaxf(m[0], m[1]), at(4 * kVecs - 2)), at(4 * kVecs - 1));
  }
  static __device__ __forceinline__ uint32_t absent() { return 0xff800000u; }
};
template <>
struct Batch<bf16> {
  static constexpr int E = 8, kVecs = 2;  // more spill: 301 rows of 50001 took 14.4 us with 2, 19.0 with 4
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

// One of 16 values by halving.
template <class F>
__device__ __forceinline__ float pick16(int j, F at) {
  float a[8], b[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = (j & 8) ? at(8 + i) : at(i);
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = (j & 4) ? a[4 + i] : a[i];
  const float c = (j & 2) ? b[2] : b[0], d = (j & 2) ? b[3] : b[1];
  return (j & 1) ? d : c;
}

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
  static_assert(Batch<T>::E * Batch<T>::kVecs == 16, "pick16");
  constexpr int E = Batch<T>::E, kVecs = Batch<T>::kVecs, N = E * kVecs;
  __shared__ Picks s_pick;
  __shared__ __align__(16) GroupMax s_max[2];
  __shared__ RowSum s_sum[kLpWarps], s_part[kMaxLpCluster];
  __shared__ float s_wmax[kLpWarps];
  __shared__ unsigned long long s_list[kMaxLpCluster][32];  // the blocks' best entries, pushed into the first one's
  // every block of the launch sees the same cluster size
  if (p.cluster > 1 && cluster_ctas() != (uint32_t)p.cluster) {
    if (threadIdx.x == 0 && p.err) atomicExch(p.err, kShapeErrorBase + 4);
    return;
  }
  // (the peers are running once all have arrived: waited for before the exchange)
  if (p.cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x / p.cluster, rank = blockIdx.x - row * p.cluster;
  const int V = p.a.V, k = p.a.top_k;
  const T *x = (const T *)p.a.logits + (size_t)row * p.a.row_stride;
  // 16-byte vectors from the boundary at or before the row on; vector j holds
  // the entries j E - lead ..; entries outside the row are not read
  const uint32_t lead = (uint32_t)(((uintptr_t)x & 15) / sizeof(T));
  const uint32_t n_vec = ((uint32_t)V + lead + E - 1) / E;  // V < 2^31: an entry's index fits 32 bits, a batch past the end too
  const uint32_t per = (n_vec + p.cluster - 1) / p.cluster;
  const uint32_t v_begin = min(n_vec, per * rank), v_end = min(n_vec, v_begin + per);
  if (threadIdx.x == 0) s_pick.n = 0;
  constexpr uint32_t kStep = (uint32_t)kLpThreads * kVecs;
  auto load = [&](Batch<T> &b, uint32_t v0) {
    const uint32_t v1 = v0 + threadIdx.x;
    if (v0 * E >= lead && v0 + kStep <= v_end && (v0 + kStep) * E - lead <= (uint32_t)V) {  // all of the batch lies in the row
      const uint4 *at = (const uint4 *)(x + (v1 * E - lead));
#pragma unroll
      for (int u = 0; u < kVecs; ++u) b.r[u] = __ldcs(at + u * kLpThreads);
      return;
    }
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const uint32_t v = v1 + u * kLpThreads;
      if (v < v_end && v * E >= lead && v * E - lead + E <= (uint32_t)V) {
        b.r[u] = __ldcs((const uint4 *)(x + (v * E - lead)));
      } else {
        uint32_t w[4] = {Batch<T>::absent(), Batch<T>::absent(), Batch<T>::absent(), Batch<T>::absent()};
        if (v < v_end) {
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (v * E + e >= lead && v * E + e - lead < (uint32_t)V) {
              const uint32_t bits = elem_bits(x + (v * E + e - lead));
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
  float bound_v = -INFINITY, kth_v = -INFINITY;  // both as values
  bool masked = false;                   // the warp has met entries of -inf
  Batch<T> cur, nxt;
  uint32_t renew = v_begin;              // the batch with which the bound is renewed
  // groups of as few threads as make 64 of those that have entries: a short row's
  // bound would else be loose (1024 entries of bf16, k = 32: 20.1 -> 7.3 us)
  const int lg = v_end - v_begin > 4 * kGroups ? 3 : v_end - v_begin > 2 * kGroups ? 2 : v_end - v_begin > kGroups ? 1 : 0;
  int turn = 0;
  load(cur, v_begin);
  // the given tokens' logits, early (the first block looks them up at the end)
  int my_id = -1;
  uint32_t my_bits = 0;
  if (rank == 0 && threadIdx.x < p.a.n_given) {
    my_id = p.a.tokens[(size_t)row * p.a.n_given + threadIdx.x];
    if (my_id >= 0 && my_id < V) my_bits = elem_bits(x + my_id);
  }
  for (uint32_t v0 = v_begin; v0 < v_end; v0 += kStep) {
    if (v0 + kStep < v_end) load(nxt, v0 + kStep);
    const float mb = fmaxf(cur.max(), -INFINITY);  // (NaN: none)
    if (mb > r.m) rebase(r, mb, p.c);
    const float m = r.m > -INFINITY ? r.m : 0.0f;
    const f32x2 minus_m = pair(-m, -m), cc = pair(p.c, p.c);
    f32x2 sum, dot;
    // An entry of -inf has weight 0, but 0 times its distance is NaN: once a warp
    // has met one, distances are held above -1000.
    auto add_up = [&](auto low) {
      sum = dot = pair(0.0f, 0.0f);
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        f32x2 d2 = mul2(add2(pair(cur.at(j), cur.at(j + 1)), minus_m), cc);
        const float2 d = split(d2);
        const f32x2 e = pair(ex2_approx(d.x), ex2_approx(d.y));
        if constexpr (decltype(low)::value) d2 = pair(fmaxf(d.x, -1000.0f), fmaxf(d.y, -1000.0f));
        sum = add2(sum, e);  // NaN here marks the row
        dot = fma2(e, d2, dot);
      }
    };
    if (!masked) {
      add_up(std::false_type());
      const float2 t = split(dot);
      masked = __any_sync(0xffffffffu, !(t.x + t.y > -INFINITY));
    }
    if (masked) add_up(std::true_type());
    const float2 sums = split(sum), dots = split(dot);
    r.s += sums.x + sums.y;
    r.a += dots.x + dots.y;
    if (k) {
      if (v0 == renew) {  // after batches 1, 4, 16 ...: from the threads' running maxima
        renew = v_begin + 4 * (renew + kStep - v_begin) - kStep;
        // a thread without entries so far has none (its first vector lies behind the end)
        bound = max(bound, group_bound(v_begin + threadIdx.x < v_end ? order_bits(r.m) : 0u, k, lg, s_max + turn));
        turn ^= 1;
        if (bound) bound_v = order_value(bound);
      }
      // later batches hold higher indices, so an equal value does not enter a full list
      if (__any_sync(0xffffffffu, mb >= bound_v && (mb > kth_v || kth == 0))) {
        // the lane's candidates (NaN among them: the exact test drops it)
        const uint32_t low = max(bound, (uint32_t)(kth >> 32));
        const float lim = low ? order_value(low) : -INFINITY;
        uint32_t mask = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) mask |= cur.at(j) < lim ? 0u : 1u << j;
        while (__any_sync(0xffffffffu, mask != 0)) {
          const int j = 31 - __clz(mask);  // the last first: rows in rising order enter fewer (1024 x 262144: 1.3 ms, else 3.3)
          const float v = pick16(j & 15, [&](int q) { return cur.at(q); });
          const uint32_t at_v = v0 + (j / E) * kLpThreads + threadIdx.x, i = at_v * E + j % E - lead;  // (before the row: past V)
          const uint32_t o = order_bits(v);
          const unsigned long long key = ((unsigned long long)o << 32) | ~i;
          unsigned todo = __ballot_sync(0xffffffffu, mask && at_v < v_end && i < (uint32_t)V && o >= bound && key > kth);
          mask &= ~(1u << (j & 31));
          while (todo) {
            const unsigned long long n = __shfl_sync(0xffffffffu, key, __ffs(todo) - 1);
            const int at = __popc(__ballot_sync(0xffffffffu, best > n));  // entries before it (32: it drops out)
            const unsigned long long up = __shfl_up_sync(0xffffffffu, best, 1);
            if (lane == at) best = n;
            else if (lane > at) best = up;
            todo &= todo - 1;
          }
          kth = __shfl_sync(0xffffffffu, best, k - 1);
        }
        if (kth) kth_v = order_value((uint32_t)(kth >> 32));
      }
    }
    cur = nxt;
  }

  // ---- the block's state, then the row's ------------------------------------------
  const float wm = lanes_max(r.m);
  if (lane == 0) s_wmax[warp] = wm;
  if (k) collect(&s_pick, best, best != 0 && (uint32_t)(best >> 32) >= bound);
  __syncthreads();
  lanes_sum(r, lanes_max(s_wmax[lane & (kLpWarps - 1)]), p.c, 32);
  if (lane == 0) s_sum[warp] = r;
  if (k) place(&s_pick, k);
  __syncthreads();
  r = s_sum[lane & (kLpWarps - 1)];
  lanes_sum(r, r.m, p.c, kLpWarps);  // in every warp
  if (p.cluster > 1) {
    // Every block pushes its sums and entries (0: none) into the first block's
    // shared memory; nothing is read from the others, which end here.
    asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
    if (warp == 0) {
      const unsigned long long key = lane < min(k, s_pick.n) ? s_pick.top[lane] : 0ull;
      asm volatile("st.shared::cluster.u64 [%0], %1;\n" ::"r"(tc::cluster_addr(tc::smem_u32(&s_list[rank][lane]), 0u)), "l"(key)
                   : "memory");
      const float v = lane == 0 ? r.m : lane == 1 ? r.s : r.a;
      if (lane < 3)
        asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(tc::cluster_addr(tc::smem_u32(&s_part[rank]) + 4 * lane, 0u)),
                     "f"(v)
                     : "memory");
    }
    __syncwarp();
    tc::cluster_sync();
    if (rank != 0) return;
    RowSum q{-INFINITY, 0.0f, 0.0f};
    unsigned long long kth_w = 0;  // no entry below some block's k-th is among the row's k best
    if (lane < p.cluster) {
      q = s_part[lane];
      if (k) kth_w = s_list[lane][k - 1];
    }
    r = q;
    lanes_sum(r, lanes_max(q.m), p.c, 32);
    if (k) {
      for (int o = 16; o; o >>= 1) kth_w = max(kth_w, __shfl_xor_sync(0xffffffffu, kth_w, o));
      if (threadIdx.x == 0) s_pick.n = 0;
      __syncthreads();
      const unsigned long long l = warp < p.cluster ? s_list[warp][lane] : 0ull;
      collect(&s_pick, l, l != 0 && l >= kth_w);
      __syncthreads();
      place(&s_pick, k);
      __syncthreads();
    }
  }
  const float nan = __int_as_float(0x7fc00000);
  const float top = r.m * p.a.inv_tau;
  const bool bad = !(r.s >= 0.0f) || top == INFINITY;  // a NaN entry, or +inf
  // every y is -inf: the entries are, or (where their lowest value fills a masked
  // row) their products with 1 / tau
  const bool none = top == -INFINITY;
  const float logs = bad ? nan : (r.s > 0.0f ? logf(r.s) : 0.0f);
  auto logprob = [&](float raw) {
    if (bad) return nan;
    const float y = __fmul_rn(raw, p.a.inv_tau);  // rounded, as top is: not part of the difference
    return y == -INFINITY ? y : (y - top) - logs;
  };
  if (threadIdx.x == 0) {
    if (p.a.lse) p.a.lse[row] = top + logs;
    if (p.a.entropy) p.a.entropy[row] = bad ? nan : none ? 0.0f : logs - kLn2f * (r.a / r.s);
  }
  if (threadIdx.x < k) {
    const unsigned long long key = s_pick.top[threadIdx.x];
    p.a.top_ids[(size_t)row * k + threadIdx.x] = (int)~(uint32_t)key;
    if (p.a.top_logprobs) p.a.top_logprobs[(size_t)row * k + threadIdx.x] = logprob(order_value((uint32_t)(key >> 32)));
  }
  for (int j = threadIdx.x; j < p.a.n_given; j += kLpThreads) {
    if (j >= kLpThreads) {
      my_id = p.a.tokens[(size_t)row * p.a.n_given + j];
      if (my_id >= 0 && my_id < V) my_bits = elem_bits(x + my_id);
    }
    float lp = 0.0f;  // -1: no token here
    if (my_id >= 0 && my_id < V) {
      lp = logprob(__uint_as_float(sizeof(T) == 4 ? my_bits : my_bits << 16));
    } else if (my_id != -1) {
      lp = nan;
      if (p.err) atomicExch(p.err + 1, kBadToken);
    }
    p.a.logprobs[(size_t)row * p.a.n_given + j] = lp;
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
      static std::atomic<unsigned long long> attr_set{0};
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
  // Blocks per row: as many as leave one to an SM, with more than 4096 entries
  // each.  One row of 262144: 20.5, 10.4, 8.2, 6.4 us with 1, 4, 8, 16; 12 rows 21.3,
  // 11.0, 8.7, 8.8; 64 rows of 131072: 15.8, 11.9, 12.3, 15.5 with 1, 2, 4, 8; 100 of
  // 32768: 7.3, 8.4, 10.9 with 1, 2, 4 (large clusters leave SMs without a block); 16
  // of 32768: 5.6 with 4, 7.4 with 8.
  int c = 1;
  while (c < kMaxLpCluster && (long long)a.rows * c * 2 <= 152 && a.V / (2 * c) > 4096) c *= 2;
  p.cluster = c;
  return a.is_bf16 ? launch<bf16>(p, st) : launch<float>(p, st);
}

}  // namespace dg
