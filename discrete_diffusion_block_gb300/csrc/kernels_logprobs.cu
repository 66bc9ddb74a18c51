// Log probabilities of given tokens under rows of logits, with each row's
// entropy and its most likely tokens.  With y = logit / tau, m = max y,
// S = sum e^(y - m), A = sum e^(y - m) (y - m):
//   log p(v) = (y_v - m) - log S,  lse = m + log S,  entropy = log S - A / S.
//
// One block per row; the row is read once.  Each thread keeps a running
// (m, S, A) of its entries and each warp a list of its 32 best entries, one a
// lane, in descending order: an entry enters it when it beats the list's last.
// Entries are ordered by a 64-bit key (order-preserving bits of the value,
// then the complement of the index), so equal values go to the lower index.
#include "internal.h"

namespace dg {

namespace {

constexpr int kLpThreads = 256;

struct RowSum {
  float m, s, a;
};

__device__ __forceinline__ RowSum merge(const RowSum &x, const RowSum &y) {
  RowSum o;
  o.m = fmaxf(x.m, y.m);
  if (o.m == -INFINITY) return RowSum{-INFINITY, 0.0f, 0.0f};
  const float dx = x.m - o.m, dy = y.m - o.m;
  const float ex = x.m == -INFINITY ? 0.0f : expf(dx), ey = y.m == -INFINITY ? 0.0f : expf(dy);
  o.s = x.s * ex + y.s * ey;
  o.a = (ex > 0.0f ? ex * (x.a + dx * x.s) : 0.0f) + (ey > 0.0f ? ey * (y.a + dy * y.s) : 0.0f);
  return o;
}

__device__ __forceinline__ unsigned long long order_key(float v, int i) {
  uint32_t b = __float_as_uint(v + 0.0f);  // -0 counts as 0
  if (v != v) b = 0xff800000u;              // NaN orders as -inf
  b = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return ((unsigned long long)b << 32) | (uint32_t)~i;
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t b = (uint32_t)(k >> 32);
  return __uint_as_float((b & 0x80000000u) ? b & 0x7fffffffu : ~b);
}

// The 32 best of two descending lists, one entry a lane, descending.
__device__ __forceinline__ unsigned long long merge_lists(unsigned long long x, unsigned long long y) {
  const int lane = threadIdx.x & 31;
  const unsigned long long r = __shfl_sync(0xffffffffu, y, 31 - lane);
  x = x > r ? x : r;  // bitonic: the 32 best
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const unsigned long long z = __shfl_xor_sync(0xffffffffu, x, o);
    x = (lane & o) ? (x < z ? x : z) : (x > z ? x : z);
  }
  return x;
}

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const bf16 *p) { return __bfloat162float(*p); }

template <typename T>
__global__ void __launch_bounds__(kLpThreads) token_logprobs_kernel(const TokenLogprobs p, int *err) {
  __shared__ RowSum s_sum[kLpThreads / 32];
  __shared__ unsigned long long s_top[kLpThreads / 32][32];
  __shared__ int s_bad;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = blockIdx.x;
  const T *x = (const T *)p.logits + row * p.row_stride;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  RowSum r{-INFINITY, 0.0f, 0.0f};
  unsigned long long best = 0;
  bool bad = false;
  for (int base = warp * 32; base < p.V; base += kLpThreads) {
    const int v = base + lane;
    const bool in = v < p.V;
    const float raw = in ? load1(x + v) : -INFINITY;
    const float y = raw * p.inv_tau;
    bad |= !(y < INFINITY);
    if (y > -INFINITY) r = merge(r, RowSum{y, 1.0f, 0.0f});
    if (p.top_k) {
      unsigned long long k = in ? order_key(raw, v) : 0;
      unsigned todo = __ballot_sync(0xffffffffu, k > __shfl_sync(0xffffffffu, best, 31));
      while (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const unsigned long long n = __shfl_sync(0xffffffffu, k, src);
        const int at = __popc(__ballot_sync(0xffffffffu, best > n));  // entries before it
        const unsigned long long up = __shfl_up_sync(0xffffffffu, best, 1);
        if (lane == at) best = n;
        else if (lane > at) best = up;
      }
    }
  }
  if (bad) s_bad = 1;
  for (int o = 16; o; o >>= 1) {
    RowSum q;
    q.m = __shfl_xor_sync(0xffffffffu, r.m, o);
    q.s = __shfl_xor_sync(0xffffffffu, r.s, o);
    q.a = __shfl_xor_sync(0xffffffffu, r.a, o);
    r = merge(r, q);
  }
  if (lane == 0) s_sum[warp] = r;
  s_top[warp][lane] = best;
  __syncthreads();
  if (warp != 0) return;
  r = s_sum[0];
  for (int w = 1; w < kLpThreads / 32; ++w) {
    r = merge(r, s_sum[w]);
    best = merge_lists(best, s_top[w][lane]);
  }
  const float nan = __int_as_float(0x7fc00000);
  const float logs = s_bad ? nan : (r.s > 0.0f ? logf(r.s) : 0.0f);
  auto logprob = [&](float raw) {
    if (s_bad) return nan;
    return raw == -INFINITY ? raw : (raw * p.inv_tau - r.m) - logs;
  };
  if (lane == 0) {
    if (p.lse) p.lse[row] = r.m + logs;
    if (p.entropy) p.entropy[row] = s_bad ? nan : (r.s > 0.0f ? logs - r.a / r.s : 0.0f);
  }
  if (lane < p.top_k) {
    p.top_ids[(long long)row * p.top_k + lane] = (int)~(uint32_t)best;
    if (p.top_logprobs) p.top_logprobs[(long long)row * p.top_k + lane] = logprob(key_value(best));
  }
  for (int j = lane; j < p.n_given; j += 32) {
    const long long at = (long long)row * p.n_given + j;
    const int id = p.tokens[at];
    float lp = 0.0f;  // -1: no token here
    if (id >= 0 && id < p.V) {
      lp = logprob(load1(x + id));
    } else if (id != -1) {
      lp = nan;
      if (err) atomicExch(err + 1, kBadToken);
    }
    p.logprobs[at] = lp;
  }
}

}  // namespace

cudaError_t token_logprobs(const TokenLogprobs &a, int *err, cudaStream_t st) {
  if (a.rows == 0) return cudaSuccess;
  if (a.is_bf16) token_logprobs_kernel<bf16><<<a.rows, kLpThreads, 0, st>>>(a, err);
  else token_logprobs_kernel<float><<<a.rows, kLpThreads, 0, st>>>(a, err);
  return cudaGetLastError();
}

}  // namespace dg
