// Attention of drafted tokens over the paged KV cache, for a batch of uneven
// sequences: token t of sequence b (row offsets[b] + t) sees the sequence's
// prefix_lens[b] cached keys and those drafted keys whose bit is set in its
// mask words (without masks: the drafted keys up to itself).
//   out[t][h] = sum_j p_j v_j,  p = softmax_j(scale q[t][h] . k_j)
// over the keys it sees; a row that sees none is zero.
//
// One warp per (token, query head): lanes along the head dimension, one key
// at a time with a running maximum and sum.
#include "internal.h"

namespace dg {

namespace {

template <int HD>
__global__ void __launch_bounds__(128) tree_attn_kernel(const TreeAttention p, int *err) {
  constexpr int E = HD / 32;  // elements per lane
  const int lane = threadIdx.x & 31, G = p.Hq / p.Hkv;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t_row = (int)(w / p.Hq), h = (int)(w - (long long)t_row * p.Hq);
  if (t_row >= p.n_tok) return;
  int b = 0;
  for (; b < p.n_seqs; ++b)
    if (t_row >= p.offsets[b] && t_row < p.offsets[b + 1]) break;
  if (b == p.n_seqs) return;
  const int t = t_row - p.offsets[b], n_new = p.offsets[b + 1] - p.offsets[b], pre = p.prefix_lens[b], g = h / G;
  if (pre < 0 || (long long)pre + n_new > (long long)p.max_pages * p.pg) {
    if (lane == 0 && err) atomicExch(err + 1, kBadSequence);
    return;
  }
  float q[E], o[E] = {}, m = -INFINITY, l = 0.0f;
  for (int e = 0; e < E; ++e) q[e] = __bfloat162float(p.q[t_row * p.q_stride + (long long)h * HD + lane * E + e]) * p.scale;
  for (int j = 0; j < pre + n_new; ++j) {
    if (j >= pre) {
      const int d = j - pre;
      const bool sees = p.mask ? d < 64 * p.mask_words && (p.mask[(long long)t_row * p.mask_words + d / 64] >> (d % 64)) & 1 : d <= t;
      if (!sees) continue;
    }
    const int page = p.page_tables[(long long)b * p.max_pages + j / p.pg], s = j % p.pg;
    if (page < 0 || page >= p.n_pages) {
      if (lane == 0 && err) atomicExch(err + 1, kBadPage);
      continue;
    }
    const long long blk = ((long long)page * p.Hkv + g) * p.pg * HD;
    const int f = lane * E;
    const long long at = blk + (long long)(f / 64) * p.pg * 64 + s * 64 + ((((f % 64) / 8) ^ (s & 7)) << 3) + f % 8;
    float x = 0.0f;
    for (int e = 0; e < E; ++e) x += q[e] * __bfloat162float(p.k_pool[at + e]);
    for (int i = 16; i; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
    const float mn = fmaxf(m, x), a = m == -INFINITY ? 0.0f : __expf(m - mn), w = __expf(x - mn);
    l = l * a + w;
    for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * __bfloat162float(p.v_pool[at + e]);
    m = mn;
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  for (int e = 0; e < E; ++e)
    p.out[t_row * p.out_stride + (long long)h * HD + lane * E + e] = __float2bfloat16_rn(o[e] * inv);
}

}  // namespace

size_t tree_attention_workspace_bytes(int, int, int, int, int) { return 0; }

cudaError_t tree_attention(const TreeAttention &a, void *, int *err, cudaStream_t st) {
  if (a.n_tok == 0 || a.n_seqs == 0) return cudaSuccess;
  const long long blocks = ((long long)a.n_tok * a.Hq + 3) / 4;
  if (a.hd == 128) tree_attn_kernel<128><<<(unsigned)blocks, 128, 0, st>>>(a, err);
  else tree_attn_kernel<64><<<(unsigned)blocks, 128, 0, st>>>(a, err);
  return cudaGetLastError();
}

}  // namespace dg
