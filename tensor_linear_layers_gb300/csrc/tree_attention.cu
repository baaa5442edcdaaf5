// Attention of a tree of drafted tokens over the paged KV cache.
//
// Request b has ctx cached tokens and n drafted ones at cache positions ctx ..
// ctx + n - 1, in draft order. Drafted token i sees the positions 0 .. ctx - 1
// and ctx + j for every bit j of its mask:
//   o_i = sum_k p_k v_k / sum_k p_k,  p_k = exp((q_i . k_k - m_i) / sqrt(hd))
// over the keys k it sees; a token that sees nothing gets 0.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gemm_tc.cuh"
#include "internal.h"

namespace tpl {

namespace {
constexpr int kHd = 128;
constexpr int kStatusShape = -2;   // TP_ERR_SHAPE
constexpr int kMaxDraft = 256;     // TP_TREE_MAX_DRAFT
}  // namespace

// One CTA per request, a thread per drafted token: it walks up its ancestors (a parent
// comes before its children, so the walk ends) and sets a bit for each and for itself.
__global__ void __launch_bounds__(kMaxDraft)
    tree_mask_kernel(int T, int max_query_len, int words, const int* __restrict__ parents, const int* __restrict__ qsl,
                     const int* __restrict__ seq_lens, int* __restrict__ mask, int* __restrict__ positions,
                     int* __restrict__ status) {
  __shared__ int par[kMaxDraft];
  const int b = blockIdx.x, i = threadIdx.x;
  const int q0 = qsl[b], n = qsl[b + 1] - q0, ctx = seq_lens[b] - n;
  if (q0 < 0 || n < 0 || n > max_query_len || q0 > T - n || ctx < 0) {
    if (i == 0) atomicExch(status, kStatusShape);
    return;
  }
  if (i < n) par[i] = parents[q0 + i];
  __syncthreads();
  if (i >= n) return;
  unsigned bits[kMaxDraft / 32];
#pragma unroll
  for (int w = 0; w < kMaxDraft / 32; ++w) bits[w] = 0u;
  int at = i, depth = -1;
  bool ok = true;
  while (at >= 0) {
#pragma unroll
    for (int w = 0; w < kMaxDraft / 32; ++w)
      if (w == at >> 5) bits[w] |= 1u << (at & 31);
    const int up = par[at];
    if (up < -1 || up >= at) {
      ok = false;
      break;
    }
    at = up;
    ++depth;
  }
  if (!ok) atomicExch(status, kStatusShape);
#pragma unroll
  for (int w = 0; w < kMaxDraft / 32; ++w)
    if (w < words) mask[(size_t)(q0 + i) * words + w] = ok ? (int)bits[w] : 0;
  if (positions != nullptr) positions[q0 + i] = ok ? ctx + depth : -1;
}

// One warp per (token, shard, q head): a lane holds four head dimensions.
__global__ void __launch_bounds__(128) tree_attn_kernel(const TreeAttnParams p) {
  const int lane = threadIdx.x & 31;
  const long long it = blockIdx.x * 4LL + (threadIdx.x >> 5);
  const int h = (int)(it % p.q_per), r = (int)(it / p.q_per % p.t);
  const long long ti = it / p.q_per / p.t;
  if (ti >= (long long)p.n_reqs * p.max_query_len) return;
  const int b = (int)(ti / p.max_query_len), i = (int)(ti % p.max_query_len);
  const int q0 = p.qsl[b], n = p.qsl[b + 1] - q0, L = p.seq_lens[b], ctx = L - n;
  if (q0 < 0 || n < 0 || n > p.max_query_len || q0 > p.T - n || ctx < 0 || L > p.max_seq_len) {
    if (lane == 0) atomicExch(p.status, kStatusShape);
    return;
  }
  if (i >= n) return;
  const int g = h / (p.q_per / p.kv_per);
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  const __nv_bfloat16* qp = p.qkv + (size_t)r * p.sstride_in + (size_t)(q0 + i) * p.rstride_in + h * kHd + lane * 4;
  for (int e = 0; e < 4; ++e) q[e] = __bfloat162float(qp[e]) * p.scale_log2;
  for (int k = 0; k < L; ++k) {
    if (k >= ctx && !((unsigned)p.mask[(size_t)(q0 + i) * p.mask_words + ((k - ctx) >> 5)] >> ((k - ctx) & 31) & 1u)) continue;
    const int blk = p.block_tables[(size_t)b * p.max_blocks + k / p.block_size];
    if (blk < 0 || blk >= p.num_blocks) {
      if (lane == 0) atomicExch(p.status, kStatusShape);
      continue;
    }
    const size_t row = ((((size_t)r * p.num_blocks + blk) * p.block_size + k % p.block_size) * p.kv_per + g) * kHd + lane * 4;
    float s = 0.f;
    for (int e = 0; e < 4; ++e) s += q[e] * __bfloat162float(p.cache_k[row + e]);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn), w = mn == -INFINITY ? 0.f : exp2f(s - mn);
    l = l * f + w;
    for (int e = 0; e < 4; ++e) o[e] = o[e] * f + w * __bfloat162float(p.cache_v[row + e]);
    m = mn;
  }
  __nv_bfloat16* op = p.out + (size_t)r * p.sstride_out + (size_t)(q0 + i) * p.rstride_out + h * kHd + lane * 4;
  for (int e = 0; e < 4; ++e) op[e] = __float2bfloat16_rn(l == 0.f ? 0.f : o[e] / l);
}

cudaError_t launch_tree_mask(int T, int n_reqs, int max_query_len, int words, const int* parents, const int* qsl,
                             const int* seq_lens, int* mask, int* positions, int* status, cudaStream_t st) {
  const int threads = (max_query_len + 31) / 32 * 32;
  tree_mask_kernel<<<n_reqs, threads, 0, st>>>(T, max_query_len, words, parents, qsl, seq_lens, mask, positions, status);
  return cudaGetLastError();
}

cudaError_t launch_tree_attention(const TreeAttnParams& p, cudaStream_t st) {
  const long long items = (long long)p.n_reqs * p.max_query_len * p.t * p.q_per;
  tree_attn_kernel<<<(unsigned)((items + 3) / 4), 128, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace tpl
