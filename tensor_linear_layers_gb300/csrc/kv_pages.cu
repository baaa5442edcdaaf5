// Pages of the paged KV cache moved inside the cache, all layers of a model in
// one launch: whole pages copied (forks, copy on write, defragmentation) and
// the accepted tokens of a drafted tree moved together. Both are copies:
// bit-exact, bound by HBM (every moved byte read once and written once) or, at
// a few pages, by the launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"

namespace tpl {

namespace {
constexpr int kHd = 128;
constexpr int kStatusShape = -2;   // TP_ERR_SHAPE
}  // namespace

// One CTA per (pair, shard) and (layer, k or v): dst page = src page.
__global__ void kv_copy_blocks_kernel(const KvLayers layers, const int2* __restrict__ pairs, long long num_blocks,
                                      long long page_vecs, int t, int* __restrict__ status) {
  const int r = blockIdx.x % t;
  const int2 pr = pairs[blockIdx.x / t];
  if (pr.x < 0) return;                              // padding entry
  if (pr.y < 0 || pr.x >= num_blocks || pr.y >= num_blocks) {
    if (threadIdx.x == 0) atomicExch(status, kStatusShape);
    return;
  }
  const int layer = blockIdx.y >> 1;
  uint4* cache = reinterpret_cast<uint4*>((blockIdx.y & 1) ? layers.v[layer] : layers.k[layer]);
  const uint4* src = cache + ((size_t)r * num_blocks + pr.x) * page_vecs;
  uint4* dst = cache + ((size_t)r * num_blocks + pr.y) * page_vecs;
  for (long long e = threadIdx.x; e < page_vecs; e += blockDim.x) dst[e] = src[e];
}

// One CTA per (request, shard) and (layer, k or v); a thread moves one 16-byte column of
// the accepted tokens' rows, in their order. Accepted indices rise, so in place (one page
// holding both positions) position ctx + j is written only after every token up to j has
// been read, and the tokens after j come from higher positions: no row is lost.
__global__ void kv_compact_kernel(const KvLayers layers, const CompactParams p) {
  const int r = blockIdx.x % p.t, b = blockIdx.x / p.t;
  const int q0 = p.qsl[b], n_new = p.qsl[b + 1] - q0, L = p.seq_lens[b], ctx = L - n_new;
  const bool first = blockIdx.y == 0 && r == 0 && threadIdx.x == 0;
  if (n_new < 0 || ctx < 0 || (L + p.block_size - 1) / p.block_size > p.max_blocks) {
    if (first) {
      atomicExch(p.status, kStatusShape);
      p.new_lens[b] = L;
    }
    return;
  }
  const int layer = blockIdx.y >> 1;
  uint4* cache = reinterpret_cast<uint4*>((blockIdx.y & 1) ? layers.v[layer] : layers.k[layer]);
  const int vec = p.kv_per * kHd / 8;
  const int* src_t = p.src_tables + (size_t)b * p.max_blocks;
  const int* dst_t = p.dst_tables + (size_t)b * p.max_blocks;
  int j = 0;
  for (int prev = -1; j < p.max_accepted; ++j) {
    const int a = p.accepted[(size_t)b * p.max_accepted + j];
    if (a < 0) break;
    const int so = ctx + a, to = ctx + j;
    const bool in = a > prev && a < n_new;
    const int sb = in ? src_t[so / p.block_size] : -1, db = in ? dst_t[to / p.block_size] : -1;
    if (sb < 0 || db < 0 || sb >= p.num_blocks || db >= p.num_blocks) {
      if (threadIdx.x == 0) atomicExch(p.status, kStatusShape);
      break;
    }
    prev = a;
    const long long s = (long long)sb * p.block_size + so % p.block_size, d = (long long)db * p.block_size + to % p.block_size;
    if (s == d) continue;
    for (int c = threadIdx.x; c < vec; c += blockDim.x)
      cache[((size_t)r * p.n_slots + d) * vec + c] = cache[((size_t)r * p.n_slots + s) * vec + c];
  }
  if (first) p.new_lens[b] = ctx + j;
}

cudaError_t launch_kv_copy_blocks(const KvLayers& layers, int n_layers, const int* pairs, int n_pairs,
                                  long long num_blocks, int block_size, int kv_per, int t, int* status,
                                  cudaStream_t st) {
  const dim3 grid((unsigned)((long long)n_pairs * t), (unsigned)(2 * n_layers));
  kv_copy_blocks_kernel<<<grid, 256, 0, st>>>(layers, reinterpret_cast<const int2*>(pairs), num_blocks,
                                              (long long)block_size * kv_per * kHd / 8, t, status);
  return cudaGetLastError();
}

cudaError_t launch_kv_compact(const KvLayers& layers, int n_layers, const CompactParams& p, int n_reqs, cudaStream_t st) {
  const dim3 grid((unsigned)((long long)n_reqs * p.t), (unsigned)(2 * n_layers));
  kv_compact_kernel<<<grid, 64, 0, st>>>(layers, p);
  return cudaGetLastError();
}

}  // namespace tpl
