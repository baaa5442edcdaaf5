// Pages of the paged KV cache moved inside the cache, all layers of a model in
// one launch: whole pages copied (forks, copy on write, defragmentation) and
// the accepted tokens of a drafted tree moved together. Both are copies:
// bit-exact, bound by HBM (every moved byte read once and written once) or, at
// a few pages, by the launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace tpl {

namespace {
constexpr int kHd = 128;
constexpr int kStatusShape = -2;   // TP_ERR_SHAPE
}  // namespace

// One CTA per (pair, shard) and (layer, k or v): dst page = src page, 16 bytes a thread. Bound by
// HBM: 96 pages of 16 tokens, 8 kv heads, 32 layers (403 MB moved) in 61 to 63 us, 0.95 to 0.98
// of the copy bandwidth; four pages 4.2 us, the launch.
__global__ void kv_copy_blocks_kernel(const KvLayers layers, const int2* pairs, long long num_blocks, long long page_vecs,
                                      int t, int* status) {
  griddep_wait();
  griddep_launch_dependents();
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

// A request's rows of all layers, k and v, and shards are one line of 16-byte columns; a CTA
// takes 256 of them, and a thread moves its column of the accepted tokens in their order, four
// or eight rows in flight. The CTA first turns the list into pairs of slots, kept in shared memory.
// (One CTA per request, layer, k or v and shard: 16 to 32 threads with work, and each read the
// list for itself; 64 requests of up to 9 tokens, 32 layers, 64 us, this 17: 74 MB, 0.64 of
// the copy bandwidth, 0.81 after the 3.5 us that one request takes, the launch and four dependent loads.)
// Accepted indices rise, so in place (one page holding both positions) position ctx + j is
// written only after every token up to j has been read, and the tokens after j come from
// higher positions: no row is lost.
constexpr int kCompactThreads = 256;
template <int ROWS>
__global__ void __launch_bounds__(kCompactThreads) kv_compact_kernel(const KvLayers layers, const CompactParams p,
                                                                     int n_layers, int strips) {
  __shared__ int2 move[kCompactThreads];             // slots (from, to) of a strip of the list
  __shared__ int s_stop;
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x / strips, strip = blockIdx.x - b * strips, tid = threadIdx.x;
  // counts of any value are compared in 64 bits: a difference that wrapped would pass for one that fits
  const long long n_drafts = (long long)p.qsl[b + 1] - p.qsl[b];
  const int L = p.seq_lens[b];
  if (n_drafts < 0 || L < n_drafts || L > (long long)p.max_blocks * p.block_size) {
    if (strip == 0 && tid == 0) {
      atomicExch(p.status, kStatusShape);
      p.new_lens[b] = L;
    }
    return;
  }
  const int n_new = (int)n_drafts, ctx = L - n_new;
  // this thread's column: 16 bytes of a (layer, k or v, shard) row
  const int vec = p.kv_per * kHd / 8;
  const long long col = (long long)strip * kCompactThreads + tid, cols = 2LL * n_layers * p.t * vec;
  const bool have = col < cols;
  const int lk = have ? (int)(col / ((long long)p.t * vec)) : 0;
  const int in = have ? (int)(col - (long long)lk * p.t * vec) : 0, r = in / vec, c = in - r * vec;
  uint4* cache = reinterpret_cast<uint4*>((lk & 1) ? layers.v[lk >> 1] : layers.k[lk >> 1]) + (size_t)r * p.n_slots * vec + c;
  const int* acc = p.accepted + (size_t)b * p.max_accepted;
  const int* src_t = p.src_tables + (size_t)b * p.max_blocks;
  const int* dst_t = p.dst_tables + (size_t)b * p.max_blocks;
  int kept = 0;
  for (int j0 = 0; j0 < p.max_accepted; j0 += kCompactThreads) {
    if (tid == 0) s_stop = kCompactThreads;
    __syncthreads();
    const int j = j0 + tid;
    const int a = j < p.max_accepted ? acc[j] : -1;
    bool good = a >= 0, error = false;
    if (good) {
      const int prev = j > 0 ? acc[j - 1] : -1;
      const int from = ctx + a, to = ctx + j;
      error = a <= prev || a >= n_new || a < j;     // rising from 0 on: a >= j, so `to` stays in the table
      if (!error) {
        const int sb = src_t[from / p.block_size], db = dst_t[to / p.block_size];
        error = sb < 0 || db < 0 || sb >= p.num_blocks || db >= p.num_blocks;
        move[tid] = make_int2(sb * p.block_size + from % p.block_size, db * p.block_size + to % p.block_size);
      }
      good = !error;
    }
    if (!good) atomicMin(&s_stop, tid);
    __syncthreads();
    const int n = min(s_stop, p.max_accepted - j0);
    if (error && tid == n && strip == 0) atomicExch(p.status, kStatusShape);   // what ended the list
    if (have) {
      for (int k0 = 0; k0 < n; k0 += ROWS) {
        uint4 v[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k)
          if (k0 + k < n) v[k] = cache[(size_t)move[k0 + k].x * vec];
#pragma unroll
        for (int k = 0; k < ROWS; ++k)
          if (k0 + k < n && move[k0 + k].x != move[k0 + k].y) cache[(size_t)move[k0 + k].y * vec] = v[k];
      }
    }
    kept += n;
    if (n < kCompactThreads) break;
    __syncthreads();
  }
  if (strip == 0 && tid == 0) p.new_lens[b] = ctx + kept;
}

cudaError_t launch_kv_copy_blocks(const KvLayers& layers, int n_layers, const int* pairs, int n_pairs,
                                  long long num_blocks, int block_size, int kv_per, int t, int* status,
                                  cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      programmatic(dim3((unsigned)((long long)n_pairs * t), (unsigned)(2 * n_layers)), 256, 0, st, attr);
  return cudaLaunchKernelEx(&cfg, kv_copy_blocks_kernel, layers, reinterpret_cast<const int2*>(pairs), num_blocks,
                            (long long)block_size * kv_per * kHd / 8, t, status);
}

cudaError_t launch_kv_compact(const KvLayers& layers, int n_layers, const CompactParams& p, int n_reqs, int nsm,
                              cudaStream_t st) {
  const long long cols = 2LL * n_layers * p.t * (p.kv_per * kHd / 8);
  const int strips = (int)((cols + kCompactThreads - 1) / kCompactThreads);
  if ((long long)n_reqs * strips > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = programmatic(dim3((unsigned)((long long)n_reqs * strips)), kCompactThreads, 0, st, attr);
  // Eight rows in flight hide the latency while every block is resident (59 registers: four blocks per
  // SM; 20 requests of 32 layers and up to 9 tokens 6.3 us, with four rows 6.7). Well beyond one wave the
  // other blocks hide it, and four rows leave room for six (24 such requests 7.6 us, with eight rows
  // 8.3; 64: 17.1 and 18.3; 64 of up to 3 tokens 8.3 and 10.3; 64 of up to 32: 46.5 and 45.7).
  const bool many = (long long)n_reqs * strips > 5LL * nsm;
  return cudaLaunchKernelEx(&cfg, many ? kv_compact_kernel<4> : kv_compact_kernel<8>, layers, p, n_layers, strips);
}

}  // namespace tpl
