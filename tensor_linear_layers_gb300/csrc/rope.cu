// Rotary positions of q and k, with an optional RMSNorm of every head in the
// same pass, on the QKV projection's output; k and v may go to their cache
// slots in the same launch.
//
//   x' = x / sqrt(mean(x^2) + eps) * gamma          (per head; q and k apart, each optional)
//   (a, b) -> (a c - b s, b c + a s)                 c, s = cos, sin of position * frequency
// where the pair (a, b) is (x'_i, x'_{i + rd/2}) in the half layout and
// (x'_2i, x'_2i+1) in the interleaved one, i < rd/2; elements from rd on pass.
// fp32 throughout, one rounding to bf16.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"

namespace tpl {

namespace {
constexpr int kStatusShape = -2;   // TP_ERR_SHAPE
constexpr int kWarps = 4;
}  // namespace

// Entry (p, i): the angle p * f_i in 64 bits (its fraction of a turn would be lost in
// 32 bits at far positions), its cosine and sine rounded to fp32. Built once per model.
__global__ void rope_table_kernel(const RopeFreqs f, long long n_pos, int half, float* __restrict__ table) {
  const long long n = n_pos * half;
  for (long long e = blockIdx.x * (long long)blockDim.x + threadIdx.x; e < n; e += (long long)gridDim.x * blockDim.x) {
    const long long p = e / half;
    const int i = (int)(e - p * half);
    double s, c;
    sincos((double)p * f.inv_freq[i], &s, &c);
    table[p * 2 * half + i] = (float)(c * f.scale);
    table[p * 2 * half + half + i] = (float)(s * f.scale);
  }
}

// One warp per (token, shard, head).
__global__ void __launch_bounds__(32 * kWarps) qk_norm_rope_kernel(const RopeParams p) {
  __shared__ float xs[kWarps][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = p.q_per + 2 * p.kv_per;
  const long long items = (long long)p.T * p.t * heads;
  const int hd = p.hd, half = p.rd / 2;
  float* x = xs[warp];
  for (long long it = blockIdx.x * (long long)kWarps + warp; it < items; it += (long long)gridDim.x * kWarps) {
    const int h = (int)(it % heads);
    const int r = (int)(it / heads % p.t);
    const int i = (int)(it / heads / p.t);
    const long long pos = p.pos[i];
    if (pos < 0) continue;                           // padding token: nothing is written for it
    if (pos >= p.n_pos) {
      if (lane == 0) atomicExch(p.status, kStatusShape);
      continue;
    }
    const size_t at = (size_t)r * p.sstride + (size_t)i * p.rstride + (size_t)h * hd;
    __nv_bfloat16* cache = nullptr;
    if (p.slots != nullptr && h >= p.q_per) {
      const long long s = p.slots[i];
      const bool v = h >= p.q_per + p.kv_per;
      if (s >= p.n_slots) {
        if (lane == 0) atomicExch(p.status, kStatusShape);
      } else if (s >= 0) {
        cache = (v ? p.cache_v : p.cache_k) + (((size_t)r * p.n_slots + s) * p.kv_per + (h - p.q_per) % p.kv_per) * hd;
      }
    }
    const bool is_v = h >= p.q_per + p.kv_per;
    const __nv_bfloat16* gamma = is_v ? nullptr : h < p.q_per ? p.q_gamma : p.k_gamma;
    float ss = 0.f;
    for (int e = lane; e < hd; e += 32) {
      x[e] = __bfloat162float(p.in[at + e]);
      ss += x[e] * x[e];
    }
    if (gamma != nullptr) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float rs = 1.0f / sqrtf(ss / hd + p.eps);
      for (int e = lane; e < hd; e += 32) x[e] *= rs * __bfloat162float(gamma[e]);
    }
    __syncwarp();
    const float* tab = p.table + pos * p.rd;
    for (int e = lane; e < hd; e += 32) {
      float y = x[e];
      if (!is_v && e < p.rd) {
        const int j = p.interleaved ? e >> 1 : e < half ? e : e - half;
        const bool first = p.interleaved ? (e & 1) == 0 : e < half;
        const float other = x[p.interleaved ? e ^ 1 : first ? e + half : e - half];
        const float c = tab[j], s = tab[half + j];
        y = first ? y * c - other * s : y * c + other * s;
      }
      const __nv_bfloat16 b = __float2bfloat16_rn(y);
      p.out[at + e] = b;
      if (cache != nullptr) cache[e] = b;
    }
    __syncwarp();
  }
}

cudaError_t launch_rope_table(const RopeFreqs& f, long long n_pos, int rotary_dim, float* table, int nsm, cudaStream_t st) {
  const long long n = n_pos * (rotary_dim / 2);
  const int grid = (int)std::min<long long>((n + 255) / 256, 16LL * nsm);
  rope_table_kernel<<<grid, 256, 0, st>>>(f, n_pos, rotary_dim / 2, table);
  return cudaGetLastError();
}

cudaError_t launch_qk_norm_rope(const RopeParams& p, int nsm, cudaStream_t st) {
  const long long items = (long long)p.T * p.t * (p.q_per + 2 * p.kv_per);
  const int grid = (int)std::min<long long>((items + kWarps - 1) / kWarps, 16LL * nsm);
  qk_norm_rope_kernel<<<grid, 32 * kWarps, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace tpl
