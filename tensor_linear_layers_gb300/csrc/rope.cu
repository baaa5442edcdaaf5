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
#include "ptx.cuh"

namespace tpl {

namespace {
constexpr int kStatusShape = -2;   // TP_ERR_SHAPE
constexpr int kWarps = 4;
constexpr int kUnroll = 3, kMinCtas = 3;   // loads of a lane in flight; CTAs of the vector kernel per SM

// two bf16 of a word as a pair of fp32, and back (rounded to nearest even)
__device__ __forceinline__ uint64_t unpack2(uint32_t w) {
  return f32x2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(uint64_t v) {
  float a, b;
  f32x2_unpack(v, a, b);
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return reinterpret_cast<const uint32_t&>(r);
}
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

// The general kernel: one warp per (token, shard, head), the head in shared memory. It takes
// the half layout with a rotary_dim that is no multiple of 16, whose pairs do not lie in
// whole 16-byte pieces (4096 tokens of 32 + 16 heads, t = 4: 113 us, where the vector kernel
// below takes 22).
__global__ void __launch_bounds__(32 * kWarps) qk_norm_rope_kernel(const RopeParams p) {
  __shared__ float xs[kWarps][kRopeMaxDim];
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
    const bool is_v = h >= p.q_per + p.kv_per;
    if (p.slots != nullptr && h >= p.q_per) {
      const long long s = p.slots[i];
      if (s >= p.n_slots) {
        if (lane == 0) atomicExch(p.status, kStatusShape);
      } else if (s >= 0) {
        cache = (is_v ? p.cache_v : p.cache_k) + (((size_t)r * p.n_slots + s) * p.kv_per + (h - p.q_per) % p.kv_per) * hd;
      }
    }
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

// The vector kernel. Bound by HBM: every q, k and v element is read once and written once.
// A head is held by G lanes, two 16-byte pieces of 8 elements each, chosen so that both
// elements of every pair are in one lane and no exchange is needed:
//   half layout         pieces l and l + rd/16 for l < rd/16 (pairs 8 l .. 8 l + 7), the
//                       unrotated pieces two by two after them
//   interleaved layout  pieces 2 l and 2 l + 1 (the same pairs 8 l .. 8 l + 7)
// A warp takes up to kUnroll steps of 32 / G heads of ONE token, all loaded at once: a lane's
// cosines and sines serve all of them. Warps are short and many (a token of 48 heads of 128
// is four of them), which fills the SMs evenly; few tokens get a step per warp (latency).
// The arithmetic goes by pairs of fp32 (fma.rn.f32x2): the first form, scalar and with the
// address of a step worked out twice, was bound by instruction issue (369 a step of 1 KB).
template <int G, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(256, kMinCtas) qk_norm_rope_vec_kernel(const RopeParams p, int steps, int parts) {
  constexpr int HPW = 32 / G;                        // heads of a step
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long wid = blockIdx.x * 8LL + (threadIdx.x >> 5);
  const int i = (int)(wid / parts), part = (int)(wid - (long long)i * parts);
  if (i >= p.T) return;
  const int heads = p.q_per + 2 * p.kv_per, total = p.t * heads;
  const int sub = lane / G, l = lane % G;
  // the pieces of this lane (va, vb < 0: none) and its rotated pairs, 8 l on
  const int nv = p.hd >> 3, half = p.rd >> 1;
  int va, vb, rot;
  if (INTERLEAVED) {
    va = 2 * l;
    vb = 2 * l + 1;
    rot = min(8, max(0, half - 8 * l));
  } else {
    const int np = p.rd >> 4;
    va = l < np ? l : 2 * l;
    vb = l < np ? l + np : 2 * l + 1;
    rot = l < np ? 8 : 0;
  }
  if (va >= nv) va = -1;
  if (vb >= nv) vb = -1;
  const int pos = p.pos[i];
  const int slot = p.slots != nullptr ? p.slots[i] : -1;
  const int h0 = part * steps * HPW + sub, h_end = min(total, (part + 1) * steps * HPW);
  const bool in_place = p.in == p.out;
  uint4 a[kUnroll], b[kUnroll];
  size_t at[kUnroll];                                // element of the head in qkv
  int kind[kUnroll];                                 // its index among the shard's heads (< 0: none), and the shard
  int shard[kUnroll];
  // h / heads as a product: 2^32 / heads rounded up is off by less than 1, and h * heads < 2^32
  const unsigned magic = 0xffffffffu / (unsigned)heads + 1u;
  const size_t token = (size_t)i * p.rstride;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int h = h0 + u * HPW;
    a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
    kind[u] = -1;
    if (h < h_end) {
      shard[u] = (int)__umulhi((unsigned)h, magic);
      kind[u] = h - shard[u] * heads;
      at[u] = token + (size_t)shard[u] * p.sstride + kind[u] * p.hd;
      if (in_place && p.slots == nullptr && kind[u] >= p.q_per + p.kv_per) {
        kind[u] = -1;                                // v stays where it is
      } else {
        const __nv_bfloat16* src = p.in + at[u];
        if (va >= 0) a[u] = *reinterpret_cast<const uint4*>(src + va * 8);
        if (vb >= 0) b[u] = *reinterpret_cast<const uint4*>(src + vb * 8);
      }
    }
  }
  if (pos < 0 || pos >= p.n_pos) {                   // padding token, or past the table: nothing is written
    if (pos >= 0 && lane == 0) atomicExch(p.status, kStatusShape);
    return;
  }
  if (slot >= p.n_slots && p.slots != nullptr && lane == 0) atomicExch(p.status, kStatusShape);
  const bool write = slot >= 0 && slot < p.n_slots;
  float c[8], s[8];
  const float* tab = p.table + (size_t)pos * p.rd + 8 * l;
  if (rot == 8 && (p.rd & 7) == 0) {
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      *reinterpret_cast<float4*>(c + k) = *reinterpret_cast<const float4*>(tab + k);
      *reinterpret_cast<float4*>(s + k) = *reinterpret_cast<const float4*>(tab + half + k);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      c[k] = k < rot ? tab[k] : 1.f;
      s[k] = k < rot ? tab[half + k] : 0.f;
    }
  }
  const float inv_hd = 1.0f / p.hd;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (h0 - sub + u * HPW >= h_end) break;          // the whole warp
    const bool is_v = kind[u] >= p.q_per + p.kv_per, is_q = kind[u] < p.q_per;
    uint4 oa = a[u], ob = b[u];
    const uint32_t* wa = &a[u].x;
    const uint32_t* wb = &b[u].x;
    uint64_t x[4], y[4];                             // elements 2 k, 2 k + 1 of the two pieces
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[k] = unpack2(wa[k]);
      y[k] = unpack2(wb[k]);
    }
    float rs = 1.f;
    if (NORM) {                                      // the whole warp: its heads share the exchange
      uint64_t q = 0ull;
#pragma unroll
      for (int k = 0; k < 4; ++k) q = f32x2_fma(y[k], y[k], f32x2_fma(x[k], x[k], q));
      float s0, s1;
      f32x2_unpack(q, s0, s1);
      s0 += s1;
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o);
      const __nv_bfloat16* gamma = is_q ? p.q_gamma : p.k_gamma;
      if (!is_v && gamma != nullptr) {
        rs = rsqrtf(s0 * inv_hd + p.eps);            // applied after the rotation, which is linear
        uint4 ga = make_uint4(0u, 0u, 0u, 0u), gb = ga;
        if (va >= 0) ga = __ldg(reinterpret_cast<const uint4*>(gamma + va * 8));
        if (vb >= 0) gb = __ldg(reinterpret_cast<const uint4*>(gamma + vb * 8));
        const uint32_t* wga = &ga.x;
        const uint32_t* wgb = &gb.x;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[k] = f32x2_mul(x[k], unpack2(wga[k]));
          y[k] = f32x2_mul(y[k], unpack2(wgb[k]));
        }
      }
    }
    if (!is_v) {
      if (INTERLEAVED) {
        // the pairs of piece a are 8 l .. 8 l + 3, of piece b 8 l + 4 .. 8 l + 7
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x0, x1, y0, y1;
          f32x2_unpack(x[k], x0, x1);
          f32x2_unpack(y[k], y0, y1);
          x[k] = f32x2_pack(x0 * c[k] - x1 * s[k], x1 * c[k] + x0 * s[k]);
          y[k] = f32x2_pack(y0 * c[4 + k] - y1 * s[4 + k], y1 * c[4 + k] + y0 * s[4 + k]);
        }
      } else if (rot) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t c2 = f32x2_pack(c[2 * k], c[2 * k + 1]), s2 = f32x2_pack(s[2 * k], s[2 * k + 1]);
          const uint64_t n2 = f32x2_pack(-s[2 * k], -s[2 * k + 1]), x0 = x[k];
          x[k] = f32x2_fma(y[k], n2, f32x2_mul(x0, c2));
          y[k] = f32x2_fma(x0, s2, f32x2_mul(y[k], c2));
        }
      }
      if (NORM) {
        const uint64_t r2 = f32x2_pack(rs, rs);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[k] = f32x2_mul(x[k], r2);
          y[k] = f32x2_mul(y[k], r2);
        }
      }
      oa = make_uint4(pack2(x[0]), pack2(x[1]), pack2(x[2]), pack2(x[3]));
      ob = make_uint4(pack2(y[0]), pack2(y[1]), pack2(y[2]), pack2(y[3]));
    }
    if (kind[u] >= 0) {
      if (!is_v || !in_place) {
        __nv_bfloat16* dst = p.out + at[u];
        if (va >= 0) *reinterpret_cast<uint4*>(dst + va * 8) = oa;
        if (vb >= 0) *reinterpret_cast<uint4*>(dst + vb * 8) = ob;
      }
      if (write && !is_q) {
        __nv_bfloat16* dst = (is_v ? p.cache_v : p.cache_k) +
                             (((size_t)shard[u] * p.n_slots + slot) * p.kv_per + (kind[u] - p.q_per - (is_v ? p.kv_per : 0))) * p.hd;
        if (va >= 0) *reinterpret_cast<uint4*>(dst + va * 8) = oa;
        if (vb >= 0) *reinterpret_cast<uint4*>(dst + vb * 8) = ob;
      }
    }
  }
}

cudaError_t launch_rope_table(const RopeFreqs& f, long long n_pos, int rotary_dim, float* table, int nsm, cudaStream_t st) {
  const long long n = n_pos * (rotary_dim / 2);
  const int grid = (int)std::min<long long>((n + 255) / 256, 16LL * nsm);
  rope_table_kernel<<<grid, 256, 0, st>>>(f, n_pos, rotary_dim / 2, table);
  return cudaGetLastError();
}

template <int G>
static cudaError_t launch_vec(const RopeParams& p, int nsm, cudaStream_t st) {
  // steps of 32 / G heads of a token: kUnroll per warp, fewer where that leaves SMs without work
  const int total = (p.t * (p.q_per + 2 * p.kv_per) * G + 31) / 32;
  int steps = kUnroll;
  while (steps > 1 && (long long)p.T * ((total + steps - 1) / steps) < 16LL * nsm) --steps;
  const int parts = (total + steps - 1) / steps;
  const long long warps = (long long)p.T * parts;
  const bool norm = p.q_gamma != nullptr || p.k_gamma != nullptr;
  auto kernel = p.interleaved ? (norm ? qk_norm_rope_vec_kernel<G, true, true> : qk_norm_rope_vec_kernel<G, true, false>)
                              : (norm ? qk_norm_rope_vec_kernel<G, false, true> : qk_norm_rope_vec_kernel<G, false, false>);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = programmatic(dim3((unsigned)((warps + 7) / 8)), 256, 0, st, attr);
  return cudaLaunchKernelEx(&cfg, kernel, p, steps, parts);
}

cudaError_t launch_qk_norm_rope(const RopeParams& p, int nsm, cudaStream_t st) {
  if (p.interleaved || p.rd % 16 == 0) {
    const int lanes = (p.hd / 8 + 1) / 2;            // of a head
    if (lanes <= 1) return launch_vec<1>(p, nsm, st);
    if (lanes <= 2) return launch_vec<2>(p, nsm, st);
    if (lanes <= 4) return launch_vec<4>(p, nsm, st);
    return lanes <= 8 ? launch_vec<8>(p, nsm, st) : launch_vec<16>(p, nsm, st);
  }
  const long long items = (long long)p.T * p.t * (p.q_per + 2 * p.kv_per);
  const int grid = (int)std::min<long long>((items + kWarps - 1) / kWarps, 16LL * nsm);
  qk_norm_rope_kernel<<<grid, 32 * kWarps, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace tpl
