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
// steps of a warp in flight, warps per SM (72 registers): 4096 tokens of 48 heads with norm 23.5 us;
// (2, 32) 27.3, (4, 20) 24.0, (4, 24) 24.5, (6, 16) 26.0
constexpr int kUnroll = 3, kMinCtas = 25;

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
__global__ void rope_table_kernel(const RopeFreqs f, long long n_pos, int half, float* table) {
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

// A head is held by G lanes, two 16-byte pieces of 8 elements each. Where it can be, both
// elements of every pair are in one lane and no exchange is needed:
//   kHalf         half layout, rd a multiple of 16: pieces l and l + rd/16 for l < rd/16 (pairs
//                 8 l .. 8 l + 7), the unrotated pieces two by two after them
//   kInterleaved  interleaved layout: pieces 2 l and 2 l + 1 (the same pairs 8 l .. 8 l + 7)
//   kHalfAny      half layout, any even rd: pieces 2 l and 2 l + 1; an element's partner comes
//                 through shared memory (4096 tokens of 48 heads, rd = 20: 54.7 us; 24.5 for rd = 128)
enum RopeMode : int { kHalf = 0, kInterleaved = 1, kHalfAny = 2 };
struct Pieces {
  int va, vb;                        // piece indices (< 0: none)
  int rot;                           // rotated pairs of this lane, 8 l on
};
template <int MODE>
__device__ __forceinline__ Pieces pieces_of(int l, int hd, int rd) {
  Pieces q;
  if (MODE != kHalf) {
    q.va = 2 * l;
    q.vb = 2 * l + 1;
    q.rot = min(8, max(0, (rd >> 1) - 8 * l));
  } else {
    const int np = rd >> 4;
    q.va = l < np ? l : 2 * l;
    q.vb = l < np ? l + np : 2 * l + 1;
    q.rot = l < np ? 8 : 0;
  }
  if (q.va >= hd >> 3) q.va = -1;
  if (q.vb >= hd >> 3) q.vb = -1;
  return q;
}

// cos and sin of a lane's pairs (1 and 0 past them) from a table row, tab = row + 8 l
__device__ __forceinline__ void load_angles(float* c, float* s, const float* tab, int rd, int rot) {
  const int half = rd >> 1;
  if (rot == 8 && (rd & 7) == 0) {
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
}

// One q or k head: this lane's two pieces, normed and rotated. The whole
// warp calls it (its heads share the exchange of the sums). The arithmetic goes by pairs of
// fp32 (fma.rn.f32x2): scalar, the kernel was bound by instruction issue (369 for 1 KB).
// kHalfAny: xs, room for the lane group's head; tab, the token's table row.
template <int G, int MODE, bool NORM>
__device__ __forceinline__ void turn(uint4& a, uint4& b, const Pieces& q, const float* c, const float* s,
                                     const __nv_bfloat16* gamma, float inv_hd, float eps, float* xs, const float* tab,
                                     int rd) {
  const uint32_t* wa = &a.x;
  const uint32_t* wb = &b.x;
  uint64_t x[4], y[4];                               // elements 2 k, 2 k + 1 of the two pieces
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[k] = unpack2(wa[k]);
    y[k] = unpack2(wb[k]);
  }
  float rs = 1.f;
  if (NORM) {
    uint64_t sq = 0ull;
#pragma unroll
    for (int k = 0; k < 4; ++k) sq = f32x2_fma(y[k], y[k], f32x2_fma(x[k], x[k], sq));
    float s0, s1;
    f32x2_unpack(sq, s0, s1);
    s0 += s1;
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o);
    if (gamma != nullptr) {
      rs = rsqrtf(s0 * inv_hd + eps);                // applied after the rotation, which is linear
      uint4 ga = make_uint4(0u, 0u, 0u, 0u), gb = ga;
      if (q.va >= 0) ga = *reinterpret_cast<const uint4*>(gamma + q.va * 8);
      if (q.vb >= 0) gb = *reinterpret_cast<const uint4*>(gamma + q.vb * 8);
      const uint32_t* wga = &ga.x;
      const uint32_t* wgb = &gb.x;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[k] = f32x2_mul(x[k], unpack2(wga[k]));
        y[k] = f32x2_mul(y[k], unpack2(wgb[k]));
      }
    }
  }
  if (MODE == kHalfAny) {
    const int l = threadIdx.x % G, half = rd >> 1;
    uint64_t* mine = reinterpret_cast<uint64_t*>(xs + 16 * l);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      mine[k] = x[k];
      mine[4 + k] = y[k];
    }
    __syncwarp();
    auto turned = [&](float v, int e) {
      if (e >= rd) return v;
      const bool first = e < half;
      const int j = first ? e : e - half;
      const float other = xs[first ? e + half : j], cj = tab[j], sj = tab[half + j];
      return first ? v * cj - other * sj : v * cj + other * sj;
    };
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x0, x1, y0, y1;
      f32x2_unpack(x[k], x0, x1);
      f32x2_unpack(y[k], y0, y1);
      x[k] = f32x2_pack(turned(x0, 16 * l + 2 * k), turned(x1, 16 * l + 2 * k + 1));
      y[k] = f32x2_pack(turned(y0, 16 * l + 8 + 2 * k), turned(y1, 16 * l + 8 + 2 * k + 1));
    }
    __syncwarp();                                    // read before the next step writes
  } else if (MODE == kInterleaved) {
    // the pairs of piece a are 8 l .. 8 l + 3, of piece b 8 l + 4 .. 8 l + 7; those past the rotated
    // ones stay as they are (turned by an angle of 0, an infinite element would make its partner NaN).
    // Both results and a selection: 2043 tokens of 36 heads with norm, half of each rotated, 10.0 us;
    // branches on the lane's rotated pairs 10.1, everything turned 9.8
    auto turned = [&](uint64_t v, int k) {
      float e0, e1;
      f32x2_unpack(v, e0, e1);
      return f32x2_pack(e0 * c[k] - e1 * s[k], e1 * c[k] + e0 * s[k]);
    };
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint64_t tx = turned(x[k], k), ty = turned(y[k], 4 + k);
      x[k] = k < q.rot ? tx : x[k];
      y[k] = 4 + k < q.rot ? ty : y[k];
    }
  } else if (q.rot) {
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
  a = make_uint4(pack2(x[0]), pack2(x[1]), pack2(x[2]), pack2(x[3]));
  b = make_uint4(pack2(y[0]), pack2(y[1]), pack2(y[2]), pack2(y[3]));
}

__device__ __forceinline__ void store_pieces(__nv_bfloat16* dst, const Pieces& q, const uint4& a, const uint4& b) {
  if (q.va >= 0) *reinterpret_cast<uint4*>(dst + q.va * 8) = a;
  if (q.vb >= 0) *reinterpret_cast<uint4*>(dst + q.vb * 8) = b;
}

// Bound by HBM: every q, k and v element is read once and written once. The heads of a token go
// in steps of 32 / G, first the q heads of all shards, then the k heads, then the v heads, so
// that a step is of one kind (steps that mixed them ran both ways: 27.4 against 24.6 us for
// 4096 tokens of 48 heads with norm). A warp takes up to kUnroll steps of one token, loaded together:
// a lane's cosines, sines and weights serve all of them. A warp is a CTA: each ends and makes room
// for the next by itself (4096 tokens of 48 heads with norm 23.5 us, 25.6 with eight warps to a CTA,
// 25.2 with four or two; 8192 tokens of 80 heads 61.5, 64.4, 62.8, 62.1), 0.75 and 0.90 of HBM. Tried
// and dropped: persistent warps with a ring of bulk copies in shared memory (8192 tokens of 80 heads
// 65.9 us, 2048 tokens of 48 heads 19.0 against 13.8).
template <int G, int MODE, bool NORM>
__global__ void __launch_bounds__(32, kMinCtas) qk_norm_rope_kernel(const RopeParams p, int steps, int parts) {
  constexpr int HPW = 32 / G;                        // heads of a step
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x;
  const int i = (int)(blockIdx.x / (unsigned)parts), part = (int)(blockIdx.x - (unsigned)i * (unsigned)parts);
  const int sub = lane / G, l = lane % G;
  const Pieces q = pieces_of<MODE>(l, p.hd, p.rd);
  const int pos = p.pos[i];
  const int slot = p.slots != nullptr ? p.slots[i] : -1;
  const bool in_place = p.in == p.out;
  const int q_steps = (p.t * p.q_per + HPW - 1) / HPW, kv_steps = (p.t * p.kv_per + HPW - 1) / HPW;
  const int step_end = min((part + 1) * steps, q_steps + (in_place && p.slots == nullptr ? 1 : 2) * kv_steps);
  uint4 a[kUnroll], b[kUnroll];
  size_t at[kUnroll];                                // element of the head in qkv
  int head[kUnroll], shard[kUnroll];                 // its index among the shard's heads of the kind (< 0: none), and the shard
  int kind[kUnroll];                                 // 0 q, 1 k, 2 v (the same in the whole warp)
  const size_t token = (size_t)i * p.rstride;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    int st = part * steps + u;
    a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
    head[u] = kind[u] = -1;
    if (st < step_end) {
      kind[u] = st < q_steps ? 0 : st < q_steps + kv_steps ? 1 : 2;
      if (kind[u] > 0) st -= q_steps + (kind[u] - 1) * kv_steps;
      const int per = kind[u] == 0 ? p.q_per : p.kv_per, h = st * HPW + sub;
      if (h < p.t * per) {
        shard[u] = (unsigned)h / (unsigned)per;
        head[u] = h - shard[u] * per;
        const int first = kind[u] == 0 ? 0 : kind[u] == 1 ? p.q_per : p.q_per + p.kv_per;
        at[u] = token + (size_t)shard[u] * p.sstride + (first + head[u]) * p.hd;
        const __nv_bfloat16* src = p.in + at[u];
        if (q.va >= 0) a[u] = *reinterpret_cast<const uint4*>(src + q.va * 8);
        if (q.vb >= 0) b[u] = *reinterpret_cast<const uint4*>(src + q.vb * 8);
      }
    }
  }
  if (pos < 0 || pos >= p.n_pos) {                   // padding token, or past the table: nothing is written
    if (pos >= 0 && lane == 0) atomicExch(p.status, kStatusShape);
    return;
  }
  if (slot >= p.n_slots && p.slots != nullptr && lane == 0) atomicExch(p.status, kStatusShape);
  const bool write = slot >= 0 && slot < p.n_slots;
  __shared__ float heads_s[MODE == kHalfAny ? 512 : 1];   // 16 elements a lane
  float* xs = MODE == kHalfAny ? heads_s + 16 * G * sub : nullptr;
  const float* tab = p.table + (size_t)pos * p.rd;
  float c[8], s[8];
  if (MODE != kHalfAny) load_angles(c, s, tab + 8 * l, p.rd, q.rot);
  const float inv_hd = 1.0f / p.hd;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (kind[u] < 0) break;
    if (kind[u] < 2) {
      turn<G, MODE, NORM>(a[u], b[u], q, c, s, kind[u] == 0 ? p.q_gamma : p.k_gamma, inv_hd, p.eps, xs, tab, p.rd);
    }
    if (head[u] >= 0) {
      if (kind[u] < 2 || !in_place) store_pieces(p.out + at[u], q, a[u], b[u]);
      if (write && kind[u] > 0)
        store_pieces((kind[u] == 2 ? p.cache_v : p.cache_k) + (((size_t)shard[u] * p.n_slots + slot) * p.kv_per + head[u]) * p.hd,
                     q, a[u], b[u]);
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
static cudaError_t launch_heads(const RopeParams& p, int nsm, cudaStream_t st) {
  constexpr int HPW = 32 / G;
  // the steps of a token: kUnroll per warp, fewer where that leaves SMs without work, until there are
  // eight warps for each (64 tokens of 80 heads 2.8 us, with a bound of four 3.4; 384 tokens of 48 heads
  // with norm 4.8, with 16 6.2; 512 tokens 5.1, with 28 7.6; 1024 tokens 6.9, with 48 13.7)
  const int q_steps = (p.t * p.q_per + HPW - 1) / HPW, kv_steps = (p.t * p.kv_per + HPW - 1) / HPW;
  const int total = q_steps + (p.in == p.out && p.slots == nullptr ? 1 : 2) * kv_steps;
  int steps = kUnroll;
  while (steps > 1 && (long long)p.T * ((total + steps - 1) / steps) < 8LL * nsm) --steps;
  const int parts = (total + steps - 1) / steps;
  const long long warps = (long long)p.T * parts;
  if (warps > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const bool norm = p.q_gamma != nullptr || p.k_gamma != nullptr;
  auto kernel = p.interleaved      ? (norm ? qk_norm_rope_kernel<G, kInterleaved, true> : qk_norm_rope_kernel<G, kInterleaved, false>)
                : p.rd % 16 == 0 ? (norm ? qk_norm_rope_kernel<G, kHalf, true> : qk_norm_rope_kernel<G, kHalf, false>)
                                 : (norm ? qk_norm_rope_kernel<G, kHalfAny, true> : qk_norm_rope_kernel<G, kHalfAny, false>);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = programmatic(dim3((unsigned)warps), 32, 0, st, attr);
  return cudaLaunchKernelEx(&cfg, kernel, p, steps, parts);
}

cudaError_t launch_qk_norm_rope(const RopeParams& p, int nsm, cudaStream_t st) {
  const int lanes = (p.hd / 8 + 1) / 2;              // of a head
  if (lanes <= 1) return launch_heads<1>(p, nsm, st);
  if (lanes <= 2) return launch_heads<2>(p, nsm, st);
  if (lanes <= 4) return launch_heads<4>(p, nsm, st);
  return lanes <= 8 ? launch_heads<8>(p, nsm, st) : launch_heads<16>(p, nsm, st);
}

}  // namespace tpl
