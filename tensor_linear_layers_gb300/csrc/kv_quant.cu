// A paged KV cache in 8 bits: k and v heads quantised as they are written, and read back.
//
// A head row x of 128 elements is stored as e4m3 codes and one scale byte s:
//   e = the smallest integer with max|x| <= 448 * 2^e, within [-100, 118];  s = e + 127
//   code_i = e4m3(x_i * 2^-e), to nearest, ties to even, at most 448 in size
//   value  = code_i * 2^e
// x * 2^-e is exact, so a code is rounded once, and every value is a bf16. A power of two costs no
// precision against max|x| / 448: codes are floating-point, and the row's largest element
// is in (224, 448] (its smallest normal code at least 2^-15 of it). A row with a NaN or an infinity
// gets s = 255 and codes 0, and stands for NaN.
//
// Both calls move bytes: write 256 in, 129 out per row, read the other way round. Eight lanes hold
// a row, 16 elements each, so that a row's codes are one 128-byte line in 16-byte pieces and its largest
// element takes three exchanges; 32 lanes of four elements would take five and four-byte stores.
// Measured: 65 536 tokens of 16 heads read in 65 us, 6.2 TB/s (93 % of a plain copy); 8192 tokens of 16
// heads written in 10.8 us, of which 7.5 are the bytes; calls of a few hundred tokens are 7 us of the host's
// call and 1.6 on the device.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gemm_tc.cuh"
#include "internal.h"

namespace tpl {

namespace {
constexpr int kHd = 128;
constexpr int kStatusShape = -2;     // TP_ERR_SHAPE
constexpr int kThreads = 256;
constexpr int kRowLanes = 8;
constexpr int kScaleNan = 255;

// two fp32 as e4m3, lo in the low byte
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// two codes (low 16 bits) as f16 pairs, exact
__device__ __forceinline__ uint32_t f16x2_of(uint32_t codes) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)codes));
  return d;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float f16_lo(uint32_t w) {
  float f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(w));
  return f;
}
__device__ __forceinline__ float f16_hi(uint32_t w) {
  float f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, hi;\n\t}" : "=f"(f) : "r"(w));
  return f;
}

// Row `at` of the 2 * t * kv_per head rows of a token: kv head fastest, then k or v, then the shard.
struct RowAt {
  int r, kv, g;
};
__device__ __forceinline__ RowAt row_at(int at, int kv_per) {
  RowAt x;
  x.g = at % kv_per;
  at /= kv_per;
  x.kv = at & 1;
  x.r = at >> 1;
  return x;
}
}  // namespace

// A row per lane group.
__global__ void __launch_bounds__(kThreads) kv_quant_write_kernel(const KvQuantParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & (kRowLanes - 1);
  const unsigned per_token = 2u * p.t * p.kv_per, total = per_token * (unsigned)p.n;
  const unsigned row = blockIdx.x * (kThreads / kRowLanes) + threadIdx.x / kRowLanes;
  uint4 x[2] = {};
  size_t dst = 0;
  int kv = -1;
  if (row < total) {
    const int i = (int)(row / per_token);
    const RowAt a = row_at((int)(row - i * per_token), p.kv_per);
    const int s = p.slots[i];
    if (s >= 0 && s < p.n_slots) {
      const uint4* src = reinterpret_cast<const uint4*>(p.qkv + (size_t)a.r * p.sstride + (size_t)i * p.rstride +
                                                        (size_t)(p.q_per + a.kv * p.kv_per + a.g) * kHd) + 2 * lane;
      x[0] = src[0];
      x[1] = src[1];
      kv = a.kv;
      dst = ((size_t)a.r * p.n_slots + s) * p.kv_per + a.g;
    } else if (s >= p.n_slots && lane == 0) {
      atomicExch(p.status, kStatusShape);
    }
  }
  const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
  // the largest size: without the sign, bf16 bits are ordered as whole numbers, NaN above infinity
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
  int m = max((int)(top & 0xffffu), (int)(top >> 16));
#pragma unroll
  for (int o = kRowLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (kv < 0) return;
  // max = 2^(E - 127) (1 + f / 128), 448 = 2^8 (1 + 96 / 128)
  const int s = m >= 0x7f80 ? kScaleNan : min(max((m >> 7) - 8 + ((m & 127) > 96 ? 1 : 0), 27), 245);
  const float inv = s == kScaleNan ? 0.f : __uint_as_float((unsigned)(254 - s) << 23);    // 2^(127 - s)
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[2 * i], b = w[2 * i + 1];
    c[i] = e4m3x2(bf16_lo(a) * inv, bf16_hi(a) * inv) | e4m3x2(bf16_lo(b) * inv, bf16_hi(b) * inv) << 16;
    if (s == kScaleNan) c[i] = 0u;
  }
  uint8_t* codes = kv ? p.codes[1] : p.codes[0];
  uint8_t* scales = kv ? p.scales[1] : p.scales[0];
  reinterpret_cast<uint4*>(codes + dst * kHd)[lane] = make_uint4(c[0], c[1], c[2], c[3]);
  if (lane == 0) scales[dst] = (uint8_t)s;
}

// ROWS rows of one lane group are loaded together (bytes in flight).
template <int ROWS>
__global__ void __launch_bounds__(kThreads) kv_quant_read_kernel(const KvQuantParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & (kRowLanes - 1);
  const unsigned per_token = 2u * p.t * p.kv_per, total = per_token * (unsigned)p.n;
  constexpr unsigned kGroups = kThreads / kRowLanes;
  const unsigned first = blockIdx.x * (kGroups * ROWS) + threadIdx.x / kRowLanes;
  uint4 x[ROWS];
  unsigned scale[ROWS];
  uint4* dst[ROWS];
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    const unsigned row = first + j * kGroups;
    x[j] = make_uint4(0, 0, 0, 0);
    scale[j] = 127;
    dst[j] = nullptr;
    if (row < total) {
      const int i = (int)(row / per_token);
      const RowAt a = row_at((int)(row - i * per_token), p.kv_per);
      const int s = p.slots[i];
      if (s >= 0 && s < p.n_slots) {
        const size_t at = ((size_t)a.r * p.n_slots + s) * p.kv_per + a.g;
        x[j] = reinterpret_cast<const uint4*>((a.kv ? p.codes[1] : p.codes[0]) + at * kHd)[lane];
        scale[j] = (a.kv ? p.scales[1] : p.scales[0])[at];
      } else if (s >= p.n_slots && lane == 0) {
        atomicExch(p.status, kStatusShape);
      }
      dst[j] = reinterpret_cast<uint4*>((a.kv ? p.out[1] : p.out[0]) + (((size_t)a.r * p.n + i) * p.kv_per + a.g) * kHd) + 2 * lane;
    }
  }
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    if (dst[j] == nullptr) continue;
    // 2^(s - 127): s = 0 is a subnormal number, 255 NaN
    const float f = __uint_as_float(scale[j] == 0 ? 0x00400000u : scale[j] == kScaleNan ? 0x7fc00000u : scale[j] << 23);
    const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = f16x2_of(w[i]), b = f16x2_of(w[i] >> 16);
      o[2 * i] = pack_bf16x2(f16_lo(a) * f, f16_hi(a) * f);
      o[2 * i + 1] = pack_bf16x2(f16_lo(b) * f, f16_hi(b) * f);
    }
    dst[j][0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[j][1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

namespace {
template <class Kernel>
cudaError_t launch_rows(Kernel kernel, int rows_each, const KvQuantParams& p, cudaStream_t st) {
  const long long rows = 2LL * p.t * p.kv_per * p.n, per = (long long)(kThreads / kRowLanes) * rows_each;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = programmatic(dim3((unsigned)((rows + per - 1) / per)), kThreads, 0, st, attr);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}
}  // namespace

// A row per lane group: 8192 tokens in 10.8 us (11.9 with four rows in flight, 32 tokens 7.9 and 8.1).
cudaError_t launch_kv_quant_write(const KvQuantParams& p, cudaStream_t st) { return launch_rows(kv_quant_write_kernel, 1, p, st); }
// Four rows in flight once every SM has blocks enough (65 536 tokens in 65 us, 71 with one row), else one (1021
// tokens in 8.3 us, 8.7 with four).
cudaError_t launch_kv_quant_read(const KvQuantParams& p, int nsm, cudaStream_t st) {
  const bool many = 2LL * p.t * p.kv_per * p.n > 8LL * (kThreads / kRowLanes) * nsm;
  return many ? launch_rows(kv_quant_read_kernel<4>, 4, p, st) : launch_rows(kv_quant_read_kernel<1>, 1, p, st);
}

}  // namespace tpl
