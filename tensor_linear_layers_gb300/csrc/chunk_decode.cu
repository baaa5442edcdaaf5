// Attention of few query rows over the paged KV cache: decoding requests, whose new tokens x the q
// heads of a kv head are up to eight rows. The mathematics, the masks and the work split are those of
// chunk_attention.cu, whose 128-row tiles such rows leave empty: there one warp does the whole
// softmax of a chunk while the other lanes have no row.
//
// Here the keys are the long side of the tiles: warp-level m16n8k16 products
//   S^T = K Q^T   (16 keys x 8 rows),   O^T = V^T P^T   (16 head dimensions x 8 rows)
// so that 8 rows cost 8 columns. A CTA's eight warps take 16 keys each of every chunk of 128 and
// keep their own running max, sum and O, all in registers. Each copies its own keys through the
// block table with 16-byte cp.async into a ring of its own, two chunks ahead across segments, so
// that within a segment no warp waits for another; they meet at its end. Segments come in batches
// of up to three, walked by warp 0 (chunk_walk.cuh), their queries loaded together.
//
// 8 bits: a warp reads the codes as they are stored, 16 bytes of a row per lane, and one
// conversion instruction makes two f16 of two codes, exactly. Which dimensions of K a lane's codes
// are is a permutation that Q's operand takes too; V's codes of two keys are interleaved by byte
// before the conversion. The scales never touch the codes:
//   x_j = s_j log2(e) + e_j (e_j: exponent of v's scale),   w_j = 2^(x_j - m)
//   m = max_j (s_j log2(e) + max(e_j, -86)) - 7
//   O = sum_j w_j code_j,   l = sum_j 2^(x_j - e_j - m)
// with k's scale in the factor of the raw product. w is 2^7 at the row's largest x, at most 2^15 (m moves when a
// row exceeds it by 2^8 more than it was taken at), and rounded to f16: 2^-11 of it down to 2^-21 of the
// largest, 2^-32 of the largest below. (-86: slots that were never written have a scale of 2^-127, and keys of
// those alone would take l to 2^134. Where all of v's scales are smaller, the largest w is smaller by as much.)
// q goes to f16 with a power of two per row that brings its largest element to [2^8, 2^9): exact for elements
// down to 2^-16 of that, off by 2^-33 of it below.
//
// bf16: operands come through ldmatrix; m = max_j x_j + 17 as in chunk_attention.cu, w in bf16.
//
// Two CTAs of 128 registers per SM in 8 bits (one CTA: 32 requests of 2000 keys 48.5 us for 39.4, 4 x 131 072
// keys 287 for 187), one of 232 in bf16, whose rings fill shared memory. HBM bounds it while it streams, 0.86 of a
// copy (4 x 131 072 keys, 64 q heads: 187 us for 160 of bytes); a batch of 32 requests of 255 - 4095 keys takes 39 us
// for 21 of bytes: 3.5 until the walk is done and 2 until the tables' and scales' dependent loads have given the first
// rows, 25 of streaming, 4 of the merge behind the grid, the rest the ends of uneven CTAs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "chunk_walk.cuh"
#include "gemm_tc.cuh"
#include "internal.h"
#include "paged_tiles.cuh"

namespace tpl {

namespace {
constexpr int kHd = 128;
constexpr int kWarps = 8;                      // consumers: 16 keys of a chunk each
constexpr int kThreads = 32 * kWarps;
constexpr int kBatch = 3;                      // segments of a batch
constexpr int kRows = 8;                       // query rows of an item
constexpr float kRescaleLog2 = 8.0f;
// 8 bits: an exponent of v's scale below this counts as this where m is taken, so that l, whose weights are without
// v's scale, is at most 2^(86 + 15) for each of 2^26 keys, and finite
constexpr float kLeastExponent = -86.0f;

template <bool Q8>
struct DecodeCfg {
  static constexpr int kCtas = Q8 ? 2 : 1;                   // per SM
  static constexpr int kRowBytes = Q8 ? kHd : 2 * kHd;
  static constexpr int kTile = 16 * kRowBytes;               // K or V of a warp's keys
  static constexpr int kStages = 3;
  static constexpr int kRing = kStages * 2 * kTile;          // of one warp
  static constexpr int kQBytes = kRows * kHd * 2;
  static constexpr int kQOff = kWarps * kRing;
  static constexpr int kFactorOff = kQOff + kBatch * kQBytes;     // [segment][row]
  static constexpr int kMlOff = kFactorOff + kBatch * kRows * 4;  // [warp][row] (max, sum)
  static constexpr int kSegOff = kMlOff + kWarps * kRows * 8;
  static constexpr int kWalkOff = kSegOff + kBatch * 64;
  static constexpr int kBarOff = kWalkOff + (int)((sizeof(ChunkWalk<true>) + 15) / 16 * 16);
  enum { READY = 0, X_FULL, X_EMPTY, NBARS };
  static constexpr int kMiscOff = kBarOff + 8 * NBARS;       // abort flag, segments of the batch
  static constexpr int kSmem = kMiscOff + 8 + 128;           // 128: alignment of the base
  static_assert((kSmem + 1024) * kCtas <= 233472, "shared memory of the CTAs of one SM");
  static_assert(2 * kTile >= 8 * kHd * 4, "eight rows of O in a place of the ring");
  static constexpr float kHead = Q8 ? -7.0f : 17.0f;         // m above the largest x when it is taken
};

// two codes (low or high 16 bits of w) as an f16 pair
__device__ __forceinline__ uint32_t f16x2_lo(uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(w));
  return d;
}
__device__ __forceinline__ uint32_t f16x2_hi(uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(d) : "r"(w));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 x 8 matrix of 16-bit elements in an operand's layout, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// 2^(s - 127) of a scale byte: 0 is a subnormal number, 255 NaN
__device__ __forceinline__ float scale_value(uint32_t s) {
  return __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7fc00000u : s << 23);
}
__device__ __forceinline__ float scale_exponent(uint32_t s) { return s == 255u ? __int_as_float(0x7fffffff) : (float)((int)s - 127); }
}  // namespace

template <bool Q8>
__global__ void __launch_bounds__(kThreads, DecodeCfg<Q8>::kCtas) chunk_decode_kernel(const ChunkAttnParams p) {
  using C = DecodeCfg<Q8>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 127u) & ~127u;
  uint8_t* base_ptr = smem_raw + (base - smem_u32(smem_raw));
  auto bar = [&](int b) { return base + C::kBarOff + 8u * b; };
  volatile int* s_abort = reinterpret_cast<volatile int*>(base_ptr + C::kMiscOff);
  volatile int* s_count = s_abort + 1;
  ChunkSegment* s_seg = reinterpret_cast<ChunkSegment*>(base_ptr + C::kSegOff);
  ChunkWalk<true>* s_walk = reinterpret_cast<ChunkWalk<true>*>(base_ptr + C::kWalkOff);   // warp 0's between batches
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;   // (known to be one for all lanes)
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int b = 0; b < C::NBARS; ++b) mbar_init(bar(b), kWarps);
    *s_abort = 0;
    fence_barrier_init();
  }
  griddep_wait();
  const int gq = p.call.gq, sc = chunk_sinks(p.call), window = p.call.window, sinks = p.call.sinks;
  const unsigned long long timeout = p.timeout_ns;
  const unsigned gq_magic = 0xffffffffu / (unsigned)gq + 1u;
  auto token_of = [&](int row) { return gq == 1 ? row : (int)__umulhi((unsigned)row, gq_magic); };
  __syncthreads();
  bool ok = true;
  // all warps arrive and wait for all (bounded: a warp that gave up arrives nowhere)
  auto meet = [&](int b, uint32_t ph) -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
    bool w = mbar_wait_bounded(bar(b), ph, s_abort, timeout);
    w = __all_sync(0xffffffffu, w);
    if (!w) {
      if (lane == 0 && !*s_abort) {
        atomicExch(p.status, kStatusTimeout);
        *s_abort = 1;
      }
      ok = false;
    }
    return w;
  };
  const int g = lane >> 2, t = lane & 3;
  const uint64_t pol = policy_evict_first();                 // every key is read once
  const uint8_t* cache_k = static_cast<const uint8_t*>(p.cache_k);
  const uint8_t* cache_v = static_cast<const uint8_t*>(p.cache_v);
  // copies: this lane brings piece `piece` of rows kPer k + sub of the warp's 16
  constexpr int kPieces = C::kRowBytes / 16, kPer = 32 / kPieces;
  const int piece = lane % kPieces, sub = lane / kPieces;
  const uint32_t ring = base + warp * C::kRing;
  uint32_t xph = 0;
  float o[8][4];
  for (uint32_t batch = 0;; ++batch) {
    if (warp == 0) {
      ChunkWalk<true> walk;
      if (batch == 0) {
        walk.load(p, lane);
        walk.start(p, lane);
      } else {
        walk.resume(*s_walk);
      }
      int n = 0;
      for (; n < kBatch; ++n) {
        const ChunkSegment s = walk.next(p, lane);
        if (s.b < 0) break;
        if (lane == 0) s_seg[n] = s;
      }
      __syncwarp();
      if (lane == 0) {
        walk.keep(*s_walk);
        *s_count = n;
      }
    }
    if (!meet(C::READY, batch & 1)) break;
    const int segs = *s_count;
    if (segs == 0) break;
    // ---------------------------------------------------------- the batch's queries, and the first keys
    for (int i = threadIdx.x; i < segs * kRows * 16; i += kThreads) {
      const int k = i / (kRows * 16), j = i / 16 % kRows, tok = token_of(j), x = i & 15;
      const ChunkSegment& s = s_seg[k];
      const bool in = j < s.rows;
      const __nv_bfloat16* q = p.qkv + (size_t)s.r * p.sstride_in + (size_t)(s.q0 + s.tok0 + tok) * p.rstride_in +
                               (s.g * gq + j - tok * gq) * kHd + x * 8;
      cp_async16(base + C::kQOff + i * 16, in ? q : p.qkv, in ? 16 : 0, pol);
    }
    cp_async_commit();
    // The issuing cursor, chunk a_c of segment a_s, and the one that looks up blocks two chunks before it;
    // lanes 0 - 15 have a key each.
    int a_s = 0, a_c = s_seg[0].c0, f_s = 0, f_c = a_c, blk = -1, blk_next = -1, issued = 0;
    struct Flight { uint32_t k, v; };                        // scale bytes of the lane's key
    auto find = [&]() {
      blk = blk_next;
      blk_next = -1;
      if (f_s < segs) {
        const ChunkSegment& s = s_seg[f_s];
        const int key = chunk_key(f_c * kChunkKeys + 16 * warp, sc, s.skip) + lane;
        if (lane < 16 && chunk_any(p.call, key, s.p0, s.p1)) {
          blk_next = p.block_tables[(size_t)s.b * p.max_blocks + chunk_page(p, key)];
          if (blk_next < 0) blk_next = p.num_blocks;         // (-1: not seen)
        }
        if (++f_c == s.c1 && ++f_s < segs) f_c = s_seg[f_s].c0;
      }
    };
    auto issue = [&](Flight& f) {
      f.k = f.v = 127u;
      if (a_s < segs) {
        const ChunkSegment& s = s_seg[a_s];
        int row = -1;                                        // cache row of the lane's key; -1: zeros
        if (blk != -1) {
          row = chunk_row(p, s.r, blk, chunk_key(a_c * kChunkKeys + 16 * warp, sc, s.skip) + lane);
          if (row < 0) atomicExch(p.status, kChunkStatusShape);
        }
        const int hg = s.g;
        if constexpr (Q8) {
          if (row >= 0) {
            const size_t at = (size_t)row * p.kv_per + hg;
            f.k = p.scales_k[at];
            f.v = p.scales_v[at];
          }
        }
        if (__any_sync(0xffffffffu, lane < 16 && blk != -1)) {
          const uint32_t kd = ring + issued % C::kStages * (2 * C::kTile) + sub * C::kRowBytes, vd = kd + C::kTile;
          const uint8_t* ck = cache_k + (size_t)hg * C::kRowBytes + piece * 16;
          const uint8_t* cv = cache_v + (size_t)hg * C::kRowBytes + piece * 16;
          const unsigned stride = (unsigned)(p.kv_per * C::kRowBytes);
#pragma unroll
          for (int k = 0; k < 16 / kPer; ++k) {
            const int rw = __shfl_sync(0xffffffffu, row, kPer * k + sub), x = kPer * k + sub;
            const size_t off = (size_t)(unsigned)max(rw, 0) * stride;
            const int bytes = rw >= 0 ? 16 : 0;
            // pieces are permuted so that the reads below meet no bank twice
            const int kp = Q8 ? piece ^ ((x & 1) << 2) : piece ^ (x & 7), vp = Q8 ? piece ^ (((x >> 1) & 3) << 1) : kp;
            cp_async16(kd + kPer * k * C::kRowBytes + kp * 16, ck + off, bytes, pol);
            cp_async16(vd + kPer * k * C::kRowBytes + vp * 16, cv + off, bytes, pol);
          }
        }
        if (++a_c == s.c1 && ++a_s < segs) a_c = s_seg[a_s].c0;
      }
      cp_async_commit();
      ++issued;
      find();
    };
    Flight f[C::kStages];
    find();
    find();
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) issue(f[i]);
    cp_async_wait<C::kStages - 1>();                         // the queries
    if (!meet(C::X_FULL, xph)) break;
    // A segment's queries by one warp to the second operand's layout, in their place: for lane and k-step the
    // two registers of row g; and the rows' factors.
    if (warp < segs) {
      const int i = warp;
      const uint32_t tile = base + C::kQOff + i * (8 * kHd * 2), qs = tile + g * 256;
      uint32_t b[8][2];
      float factor = p.scale_log2;                           // log2(e) / sqrt(hd), and (8 bits) q's power of two
      if constexpr (Q8) {
        // the 32 elements of dimensions 64 j + 16 t + (0 .. 15)
        uint4 x[4];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = lds128(qs + (j >> 1) * 128 + t * 32 + (j & 1) * 16);
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[j].x & 0x7fff7fffu, x[j].y & 0x7fff7fffu),
                                       __vmaxu2(x[j].z & 0x7fff7fffu, x[j].w & 0x7fff7fffu)));
        }
        uint32_t m = max(top & 0xffffu, top >> 16);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int e = max((int)(m >> 7), 10);                // biased exponent of the row's largest element
        const float f = __uint_as_float((unsigned)(262 - e) << 23);            // 2^(8 - (e - 127))
        factor *= __uint_as_float((unsigned)(e - 8) << 23);
        auto half2 = [&](uint32_t w) { return pack_f16x2(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f); };
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          b[2 * j][0] = half2(x[j].x);
          b[2 * j][1] = half2(x[j].y);
          b[2 * j + 1][0] = half2(x[j].z);
          b[2 * j + 1][1] = half2(x[j].w);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          b[k][0] = lds32(qs + k * 32 + t * 4);
          b[k][1] = lds32(qs + k * 32 + 16 + t * 4);
        }
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k) sts128(tile + k * 512 + lane * 16, b[2 * k][0], b[2 * k][1], b[2 * k + 1][0], b[2 * k + 1][1]);
      if (t == 0) reinterpret_cast<float*>(base_ptr + C::kFactorOff)[i * 8 + g] = factor;
    }
    if (!meet(C::X_EMPTY, xph)) break;
    xph ^= 1u;
    int used = 0;                                            // chunks computed
    for (int u = 0; u < segs; ++u) {
      const int c0 = s_seg[u].c0, c1 = s_seg[u].c1, p0 = s_seg[u].p0, p1 = s_seg[u].p1, skip = s_seg[u].skip;
      const uint32_t qs = base + C::kQOff + u * C::kQBytes + lane * 16;
      const float2 factor = reinterpret_cast<const float2*>(base_ptr + C::kFactorOff)[u * 4 + t];   // of rows 2 t, 2 t + 1
      int pos[2];                                              // positions of rows 2 t, 2 t + 1
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) pos[h] = min(p0 + token_of(2 * t + h), p1);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < 4; ++h) o[i][h] = 0.f;
      bool bad = false;                                        // bf16: a V that only some rows see was not finite
      for (int c = c0; c < c1; ++c) {
        issue(f[C::kStages - 1]);
        cp_async_wait<C::kStages - 1>();
        __syncwarp();
        const int key = chunk_key(c * kChunkKeys + 16 * warp, sc, skip);         // the warp's first key
        const uint32_t ks = ring + used % C::kStages * (2 * C::kTile), vs = ks + C::kTile;
        // else nothing of the warp's keys is seen: past the last token, or in the gap before the window
        if (key <= p1 && (window == 0 || key + 15 > p0 - window || key < sinks)) {
          float s[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t k0 = 127u, k1 = 127u;                       // scales of keys g, g + 8: k's byte, v's exponent
          float e0 = 0.f, e1 = 0.f;
          if constexpr (Q8) {
            k0 = __shfl_sync(0xffffffffu, f[0].k, g);
            k1 = __shfl_sync(0xffffffffu, f[0].k, g + 8);
            e0 = scale_exponent(__shfl_sync(0xffffffffu, f[0].v, g));
            e1 = scale_exponent(__shfl_sync(0xffffffffu, f[0].v, g + 8));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t at = ks + g * 128 + (((4 * j + t) ^ ((g & 1) << 2)) << 4);
              const uint4 a = lds128(at), b = lds128(at + 8 * 128);
              const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
              for (int w = 0; w < 4; w += 2) {
                const uint4 q = lds128(qs + (2 * j + w / 2) * 512);   // k-steps 4 j + w and the next
                uint32_t a0 = f16x2_lo(aw[w]), a1 = f16x2_lo(bw[w]), a2 = f16x2_hi(aw[w]), a3 = f16x2_hi(bw[w]);
                mma16816<true>(s, a0, a1, a2, a3, q.x, q.y);
                a0 = f16x2_lo(aw[w + 1]), a1 = f16x2_lo(bw[w + 1]), a2 = f16x2_hi(aw[w + 1]), a3 = f16x2_hi(bw[w + 1]);
                mma16816<true>(s, a0, a1, a2, a3, q.z, q.w);
              }
            }
          } else {
            const int r = lane & 15;
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
              uint32_t a[4], a2[4];
              const uint4 q = lds128(qs + k * 256);
              ldsm4(a, ks + r * 256 + (((2 * k + (lane >> 4)) ^ (r & 7)) << 4));
              ldsm4(a2, ks + r * 256 + (((2 * k + 2 + (lane >> 4)) ^ (r & 7)) << 4));
              mma16816<false>(s, a[0], a[1], a[2], a[3], q.x, q.y);
              mma16816<false>(s, a2[0], a2[1], a2[2], a2[3], q.z, q.w);
            }
          }
          // s, and v's exponent x: elements 0, 1 of key g, 2, 3 of key g + 8
          const bool partly = key + 15 > p0 || (window > 0 && key <= p1 - window && key + 15 >= sinks);
          if constexpr (Q8) {
            // k's scale before the row's factor where it is below one, after it where it is above, so that nothing on the
            // way is larger than the raw product and the score are (the product of both factors may well be)
            const float low0 = scale_value(min(k0, 127u)), high0 = scale_value(max(k0, 127u));
            const float low1 = scale_value(min(k1, 127u)), high1 = scale_value(max(k1, 127u));
            s[0] = s[0] * low0 * factor.x * high0;
            s[1] = s[1] * low0 * factor.y * high0;
            s[2] = s[2] * low1 * factor.x * high1;
            s[3] = s[3] * low1 * factor.y * high1;
          } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) s[h] *= h & 1 ? factor.y : factor.x;
          }
          float x[4] = {e0, e0, e1, e1};
          if (partly) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const int j = key + g + (h >> 1) * 8, at = pos[h & 1];
              if (!(j <= at && (window == 0 || j > at - window || j < sinks))) {
                s[h] = -INFINITY;
                x[h] = 0.f;                                    // (v's scale may be NaN)
              }
            }
          }
          float y[4];                                          // what m is taken from
#pragma unroll
          for (int h = 0; h < 4; ++h) y[h] = Q8 ? s[h] + fmaxf(x[h], kLeastExponent) : s[h];
          const bool over = fmaxf(y[0], y[2]) > m[0] + (kRescaleLog2 - C::kHead) || fmaxf(y[1], y[3]) > m[1] + (kRescaleLog2 - C::kHead);
          if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float top = fmaxf(y[h], y[2 + h]);
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
              // each row by its own threshold, as `over`: another row's scores do not move its reference
              if (top > m[h] + (kRescaleLog2 - C::kHead)) {
                top += C::kHead;
                const float f = fast_exp2(m[h] - top);         // 0 where nothing was seen before
                m[h] = top;
                l[h] *= f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  o[i][h] *= f;
                  o[i][2 + h] *= f;
                }
              }
            }
          }
          float w[4];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const float mu = m[h & 1] == -INFINITY ? 0.f : m[h & 1];             // nothing seen yet: s = -inf, w = 0
            const float p = fast_exp2(s[h] - mu);
            // (v's exponent after the difference, which is small: beside a large score it would be rounded away)
            w[h] = Q8 ? fast_exp2((s[h] - mu) + x[h]) : p;
            l[h & 1] += p;
          }
          const uint32_t pb0 = transpose8(Q8 ? pack_f16x2(w[0], w[1]) : pack_bf16x2(w[0], w[1]));
          const uint32_t pb1 = transpose8(Q8 ? pack_f16x2(w[2], w[3]) : pack_bf16x2(w[2], w[3]));
          if constexpr (Q8) {
            // 16 codes (dimensions 16 g ..) of keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
            const uint32_t at = vs + 2 * t * 128 + ((g ^ (2 * t)) << 4);
            const uint4 v0 = lds128(at), v1 = lds128(at + 128), v2 = lds128(at + 8 * 128), v3 = lds128(at + 9 * 128);
            const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
            const uint32_t w2[4] = {v2.x, v2.y, v2.z, v2.w}, w3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t a = __byte_perm(w0[j], w1[j], h ? 0x7362 : 0x5140), b = __byte_perm(w2[j], w3[j], h ? 0x7362 : 0x5140);
                const uint32_t a0 = f16x2_lo(a), a1 = f16x2_hi(a), a2 = f16x2_lo(b), a3 = f16x2_hi(b);
                mma16816<true>(o[2 * j + h], a0, a1, a2, a3, pb0, pb1);
              }
            }
          } else {
            if (partly && p1 > p0) {
              // values that some rows do not see and that are not finite: zeros (added again below)
              uint8_t* v = base_ptr + (vs - base);
              bool found = false;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int row = 2 * k + (lane >> 4);
                if (!chunk_partly(p.call, key + row, p0, p1)) continue;
                uint4* at = reinterpret_cast<uint4*>(v + row * 256 + (lane & 15) * 16);
                uint4 d = *at;
                const bool a = drop_nonfinite(d.x), b = drop_nonfinite(d.y), e = drop_nonfinite(d.z), f = drop_nonfinite(d.w);
                if (a || b || e || f) {
                  *at = d;
                  found = true;
                }
              }
              bad |= __any_sync(0xffffffffu, found);
              __syncwarp();
            }
            const int r = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t a[4];
              ldsm4_t(a, vs + r * 256 + (((2 * i + ((lane >> 3) & 1)) ^ (r & 7)) << 4));
              mma16816<false>(o[i], a[0], a[1], a[2], a[3], pb0, pb1);
            }
          }
        }
        __syncwarp();                                          // the ring's place is free for the copies issued next
        ++used;
#pragma unroll
        for (int i = 0; i + 1 < C::kStages; ++i) f[i] = f[i + 1];
      }
      // ------------------------------------------------------------ the warps' parts of the segment, joined in order
      float2* s_ml = reinterpret_cast<float2*>(base_ptr + C::kMlOff);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = l[h];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (g == 0) s_ml[warp * kRows + 2 * t + h] = make_float2(m[h], x);
      }
      if (bad && lane == 0) *reinterpret_cast<volatile int*>(&s_seg[u].bad) = 1;
      const int r = s_seg[u].r, hg = s_seg[u].g, part = s_seg[u].part, rows = s_seg[u].rows, b = s_seg[u].b;
      const int q0 = s_seg[u].q0 + s_seg[u].tok0;
      // O of eight rows, [row][128] fp32 in pieces of four dimensions, goes to the place of every warp's ring
      // that its last chunk left; pieces are permuted by row so that neither side meets a bank twice. Warp w
      // then joins row w, four dimensions per lane.
      const uint32_t place = (used + C::kStages - 1) % C::kStages * (2 * C::kTile);
      auto piece_of = [](int x, int row) { return x ^ (Q8 ? row >> 1 : row & 6); };
      float* mine = reinterpret_cast<float*>(base_ptr + warp * C::kRing + place);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 2 * t + h;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (Q8) {                                // dimensions 16 g + 4 k ..
            *reinterpret_cast<float4*>(mine + row * kHd + 4 * piece_of(4 * g + k, row)) =
                make_float4(o[2 * k][h], o[2 * k][2 + h], o[2 * k + 1][h], o[2 * k + 1][2 + h]);
          } else {                                           // 32 k + g, + 8, + 16, + 24
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int dim = 32 * k + 8 * e + g;
              mine[row * kHd + 4 * piece_of(dim >> 2, row) + (dim & 3)] = o[2 * k + (e >> 1)][2 * (e & 1) + h];
            }
          }
        }
      }
      if (!meet(C::X_FULL, xph)) break;
      const int row = warp;
      float mt = -INFINITY, lt = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, s_ml[w * kRows + row].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 y = s_ml[w * kRows + row];
        const float4 x = *reinterpret_cast<const float4*>(base_ptr + w * C::kRing + place + 4 * (warp * kHd + 4 * piece_of(lane, warp)));
        if (y.y != 0.f) {                                    // else the row sees none of the warp's keys
          const float f = fast_exp2(y.x - mt);
          // in the exponent: where v's scales differ much, l is far from 1
          lt += fast_exp2(__log2f(y.y) + (y.x - mt));
          v.x += f * x.x;
          v.y += f * x.y;
          v.z += f * x.z;
          v.w += f * x.w;
        }
      }
      if (row < rows) {
        const int tok = token_of(row);
        if constexpr (!Q8) {
          if (*reinterpret_cast<volatile int*>(&s_seg[u].bad)) {
            // V values that were dropped, added to the rows that see their keys
            const int* bt = p.block_tables + (size_t)b * p.max_blocks;
            for (int c = c0; c < c1; ++c) {
              if (!chunk_mixed(p.call, c, sc, skip, p0, p1)) continue;
              for (int x = c * kChunkKeys; x < (c + 1) * kChunkKeys; ++x) {
                const int key = chunk_key(x, sc, skip);
                if (!chunk_partly(p.call, key, p0, p1) || !chunk_any(p.call, key, p0 + tok, p0 + tok)) continue;
                const int rw = chunk_row(p, r, bt[chunk_page(p, key)], key);
                if (rw < 0) continue;
                const __nv_bfloat16* y = static_cast<const __nv_bfloat16*>(p.cache_v) + ((size_t)rw * p.kv_per + hg) * kHd + 4 * lane;
                auto add = [](float& to, __nv_bfloat16 from) {
                  const float z = __bfloat162float(from);
                  if (!(fabsf(z) < INFINITY)) to += z;
                };
                add(v.x, y[0]);
                add(v.y, y[1]);
                add(v.z, y[2]);
                add(v.w, y[3]);
              }
            }
          }
        }
        if (part >= 0) {
          *reinterpret_cast<float4*>(chunk_part_o(p, part, row, 4 * lane)) = v;
          if (lane == 0) *chunk_part_ml(p, part, row) = make_float2(mt, lt);
        } else {
          const float inv = 1.0f / lt;                         // (0: all the row's scores are -inf, and the output is NaN)
          uint2 out;
          out.x = pack_bf16x2(v.x * inv, v.y * inv);
          out.y = pack_bf16x2(v.z * inv, v.w * inv);
          *reinterpret_cast<uint2*>(p.out + (size_t)r * p.sstride_out + (size_t)(q0 + tok) * p.rstride_out +
                                    (hg * gq + row - tok * gq) * kHd + 4 * lane) = out;
        }
      }
      if (!meet(C::X_EMPTY, xph)) break;
      xph ^= 1u;
      if (!ok) break;
    }
    if (!ok || segs < kBatch) break;
  }
  cp_async_wait_all();       // no copy into this CTA's shared memory may outlive it
}

template <bool Q8>
static cudaError_t launch_decode(const ChunkAttnParams& p, int grid, cudaStream_t st) {
  using C = DecodeCfg<Q8>;
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(chunk_decode_kernel<Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = programmatic(dim3(grid), kThreads, C::kSmem, st, attr);
  return cudaLaunchKernelEx(&cfg, chunk_decode_kernel<Q8>, p);
}

int chunk_decode_ctas(bool q8) { return q8 ? DecodeCfg<true>::kCtas : DecodeCfg<false>::kCtas; }

cudaError_t launch_chunk_decode(const ChunkAttnParams& p, int grid, cudaStream_t st) {
  return p.scales_k != nullptr ? launch_decode<true>(p, grid, st) : launch_decode<false>(p, grid, st);
}

}  // namespace tpl
