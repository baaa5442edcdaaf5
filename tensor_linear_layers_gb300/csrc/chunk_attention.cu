// Attention of chunks of new tokens over the paged KV cache, the cache in bf16 or in 8 bits, with
// an optional sliding window and a few first tokens that stay visible.
//
// Request b has ctx cached tokens and n new ones at positions ctx .. ctx + n - 1, all in the
// cache. The token at position p sees key j if j <= p and (no window, or j > p - window, or
// j < sinks):
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp((q . k_j - m) / sqrt(hd))
// An 8-bit cache stands for k = code * 2^(scale - 127) (kv_quant.cu), each exactly a bf16.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "chunk_walk.cuh"
#include "gemm_tc.cuh"
#include "internal.h"
#include "paged_tiles.cuh"

namespace tpl {

// ---------------------------------------------------------------- kernel
// The queries of a group of whole tokens (tokens x the q heads of one kv head) are the rows of
// 128-row tensor-core tiles; the keys that any of them sees go by in chunks of 128, read once
// from the cache for all of them:
//   S = Q K^T  (tcgen05, fp32 in tensor memory)
//   P = 2^(s c - m) as bf16, written over S (tensor memory, the A operand of P V)
//   O += P V   (tcgen05, O in tensor memory)
// with the running max m and sum l of every row in its thread's registers. Persistent, one CTA
// per SM; the chunks of all items are one line cut into equal ranges (chunk_plan.h), so decoding
// requests and chunks of prompts share a call, and few long requests still fill the GPU.
//
// MT = 1: up to 128 rows per item; S of a chunk in one of three buffers of 128 columns; two Q
// buffers. MT = 2: up to 256 rows as two tiles on the same K and V. Tensor memory holds 512
// columns, 2 x 128 of them O: S goes by halves of a chunk (64 keys), two buffers of 64 columns
// per tile.
//
//   warp 0      issues S;  warp 1 issues P V (an elected lane of a converged warp);
//   warp 2      walks the CTA's range, publishes segments and copies their queries (TMA)
//   warp 3      bf16: looks over the V rows that only some rows of the item see (below);
//               8 bits: finds the cache rows and scales of every chunk, up to three chunks ahead
//   4 warps     (bf16) copy K and V rows through the block table with 16-byte cp.async into
//               128-byte-swizzled tiles (any block size: a key's row is found on its own);
//   8 warps     (8 bits) copy the codes to buffers of their own, three tiles ahead; each thread
//               turns the codes that it copied into bf16 and stores those (four warps: 1606 us for 1048)
//   the others  softmax, a row per thread, four warps per tile; at a segment's end O / l to
//               global memory, or the unnormalised O with (m, l) to a partial slot
//
// Keys that no row of the item sees are filled with zeros, not read. In chunks with keys that
// some of its rows see and others do not (the new tokens themselves, and the keys that leave the
// window between the first and the last of them), values of V that are not finite become zero in
// shared memory, so that 0 * v stays 0 for the rows that do not see the key; the rows that see it
// get the value added at the end.
//
// What bounds it, at two tiles. bf16: 1.63 us a chunk of 128 keys x 256 rows (2048 tokens over 32 049 keys 690 us,
// 0.78 of what a large matrix product reaches; 725 to 740 where the power limit holds the clock): S by halves reads Q again for each, 48 cycles of shared memory an
// MMA for 32 of products, and the softmax of 64 keys is a chain of some 1200 cycles after it, behind which two
// buffers per tile hide most of that. (S by whole chunks, without that, takes turns with softmax and P V: 895 us.)
// 8 bits: 1.88 to 1.96 us a chunk (793 to 828 us, by box and clock); 68 % of the issue slots go to the conversion and the softmax.
// Code size counts here: all roles run at once, and with twenty warps' hot code beyond the SM's instruction cache
// every chunk fetched it again from the cache that the SMs of a GPC share (8 bits: 1019 us; the SMs of the GPC that
// has fewest ran 15 % faster). So loops that are seldom run or have time are rolled, each step of a role stands at
// one place in the code, and the warp's index is known to be uniform.
// An item costs some 3 us besides its chunks (chunk_item_cost): the drain of the last products, its output.
//
// Codes become bf16 with integer operations and one product: e4m3 is s eeee mmm with bias 7, and
// those bits put at s 0000eeee mmm0000 of a bf16 (bias 127) are the value times 2^-120, subnormal
// numbers too; a product with 2^120 and the head's scale, exact, gives the value.
namespace {
constexpr int kHd = 128;
constexpr int kTileBytes = 128 * 128 * 2;      // 128 rows x 128 bf16: two 64-column boxes
constexpr int kCodeBytes = 128 * 128;          // codes of 128 keys
constexpr int kUnitSlots = 4;
// What is known of a chunk of codes: cache rows of its keys (-1: zeros), then four factors of each, k's two
// and v's two (below), then the kv head (-1: no more chunks) and whether a second factor is not one.
constexpr int kLookBytes = 128 * 5 * 4 + 16;
constexpr float kRescaleLog2 = 8.0f;           // rescale O when the row max grows by more than this
// m is the row max and this much more, so that weights are at most 2^(8 - 17): a sum of 512 weighted
// bf16 numbers fits fp32 (any v < 2^137 / L does for L keys), and so do products with v of 2^-100
constexpr float kHeadroomLog2 = 17.0f;
constexpr uint32_t kIdescO = idesc_bf16_f32(128, 128) | kIdescBMnMajor;
constexpr int kTmemCols = 512;

template <int MT, bool Q8>
struct ChunkCfg {
  static constexpr int kCopyWarps = Q8 ? 8 : 4;
  static constexpr int kThreads = 128 + 32 * kCopyWarps + 128 * MT;
  static constexpr int kTiles = Q8 ? 3 : 5;                // K/V ring
  static constexpr int kAhead = 3;                         // tiles of codes in flight
  static constexpr int kLooks = 4;                         // chunks that are looked up
  static constexpr int kQBufs = MT == 1 ? 2 : 1;
  static constexpr int kSub = MT == 1 ? 128 : 64;          // keys of one S, softmax and P V
  static constexpr int kSubs = kChunkKeys / kSub;
  static constexpr int kSBufs = MT == 1 ? 3 : 2;           // S/P buffers of a tile
  static constexpr uint32_t kIdescS = idesc_bf16_f32(128, kSub);
  static constexpr int kRingOff = MT * kQBufs * kTileBytes;   // after Q
  static constexpr int kCodeOff = kRingOff + kTiles * kTileBytes;
  static constexpr int kLookOff = kCodeOff + (Q8 ? kAhead * kCodeBytes : 0);
  static constexpr int kBarOff = kLookOff + (Q8 ? kLooks * kLookBytes : 0);
  // registers: issuers, copies, softmax
  static constexpr int kRegs0 = 80, kRegs1 = Q8 ? (MT == 1 ? 88 : 48) : MT == 1 ? 152 : 96;
  static constexpr int kRegsS = MT == 1 ? (Q8 ? 216 : 232) : Q8 ? 152 : 168;
  static constexpr int kRegsAll = 128 * kRegs0 + 32 * kCopyWarps * kRegs1 + 128 * MT * kRegsS;
  static constexpr int kLaunchRegs = MT == 1 ? (Q8 ? 128 : 168) : Q8 ? 96 : 128;
  static_assert(kRegsAll <= kThreads * kLaunchRegs, "register split within the launch's");
  static_assert(kRegs0 <= kLaunchRegs && kRegs1 <= kLaunchRegs && kRegsS >= kLaunchRegs, "who gives registers up, and who takes them");
  // tensor memory: MT = 1: S/P at 0, 128, 256, O at 384; MT = 2: tile m S/P at 256 m and 256 m + 64, O at 256 m + 128
  static __device__ __forceinline__ uint32_t s_col(int tile, int buf) { return tile * 256 + (buf - tile * kSBufs) * kSub; }
  static __device__ __forceinline__ uint32_t o_col(int tile) { return MT == 1 ? 384 : tile * 256 + 128; }
  enum {
    Q_FULL = 0, Q_EMPTY = Q_FULL + kQBufs, FULL = Q_EMPTY + kQBufs, EMPTY = FULL + kTiles,
    S_FULL = EMPTY + kTiles,          // per S/P buffer of every tile
    P_READY = S_FULL + MT * kSBufs,
    S_FREE = P_READY + MT * kSBufs,   // its P V has completed
    O_FREE = S_FREE + MT * kSBufs,    // per tile
    LANDED = O_FREE + MT,             // bf16: a V tile to be looked over, per ring tile
    U_FULL = LANDED + kTiles, U_EMPTY = U_FULL + kUnitSlots,
    L_FULL = U_EMPTY + kUnitSlots, L_EMPTY = L_FULL + kLooks, DONE_S = L_EMPTY + kLooks, DONE_PV, NBARS
  };
  static constexpr int kMiscOff = kBarOff + 8 * NBARS;     // tensor memory address, abort flag
  static constexpr int kUnitOff = (kMiscOff + 8 + 15) / 16 * 16;
  static constexpr int kSmem = 1024 + kUnitOff + kUnitSlots * 64;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Codes 2 h and 2 h + 1 of a word as bf16, 2^-120 of their values: each code widened with its sign to 16
// bits (a byte permutation can repeat a byte's sign), times 16, and the sign's copies between taken out.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int h) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(w), "r"(h == 0 ? 0x9180 : 0xb3a2));
  return (r * 16u) & 0x87f087f0u;
}
// 2^(s - 127 + 120) of a scale byte twice as bf16; past the largest power the rest is in the second
// factor. kDropRow: 0.
constexpr uint32_t kScaleNan = 255u, kDropRow = 256u, kScaleOne = 134u;   // up to kScaleOne the second factor is one
__device__ __forceinline__ uint32_t scale_factor(uint32_t s) {
  return (s == kDropRow ? 0u : s == kScaleNan ? 0x7fc0u : min(s + 120u, 254u) << 7) * 0x10001u;
}
__device__ __forceinline__ uint32_t scale_rest(uint32_t s) {
  return (s > 134u && s < kScaleNan ? s - 7u << 7 : 0x3f80u) * 0x10001u;
}
}  // namespace

// Parts of an item that several CTAs compute, joined in the order of their keys (the same bits every time):
//   o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,  m = max_i m_i
// Where the call has many items the CTAs' warps of the same 32 rows count their parts, and the one that comes
// last joins them. Mostly that is the CTA that began the item, at the end of its range: the others are there
// then, and its own part goes into the sum from tensor memory (a kernel after this one took 13 us of a prompt's
// 135). Where it has few, whose parts are many, a kernel does (below).
__device__ __forceinline__ int chunk_part_slot(int c, int first) { return c == first ? 2 * c + 1 : 2 * c; }
// o += the part of CTA c, dimensions k to k + N - 1 of a row
template <int N>
__device__ __forceinline__ void chunk_add_part(const ChunkAttnParams& p, int slot, int row, int k, float m, float* o) {
  const float2 x = __ldcg(chunk_part_ml(p, slot, row));
  float v[N / 8][8];
#pragma unroll
  for (int i = 0; i < N / 8; ++i) ld_global_v8_cg(v[i], chunk_part_o(p, slot, row, k + 8 * i));
  if (x.y == 0.f) return;                             // the row sees no key of that part
  const float w = exp2f(x.x - m);
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] += w * v[i / 8][i % 8];
}
// In the exponent: l is far from 1 where v's scales differ much.
__device__ __forceinline__ float chunk_part_l(float m, float l, float mt) { return l == 0.f ? 0.f : exp2f(log2f(l) + (m - mt)); }
// Four rows of an item from row0 on (those past its last one repeat that), by one warp, four dimensions per lane;
// out: shard's and head's first element of the item's first token.
__device__ __forceinline__ void chunk_join_rows(const ChunkAttnParams& p, int first, int last, int row0, int rows, __nv_bfloat16* out) {
  const int lane = threadIdx.x & 31, gq = p.call.gq;
  int row[4];
  float m[4], l[4];
  float4 o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    row[j] = min(row0 + j, rows - 1);
    m[j] = -INFINITY;
    l[j] = 0.f;
    o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int c = first + lane; c <= last; c += 32)
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = fmaxf(m[j], __ldcg(chunk_part_ml(p, chunk_part_slot(c, first), row[j])).x);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], x));
#pragma unroll 2
  for (int c = first; c <= last; ++c) {
    float2 x[4];
    float4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = __ldcg(chunk_part_ml(p, chunk_part_slot(c, first), row[j]));
      v[j] = __ldcg(reinterpret_cast<const float4*>(chunk_part_o(p, chunk_part_slot(c, first), row[j], 4 * lane)));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (x[j].y == 0.f) continue;                    // the row sees no key of that part
      const float w = exp2f(x[j].x - m[j]);
      l[j] += chunk_part_l(x[j].x, x[j].y, m[j]);
      o[j].x += w * v[j].x;
      o[j].y += w * v[j].y;
      o[j].z += w * v[j].z;
      o[j].w += w * v[j].w;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (row0 + j >= rows) break;
    const float inv = 1.0f / l[j];                     // (a sum of 0: see the softmax)
    const int tok = row[j] / gq;
    uint2 y;
    y.x = pack_bf16x2(o[j].x * inv, o[j].y * inv);
    y.y = pack_bf16x2(o[j].z * inv, o[j].w * inv);
    *reinterpret_cast<uint2*>(out + (size_t)tok * p.rstride_out + (row[j] - tok * gq) * kHd + 4 * lane) = y;
  }
}
// After a part of this warp's 32 rows has been written: counted, and joined if it was the last.
__device__ __forceinline__ void chunk_join(const ChunkAttnParams& p, int first, int last, unsigned* counter, int row0, int rows, __nv_bfloat16* out) {
  __syncwarp();
  unsigned before = 0;
  if ((threadIdx.x & 31) == 0) before = atom_acq_rel_add(counter, 1);   // after every lane's part (__syncwarp)
  before = __shfl_sync(0xffffffffu, before, 0);
  __syncwarp();
  if (before != (unsigned)(last - first)) return;
  if ((threadIdx.x & 31) == 0) *counter = 0;          // as the next call needs it
#pragma unroll 1
  for (int j = 0; j < 32 && row0 + j < rows; j += 4) chunk_join_rows(p, first, last, row0 + j, rows, out);
}

template <int MT, bool Q8>
__global__ void __launch_bounds__(ChunkCfg<MT, Q8>::kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap map_q, const ChunkAttnParams p) {
  using C = ChunkCfg<MT, Q8>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw_addr);
  auto bar = [&](int b) { return base + C::kBarOff + 8u * b; };
  volatile uint32_t* s_tmem = reinterpret_cast<volatile uint32_t*>(base_ptr + C::kMiscOff);
  volatile int* s_abort = reinterpret_cast<volatile int*>(base_ptr + C::kMiscOff + 4);
  ChunkSegment* s_seg = reinterpret_cast<ChunkSegment*>(base_ptr + C::kUnitOff);
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;   // (known to be one for all lanes)
  griddep_launch_dependents();   // the grid after this one may be scheduled; it waits for this one to complete
  if (warp == 0) {
    for (int b = lane; b < C::NBARS; b += 32) {
      int count = 1;
      if (b >= C::FULL && b < C::EMPTY) count = Q8 ? C::kCopyWarps : 128;        // every copying warp or thread
      if (b >= C::P_READY && b < C::S_FREE) count = 4;                          // the tile's softmax warps
      if (b >= C::S_FREE && b < C::O_FREE) count = 2;                           // the MMAs, and their issuer
      if (b >= C::O_FREE && b < C::LANDED) count = 4;
      if (b >= C::LANDED && b < C::U_FULL) count = 128;
      if (b >= C::U_EMPTY && b < C::L_FULL) count = 3 + (Q8 ? 0 : 4) + 4 * MT;   // issuers, warp 3, bf16 copies, softmax warps
      if (b >= C::L_FULL && b < C::L_EMPTY) count = 32;
      if (b >= C::L_EMPTY && b < C::DONE_S) count = C::kCopyWarps;
      mbar_init(bar(b), count);
    }
    if (lane == 0) *s_abort = 0;
    fence_barrier_init();
  }
  if (threadIdx.x == 64) prefetch_tensormap(&map_q);
  if (warp == 1) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(s_tmem)), kTmemCols);
    tmem_relinquish();
  }
  // the set-up above may overlap the grid before (programmatic launch); nothing that grid
  // wrote is read before this
  griddep_wait();
  const int gq = p.call.gq;                         // q heads of a kv head
  const int sc = chunk_sinks(p.call), window = p.call.window, sinks = p.call.sinks;
  ChunkWalk<false> walk;                                   // warp 2's; the first requests' counts load beside the set-up
  if (warp == 2) walk.load(p, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // a value that is one for the whole warp, known as such to the compiler (uniform registers, no divergent branches)
  auto uni = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  const uint32_t tmem_base = (uint32_t)uni((int)*s_tmem);
  const unsigned long long timeout = p.timeout_ns;
  // row / gq as a product: 2^32 / gq rounded up is off by less than 1, and row * gq < 2^32
  const unsigned gq_magic = 0xffffffffu / (unsigned)gq + 1u;
  auto token_of = [&](int row) { return gq == 1 ? row : (int)__umulhi((unsigned)row, gq_magic); };
  bool ok = true;
  // a wait of a whole warp
  auto wait = [&](int b, uint32_t ph) -> bool {
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
  // the next segment's slot, or -1 at the end
  int nu = 0;
  auto next_segment = [&]() -> int {
    const int slot = nu % kUnitSlots;
    if (!wait(C::U_FULL + slot, (nu / kUnitSlots) & 1)) return -1;
    ++nu;
    return uni(s_seg[slot].b) < 0 ? -1 : slot;
  };
  auto release_segment = [&](int slot) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::U_EMPTY + slot));
  };
  auto partly_seen = [&](int key, int p0, int p1) { return chunk_partly(p.call, key, p0, p1); };
  auto mixed_chunk = [&](int j, int skip, int p0, int p1) { return chunk_mixed(p.call, j, sc, skip, p0, p1); };
  auto any_sees = [&](int key, int p0, int p1) { return chunk_any(p.call, key, p0, p1); };
  auto cache_row = [&](int r, int blk, int key) { return chunk_row(p, r, blk, key); };

  if (warp < 4) {
    regs_dec<C::kRegs0>();
    if (warp == 0) {
      // ------------------------------------------------------------ S = Q K^T
      const uint64_t q_desc = smem_desc_k128(base);
      const uint64_t k_desc = smem_desc_k128(base + C::kRingOff);
      constexpr uint64_t kTileDesc = kTileBytes >> 4;
      int ring = 0;                                   // tile of the next K
      uint32_t ring_ph = 0;
      int cnt[MT] = {};                               // S of each tile so far
      for (int seg_no = 0;; ++seg_no) {
        const int slot = next_segment();
        if (slot < 0) break;
        const int n = uni(s_seg[slot].c1 - s_seg[slot].c0), rows = uni(s_seg[slot].rows);
        release_segment(slot);
        const int qb = seg_no % C::kQBufs;
        if (!wait(C::Q_FULL + qb, (seg_no / C::kQBufs) & 1)) break;
        for (int j = 0; j < n && ok; ++j) {
          // The first S of the chunk waits for its buffer before it waits for K: that P V is done, so the
          // V that the ring's tile held before, handed on late by warp 3, has been counted, and the next
          // phase of the tile's barrier is this K's (two phases ahead would look like the one before).
          if (!wait(C::S_FREE + cnt[0] % C::kSBufs, ((cnt[0] / C::kSBufs) & 1) ^ 1)) break;
          if (!wait(C::FULL + ring, ring_ph)) break;
          fence_async_proxy();
#pragma unroll(Q8 ? 1 : C::kSubs)                       // (code size)
          for (int h = 0; h < C::kSubs; ++h) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              if (m * 128 >= rows) break;
              const int buf = m * C::kSBufs + cnt[m] % C::kSBufs;
              if ((h > 0 || m > 0) && !wait(C::S_FREE + buf, ((cnt[m] / C::kSBufs) & 1) ^ 1)) break;
              ++cnt[m];
              tc_fence_after();
              if (elect_one()) {
                const uint32_t d = tmem_base + C::s_col(m, buf);
                // half h of the chunk: 64 K rows of 128 bytes further
                const uint64_t qd = q_desc + qb * MT * kTileDesc + m * (kTileDesc / 2), kd = k_desc + ring * kTileDesc + h * ((64 * 128) >> 4);
                tc_mma_bf16_c<false>(d, qd, kd, C::kIdescS);
#pragma unroll
                for (int k = 1; k < 8; ++k) {
                  const int box = (k >> 2) * (kTileBytes / 2), in = (k & 3) * 32;
                  tc_mma_bf16_c<true>(d, qd + (uint64_t)((MT * box + in) >> 4), kd + (uint64_t)((box + in) >> 4), C::kIdescS);
                }
                tc_commit(bar(C::S_FULL + buf));
              }
              __syncwarp();
            }
            if (!ok) break;
          }
          if (!ok) break;
          if (elect_one()) {
            tc_commit(bar(C::EMPTY + ring));
            if (j == n - 1) tc_commit(bar(C::Q_EMPTY + qb));
          }
          __syncwarp();
          ring += 2;
          if (ring >= C::kTiles) {
            ring -= C::kTiles;
            ring_ph ^= 1u;
          }
        }
        if (!ok) break;
      }
      if (elect_one()) tc_commit(bar(C::DONE_S));
      __syncwarp();
      mbar_wait_bounded(bar(C::DONE_S), 0, nullptr, kTeardownNs);
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ O += P V
      const uint64_t v_desc = smem_desc_mn128(base + C::kRingOff, kTileBytes / 2);
      constexpr uint64_t kTileDesc = kTileBytes >> 4;
      int ring = 1;                                   // tile of the next V
      uint32_t ring_ph = 0;
      int cnt[MT] = {}, segs[MT] = {};
      for (;;) {
        const int slot = next_segment();
        if (slot < 0) break;
        const int n = uni(s_seg[slot].c1 - s_seg[slot].c0), rows = uni(s_seg[slot].rows);
        release_segment(slot);
        for (int j = 0; j < n && ok; ++j) {
          if (!wait(C::FULL + ring, ring_ph)) break;
          fence_async_proxy();
#pragma unroll(Q8 ? 1 : C::kSubs)                       // (code size)
          for (int h = 0; h < C::kSubs; ++h) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              if (m * 128 >= rows) break;
              const int buf = m * C::kSBufs + cnt[m] % C::kSBufs;
              if (!wait(C::P_READY + buf, (cnt[m] / C::kSBufs) & 1)) break;
              const bool first = j == 0 && h == 0;
              if (first && !wait(C::O_FREE + m, (segs[m]++ & 1) ^ 1)) break;
              ++cnt[m];
              tc_fence_after();
              if (elect_one()) {
                const uint32_t pa = tmem_base + C::s_col(m, buf), d = tmem_base + C::o_col(m);
                const uint64_t vd = v_desc + ring * kTileDesc + h * ((64 * 128) >> 4);
                // 16 keys = two 8-row groups of V (2048 B) and 8 columns of P
                if (first)
                  tc_mma_bf16_ta_c<false>(d, pa, vd, kIdescO);
                else
                  tc_mma_bf16_ta_c<true>(d, pa, vd, kIdescO);
#pragma unroll
                for (int k = 1; k < C::kSub / 16; ++k)
                  tc_mma_bf16_ta_c<true>(d, pa + k * 8, vd + (uint64_t)(k * (2048 >> 4)), kIdescO);
                tc_commit(bar(C::S_FREE + buf));
                mbar_arrive(bar(C::S_FREE + buf));    // carries the `bad` mark to the softmax
              }
              __syncwarp();
            }
            if (!ok) break;
          }
          if (!ok) break;
          if (elect_one()) tc_commit(bar(C::EMPTY + ring));
          __syncwarp();
          ring += 2;
          if (ring >= C::kTiles) {
            ring -= C::kTiles;
            ring_ph ^= 1u;
          }
        }
        if (!ok) break;
      }
      if (elect_one()) tc_commit(bar(C::DONE_PV));
      __syncwarp();
      mbar_wait_bounded(bar(C::DONE_PV), 0, nullptr, kTeardownNs);
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------------------ segments
      walk.start(p, lane);
      const uint64_t pol = policy_evict_normal();
      int u = 0;
      for (;; ++u) {
        const int slot = u % kUnitSlots;
        if (!wait(C::U_EMPTY + slot, ((u / kUnitSlots) & 1) ^ 1)) break;
        const ChunkSegment s = walk.next(p, lane);
        if (lane == 0) {
          s_seg[slot] = s;
          mbar_arrive(bar(C::U_FULL + slot));
        }
        __syncwarp();
        if (s.b < 0) break;
        // The segment's queries, once those that the buffer held are no longer read: a box of 64 dimensions x the heads
        // x the group's tokens is the tiles' rows in order. What it holds past the item's tokens (other tokens, or
        // zeros past the last) only reaches rows of S and O of its own.
        const int qb = u % C::kQBufs, head = s.g * gq, tok = s.q0 + s.tok0;
        if (elect_one()) {
          tma_prefetch_4d(&map_q, 0, head, tok, s.r);
          tma_prefetch_4d(&map_q, 64, head, tok, s.r);
        }
        __syncwarp();
        if (!wait(C::Q_EMPTY + qb, ((u / C::kQBufs) & 1) ^ 1)) break;
        if (elect_one()) {
          const uint32_t dst = base + qb * MT * kTileBytes;
          mbar_arrive_expect_tx(bar(C::Q_FULL + qb), 2 * p.q_box_rows * 128);
          tma_load_4d(dst, &map_q, bar(C::Q_FULL + qb), 0, head, tok, s.r, pol);
          tma_load_4d(dst + MT * (kTileBytes / 2), &map_q, bar(C::Q_FULL + qb), 64, head, tok, s.r, pol);
        }
        __syncwarp();
      }
      // no copy into this CTA's shared memory may outlive it
      for (int i = max(u - C::kQBufs, 0); i < u; ++i)
        mbar_wait_bounded(bar(C::Q_FULL + i % C::kQBufs), (i / C::kQBufs) & 1, nullptr, kTeardownNs);
      __syncwarp();
    } else if (Q8) {
      // ------------------------------------------------------------ rows and scales of the chunks
      // A lane has four keys on end, of one page where pages are multiples of four. The chunk's factors follow
      // one chunk later, when its scale bytes have come.
      const bool quads = (p.block_size & 3) == 0;
      int n = 0;                                      // chunks begun
      uint32_t ks[4] = {}, vs[4] = {};                // scale bytes of the last one
      unsigned part = 0;                              // bit i: its key 4 lane + i is only partly seen
      int at = -1, seg = 0;                           // its place, and its segment's slot
      auto hand_on = [&]() {
        if (at < 0) return;
        const uint32_t look = base + C::kLookOff + at * kLookBytes;
        const uint32_t top = max(max(max(ks[0], ks[1]), max(ks[2], ks[3])), max(max(vs[0], vs[1]), max(vs[2], vs[3])));
        const bool large = __any_sync(0xffffffffu, top > kScaleOne);
        if (large) {
          bool bad = false;
#pragma unroll
          for (int i = 0; i < 4; ++i)                 // a V row that is not finite and only partly seen: zeros, and the mark
            if ((part >> i & 1u) && vs[i] == kScaleNan) {
              vs[i] = kDropRow;
              bad = true;
            }
          if (bad) *reinterpret_cast<volatile int*>(&s_seg[seg].bad) = 1;
          sts128(look + 256 * 4 + 16 * lane, scale_rest(ks[0]), scale_rest(ks[1]), scale_rest(ks[2]), scale_rest(ks[3]));
          sts128(look + 512 * 4 + 16 * lane, scale_rest(vs[0]), scale_rest(vs[1]), scale_rest(vs[2]), scale_rest(vs[3]));
          sts128(look + 128 * 4 + 16 * lane, scale_factor(ks[0]), scale_factor(ks[1]), scale_factor(ks[2]), scale_factor(ks[3]));
          sts128(look + 384 * 4 + 16 * lane, scale_factor(vs[0]), scale_factor(vs[1]), scale_factor(vs[2]), scale_factor(vs[3]));
        } else {                                      // every power of two in range: its bf16 bits twice
          constexpr uint32_t kTwice = 0x00800080u;
          sts128(look + 128 * 4 + 16 * lane, (ks[0] + 120u) * kTwice, (ks[1] + 120u) * kTwice, (ks[2] + 120u) * kTwice, (ks[3] + 120u) * kTwice);
          sts128(look + 384 * 4 + 16 * lane, (vs[0] + 120u) * kTwice, (vs[1] + 120u) * kTwice, (vs[2] + 120u) * kTwice, (vs[3] + 120u) * kTwice);
        }
        if (lane == 0) *reinterpret_cast<uint32_t*>(base_ptr + C::kLookOff + at * kLookBytes + 641 * 4) = large ? 1u : 0u;
        mbar_arrive(bar(C::L_FULL + at));
      };
      for (;;) {
        const int slot = next_segment();
        if (slot < 0) break;
        const int r = s_seg[slot].r, g = s_seg[slot].g, c1 = s_seg[slot].c1, p0 = s_seg[slot].p0, p1 = s_seg[slot].p1, skip = s_seg[slot].skip;
        const int* bt = p.block_tables + (size_t)s_seg[slot].b * p.max_blocks;
        // every step at one place in the code: a turn before the first chunk looks up its blocks, one after the last
        // hands that on
        const int c0 = s_seg[slot].c0;
        int key = 0, blk[4] = {};
        for (int c = c0 - 1;; ++c) {
          const bool here = c >= c0 && c < c1;
          const int place = n % C::kLooks;
          int row[4] = {-1, -1, -1, -1};              // cache rows of the lane's keys (-1: zeros)
          unsigned mixed = 0;
          if (here) {
            if (!wait(C::L_EMPTY + place, ((n / C::kLooks) & 1) ^ 1)) break;
            const int first = cache_row(r, blk[0], key);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (any_sees(key + i, p0, p1)) {
                row[i] = quads ? (first < 0 ? -1 : first + i) : cache_row(r, blk[i], key + i);
                if (row[i] < 0) atomicExch(p.status, kChunkStatusShape);
              }
            sts128(base + C::kLookOff + place * kLookBytes + 16 * lane, row[0], row[1], row[2], row[3]);
            if (lane == 0) *reinterpret_cast<int*>(base_ptr + C::kLookOff + place * kLookBytes + 640 * 4) = g;
            if (mixed_chunk(c, skip, p0, p1))
#pragma unroll
              for (int i = 0; i < 4; ++i) mixed |= partly_seen(key + i, p0, p1) ? 1u << i : 0u;
          }
          if (c + 1 < c1) {
            key = chunk_key((c + 1) * kChunkKeys + 4 * lane, sc, skip);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (i > 0 && quads) break;              // one block for the four
              const bool seen = key + i <= p1 && (window == 0 || key + (quads ? 3 : i) > p0 - window || key + i < sinks);
              blk[i] = seen ? bt[chunk_page(p, key + i)] : 0;
            }
          }
          hand_on();                                  // (the mark belongs to this segment)
          at = -1;
          if (c == c1) break;
          if (here) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const size_t x = (size_t)(unsigned)max(row[i], 0) * (unsigned)p.kv_per + g;
              ks[i] = row[i] >= 0 ? p.scales_k[x] : 127u;
              vs[i] = row[i] >= 0 ? p.scales_v[x] : 127u;
            }
            part = mixed;
            at = place;
            seg = slot;
            ++n;
          }
        }
        if (!ok) break;
        release_segment(slot);
      }
      if (ok) {                                       // no more chunks
        const int place = n % C::kLooks;
        if (wait(C::L_EMPTY + place, ((n / C::kLooks) & 1) ^ 1)) {
          if (lane == 0) *reinterpret_cast<int*>(base_ptr + C::kLookOff + place * kLookBytes + 640 * 4) = -1;
          mbar_arrive(bar(C::L_FULL + place));
        }
      }
    } else {
      // ------------------------------------------------------------ V that only some rows see
      int ring = 1;                                   // tile of the next V
      uint32_t phases = 0;                            // bit i: phase of LANDED + i
      for (;;) {
        const int slot = next_segment();
        if (slot < 0) break;
        const int c0 = s_seg[slot].c0, c1 = s_seg[slot].c1, p0 = s_seg[slot].p0, p1 = s_seg[slot].p1, skip = s_seg[slot].skip;
        bool bad = false;
        for (int c = c0; c < c1; ++c) {
          if (mixed_chunk(c, skip, p0, p1)) {
            if (!wait(C::LANDED + ring, phases >> ring & 1u)) break;
            phases ^= 1u << ring;
            // a row is 8 pieces of 16 bytes in each of two boxes, in any order; a lane has piece `piece` of box `box`
            // of rows lane / 16, + 2, ..: of those that are partly seen the largest size first, as whole numbers
            // (without the sign, bf16 bits are ordered so, infinity and NaN last)
            const int x0 = c * kChunkKeys, k0 = x0 + skip, box = (lane >> 3) & 1, piece = lane & 7;
            uint8_t* v = base_ptr + C::kRingOff + ring * kTileBytes + box * (kTileBytes / 2) + piece * 16;
            // rows [0, a1) are before the window of the item's last token (or sinks), rows [b0, 128) after its first token
            const int a1 = window > 0 ? min(max(p1 - window + 1 - k0, 0), kChunkKeys) : 0, b0 = max(p0 + 1 - k0, 0);
            unsigned top = 0u;
#pragma unroll 8
            for (int row = lane >> 4; row < a1; row += 2) {
              const uint4 d = *reinterpret_cast<const uint4*>(v + row * 128);
              top = __vmaxu2(top, __vmaxu2(__vmaxu2(d.x & 0x7fff7fffu, d.y & 0x7fff7fffu), __vmaxu2(d.z & 0x7fff7fffu, d.w & 0x7fff7fffu)));
            }
            // (the rows past the last token are zeros)
#pragma unroll 8
            for (int row = b0 + (lane >> 4); row < min(p1 + 1 - k0, kChunkKeys); row += 2) {
              const uint4 d = *reinterpret_cast<const uint4*>(v + row * 128);
              top = __vmaxu2(top, __vmaxu2(__vmaxu2(d.x & 0x7fff7fffu, d.y & 0x7fff7fffu), __vmaxu2(d.z & 0x7fff7fffu, d.w & 0x7fff7fffu)));
            }
            if (__any_sync(0xffffffffu, (top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u)) {
              for (int row = lane >> 4; row < kChunkKeys; row += 2) {
                if (!partly_seen(chunk_key(x0 + row, sc, skip), p0, p1)) continue;
                uint4* q = reinterpret_cast<uint4*>(v + row * 128);
                uint4 d = *q;
                const bool x = drop_nonfinite(d.x), y = drop_nonfinite(d.y), z = drop_nonfinite(d.z), w = drop_nonfinite(d.w);
                if (x || y || z || w) {
                  *q = d;
                  bad = true;
                }
              }
            }
            bad = __any_sync(0xffffffffu, bad);
            __syncwarp();                             // every lane's stores, before lane 0 hands the tile on
            if (lane == 0) {
              if (bad) *reinterpret_cast<volatile int*>(&s_seg[slot].bad) = 1;
              mbar_arrive_n(bar(C::FULL + ring), 128);   // for the copying threads
            }
          }
          ring += 2;
          if (ring >= C::kTiles) ring -= C::kTiles;
        }
        if (!ok) break;
        release_segment(slot);
      }
    }
  } else if (warp < 4 + C::kCopyWarps) {
    // ------------------------------------------------------------ copies
    regs_dec<C::kRegs1>();
    const int w4 = warp - 4;
    // the cache is read once a call by one item (evicted first: 8 requests of 30 new tokens each over 4000 keys 50.2 us,
    // 52.4 without, 32 of 4 over 2000 keys 51.8 and 54.3) or by its groups of rows
    const uint64_t pol = p.call.max_query_len > p.call.tg ? policy_evict_normal() : policy_evict_first();
    int ring = 0;
    uint32_t ring_ph = 0;
    auto advance = [&]() {
      if (++ring == C::kTiles) {
        ring = 0;
        ring_ph ^= 1u;
      }
    };
    if constexpr (!Q8) {
      const int c16 = lane & 15, half = lane >> 4;
      // this thread copies 16-byte piece c16 of rows 2 w4 + half + 8 k; lane i of the warp finds the
      // cache row of row 8 (i / 2) + 2 w4 + i % 2
      const int row_of = 2 * w4 + half, my_row = 8 * (lane >> 1) + 2 * w4 + (lane & 1);
      const uint32_t dst0 = (c16 >> 3) * (kTileBytes / 2) + row_of * 128 + (((c16 & 7) ^ (row_of & 7)) << 4);
      const __nv_bfloat16* cache_k = static_cast<const __nv_bfloat16*>(p.cache_k);
      const __nv_bfloat16* cache_v = static_cast<const __nv_bfloat16*>(p.cache_v);
      for (;;) {
        const int slot = next_segment();
        if (slot < 0) break;
        const ChunkSegment s = s_seg[slot];
        const int* bt = p.block_tables + (size_t)s.b * p.max_blocks;
        auto block_of = [&](int c) -> int {            // block id of this lane's key of chunk c
          const int key = chunk_key(c * kChunkKeys + my_row, sc, s.skip);
          return any_sees(key, s.p0, s.p1) ? bt[chunk_page(p, key)] : 0;
        };
        int blk = block_of(s.c0);
        for (int c = s.c0; c < s.c1 && ok; ++c) {
          const int key = chunk_key(c * kChunkKeys + my_row, sc, s.skip);
          int row = -1;                                // cache row of this lane's key (-1: zeros)
          if (any_sees(key, s.p0, s.p1)) {
            row = cache_row(s.r, blk, key);
            if (row < 0) atomicExch(p.status, kChunkStatusShape);
          }
          if (c + 1 < s.c1) blk = block_of(c + 1);
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            if (!wait(C::EMPTY + ring, ring_ph ^ 1)) break;
            const __nv_bfloat16* src = (kv ? cache_v : cache_k) + s.g * kHd + c16 * 8;
            const uint32_t dst = base + C::kRingOff + ring * kTileBytes + dst0;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int rw = __shfl_sync(0xffffffffu, row, 2 * k + half);
              cp_async16(dst + k * 1024, src + (size_t)max(rw, 0) * p.kv_per * kHd, rw >= 0 ? 16 : 0, pol);
            }
            cp_async_arrive(bar((kv == 1 && mixed_chunk(c, s.skip, s.p0, s.p1) ? C::LANDED : C::FULL) + ring));
            advance();
            if (!ok) break;
          }
        }
        if (!ok) break;
        release_segment(slot);
      }
    } else {
      // this warp has rows 16 w4 + (0 .. 15) of a tile; the thread copies and converts 16-byte piece c8 of
      // rows 16 w4 + 4 k + sub. Eight lanes have four pieces of one box of two rows, which they write to
      // eight different groups of banks.
      const int c8 = (lane & 3) | (lane >> 3 & 1) << 2, sub = (lane >> 2 & 1) | lane >> 4 << 1;
      const uint8_t* cache_k = static_cast<const uint8_t*>(p.cache_k) + c8 * 16;
      const uint8_t* cache_v = static_cast<const uint8_t*>(p.cache_v) + c8 * 16;
      const uint32_t raw = base + C::kCodeOff + (threadIdx.x - 128) * 16;    // + tile, + 4096 k: read by this thread alone
      const uint32_t looks = base + C::kLookOff + (16 * w4 + sub) * 4;
      const unsigned stride = (unsigned)(p.kv_per * kHd);
      // tiles K0 V0 K1 V1 ..: copied, and converted kAhead later
      int issued = 0, converted = 0, last = -1;       // last: tiles in all, once known
      bool more = true;
      auto issue = [&]() {
        const int c = issued >> 1, place = c % C::kLooks;
        if (more && (issued & 1) == 0) {
          if (!wait(C::L_FULL + place, (c / C::kLooks) & 1)) return;
          more = (int)lds32(base + C::kLookOff + place * kLookBytes + 640 * 4) >= 0;
          if (!more) last = issued;
        }
        if (more) {
          const uint32_t look = looks + place * kLookBytes;
          const uint8_t* src = (issued & 1 ? cache_v : cache_k) + (size_t)lds32(base + C::kLookOff + place * kLookBytes + 640 * 4) * kHd;
          const uint32_t dst = raw + (issued % C::kAhead) * kCodeBytes;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int rw = (int)lds32(look + 16 * k);
            cp_async16(dst + k * 4096, src + (size_t)(unsigned)max(rw, 0) * stride, rw >= 0 ? 16 : 0, pol);
          }
        }
        cp_async_commit();
        ++issued;
      };
      for (;;) {
        issue();
        if (!ok) break;
        if (issued < C::kAhead) continue;
        if (converted == last) break;
        const int c = converted >> 1, place = c % C::kLooks;
        cp_async_wait<C::kAhead - 1>();
        const uint32_t look = looks + place * kLookBytes + (converted & 1 ? 384 : 128) * 4;
        const uint32_t src = raw + (converted % C::kAhead) * kCodeBytes;
        uint4 w[4];
        uint32_t f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[k] = lds128(src + k * 4096);
          f[k] = lds32(look + 16 * k);
        }
        const bool large = lds32(base + C::kLookOff + place * kLookBytes + 641 * 4) != 0u;
        if (!wait(C::EMPTY + ring, ring_ph ^ 1)) break;
        // the piece's two halves: 16-byte chunks 2 c8 and 2 c8 + 1 of the row's sixteen; row & 7 is 4 (k & 1) + sub
        const uint32_t dst = base + C::kRingOff + ring * kTileBytes + (c8 >> 2) * (kTileBytes / 2) + (16 * w4 + sub) * 128;
        const uint32_t even = ((2 * (c8 & 3)) ^ sub) << 4, odd = ((2 * (c8 & 3) + 1) ^ sub) << 4;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t x[8] = {code_pair(w[k].x, 0), code_pair(w[k].x, 1), code_pair(w[k].y, 0), code_pair(w[k].y, 1),
                           code_pair(w[k].z, 0), code_pair(w[k].z, 1), code_pair(w[k].w, 0), code_pair(w[k].w, 1)};
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = mul_bf16x2(x[i], f[k]);
          if (large) {
            const uint32_t rest = lds32(look + 512 + 16 * k);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = mul_bf16x2(x[i], rest);
          }
          const uint32_t to = dst + 4 * k * 128, flip = (k & 1) << 6;
          sts128(to + (even ^ flip), x[0], x[1], x[2], x[3]);
          sts128(to + (odd ^ flip), x[4], x[5], x[6], x[7]);
        }
        fence_async_proxy();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(C::FULL + ring));
          if (converted & 1) mbar_arrive(bar(C::L_EMPTY + place));
        }
        advance();
        ++converted;
      }
    }
    cp_async_wait_all();       // no copy into this CTA's shared memory may outlive it
  } else {
    // ------------------------------------------------------------ softmax
    regs_inc<C::kRegsS>();
    const int tile = (warp - 4 - C::kCopyWarps) >> 2, q4 = warp & 3;
    const int row = tile * 128 + q4 * 32 + lane;      // row of the item; tensor-memory lane row % 128
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(q4 * 32) << 16);
    const float c = p.scale_log2;
    int cnt = 0;
    // The last P V of this tile, known by its own buffer: the issuer arrives there again only
    // after this warp has written the P that comes kSBufs later.
    auto wait_last_pv = [&]() -> bool {
      return wait(C::S_FREE + tile * C::kSBufs + (cnt - 1) % C::kSBufs, ((cnt - 1) / C::kSBufs) & 1);
    };
    float s[C::kSub];
    for (;;) {
      const int slot = next_segment();
      if (slot < 0) break;
      const int c0 = s_seg[slot].c0, c1 = s_seg[slot].c1, rows = s_seg[slot].rows;
      if (tile * 128 >= rows) {
        release_segment(slot);
        continue;
      }
      const int p0 = s_seg[slot].p0, p1 = s_seg[slot].p1, skip = s_seg[slot].skip;
      const bool idle = tile * 128 + q4 * 32 >= rows;  // no row of this warp
      const int tok = token_of(min(row, rows - 1)), pos = p0 + tok;
      float m = -INFINITY, l = 0.f;
      for (int j = c0 * C::kSubs; j < c1 * C::kSubs; ++j) {
        const int buf = tile * C::kSBufs + cnt % C::kSBufs;
        if (!wait(C::S_FULL + buf, (cnt / C::kSBufs) & 1)) break;
        if (!idle) {
          tc_fence_after();
          const uint32_t sa = lane_addr + C::s_col(tile, buf);
#pragma unroll
          for (int k = 0; k < C::kSub; k += 32) tmem_ld32(sa + k, s + k);
          tc_wait_ld();
          const int x = j * C::kSub;                  // the item's keys x, x + 1 ..
          // those that not all of its tokens see: the row's mask
          if (__builtin_expect(chunk_masked(p.call, x, C::kSub, sc, skip, p0, p1), 0)) {
#pragma unroll
            for (int w = 0; w < C::kSub / 32; ++w) {
              const unsigned bits = chunk_item_sees(x + 32 * w, sc, skip, pos, window, sinks);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(bits >> i & 1u)) s[32 * w + i] = -INFINITY;
            }
          }
          float mk[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) mk[i] = fmaxf(s[i], s[8 + i]);
#pragma unroll
          for (int k = 16; k < C::kSub; k += 16)
#pragma unroll
            for (int i = 0; i < 8; ++i) mk[i] = fmax3(mk[i], s[k + i], s[k + 8 + i]);
          const float mx = fmaf(c, fmax3(fmax3(mk[0], mk[1], mk[2]), fmax3(mk[3], mk[4], mk[5]), fmaxf(mk[6], mk[7])), kHeadroomLog2);
          if (j == c0 * C::kSubs) {
            m = mx;                                   // the first P V overwrites O
          } else if (__any_sync(0xffffffffu, mx > m + kRescaleLog2)) {
            // the warp rescales together, every row by its own factor (1 where the max held);
            // a row that saw nothing so far (m = -inf) has O = 0 and l = 0
            float f = 1.0f;
            if (mx > m + kRescaleLog2) {
              f = fast_exp2(m - mx);
              l *= f;
              m = mx;
            }
            if (!wait_last_pv()) break;
            tc_fence_after();
            float o[32];
#pragma unroll(Q8 ? 1 : 4)                            // (see above: code size)
            for (int k = 0; k < 128; k += 32) {
              tmem_ld32(lane_addr + C::o_col(tile) + k, o);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= f;
              tmem_st32(lane_addr + C::o_col(tile) + k, o);
            }
          }
          // P = 2^(s c - m) as bf16 pairs into the first half of the buffer's columns (the rounding:
          // the tensor core's A operand shares V's type; at most 2^-8 of a weight)
          const float mu = m == -INFINITY ? 0.f : m;  // nothing seen yet: every s is -inf, p = 0
          const uint64_t c2 = f32x2_pack(c, c), nm2 = f32x2_pack(-mu, -mu);
          uint64_t lk[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int h = 0; h < C::kSub / 64; ++h) {
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float x0, x1;
              f32x2_unpack(f32x2_fma(f32x2_pack(s[h * 64 + 2 * i], s[h * 64 + 2 * i + 1]), c2, nm2), x0, x1);
              const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
              lk[i & 3] = f32x2_add(lk[i & 3], f32x2_pack(e0, e1));
              pk[i] = pack_bf16x2(e0, e1);
            }
            tmem_st32(sa + h * 32, reinterpret_cast<const float*>(pk));
          }
          float la[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) f32x2_unpack(lk[i], la[2 * i], la[2 * i + 1]);
          l += ((la[0] + la[1]) + (la[2] + la[3])) + ((la[4] + la[5]) + (la[6] + la[7]));
          tc_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::P_READY + buf));
        ++cnt;
      }
      if (!ok) break;
      // a part of an item, and whether the other ones are there already
      const int part = uni(s_seg[slot].part), first = uni(s_seg[slot].first), last = uni(s_seg[slot].last);
      unsigned* counter = p.counters + first * 8 + tile * 4 + q4;
      bool join = false;
      if (part >= 0 && p.counters != nullptr && first == (int)blockIdx.x && last - first < 8 && !idle) {
        unsigned n = 0;
        if (lane == 0) n = ld_acquire(counter);
        join = uni((int)n) == last - first;
        __syncwarp();
      }
      float mt = m, lt = l;
      if (join) {
        if (lane == 0) *counter = 0;                  // as the next call needs it
        const int at = min(row, rows - 1);
        for (int c = first + 1; c <= last; ++c) mt = fmaxf(mt, __ldcg(chunk_part_ml(p, 2 * c, at)).x);
        lt = chunk_part_l(m, l, mt);
        for (int c = first + 1; c <= last; ++c) {
          const float2 x = __ldcg(chunk_part_ml(p, 2 * c, at));
          lt += chunk_part_l(x.x, x.y, mt);
        }
      }
      if (!wait_last_pv()) break;
      if (!idle) {
        tc_fence_after();
        const int bad = *reinterpret_cast<volatile int*>(&s_seg[slot].bad);
        const int r = s_seg[slot].r, g = s_seg[slot].g, b = s_seg[slot].b;
        // A token sees itself at least: a sum of 0 is a row whose scores are all -inf, and 0 * inf gives the NaN that
        // its softmax is. (Unused for a part that another joins, whose sum may well be 0.)
        const float inv = 1.0f / lt;
        __nv_bfloat16* dst = p.out + (size_t)r * p.sstride_out +
                             (size_t)(s_seg[slot].q0 + s_seg[slot].tok0 + tok) * p.rstride_out + (g * gq + row - tok * gq) * kHd;
        // (32 dimensions at a time, not unrolled: what this code costs most is the fetch of its instructions)
#pragma unroll 1
        for (int k = 0; k < 128; k += 32) {
          __syncwarp();
          tmem_ld32(lane_addr + C::o_col(tile) + k, s);
          tc_wait_ld();
          if (bad && row < rows) {
            // V values that were dropped, added to the rows that see their keys
            const int* bt = p.block_tables + (size_t)b * p.max_blocks;
            for (int j = c0; j < c1; ++j) {
              if (!mixed_chunk(j, skip, p0, p1)) continue;
              for (int x = j * kChunkKeys; x < (j + 1) * kChunkKeys; ++x) {
                const int key = chunk_key(x, sc, skip);
                if (!partly_seen(key, p0, p1) || !any_sees(key, pos, pos)) continue;
                const int rw = cache_row(r, bt[chunk_page(p, key)], key);
                if (rw < 0) continue;
                const size_t at = (size_t)rw * p.kv_per + g;
                if constexpr (Q8) {
                  if (p.scales_v[at] != kScaleNan) continue;
#pragma unroll
                  for (int i = 0; i < 32; ++i) s[i] = __int_as_float(0x7fffffff);
                } else {
                  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.cache_v) + at * kHd + k;
#pragma unroll
                  for (int i = 0; i < 32; ++i) {
                    const float x = __bfloat162float(v[i]);
                    if (!(fabsf(x) < INFINITY)) s[i] += x;
                  }
                }
              }
            }
          }
          if (join) {
            const float w = l == 0.f ? 0.f : exp2f(m - mt);
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] = l == 0.f ? 0.f : w * s[i];
            for (int c = first + 1; c <= last; ++c) chunk_add_part<32>(p, 2 * c, min(row, rows - 1), k, mt, s);
          }
          if (row < rows) {
            if (part >= 0 && !join) {
#pragma unroll
              for (int i = 0; i < 32; i += 8)
                st_global_v8(chunk_part_o(p, part, row, k + i), *reinterpret_cast<const uint32_t(*)[8]>(s + i));
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 16) {
                uint32_t v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = pack_bf16x2(s[i + 2 * e] * inv, s[i + 2 * e + 1] * inv);
                if (p.out_align32) {
                  st_global_v8(dst + k + i, v);
                } else {
                  *reinterpret_cast<uint4*>(dst + k + i) = make_uint4(v[0], v[1], v[2], v[3]);
                  *reinterpret_cast<uint4*>(dst + k + i + 8) = make_uint4(v[4], v[5], v[6], v[7]);
                }
              }
            }
          }
        }
        if (row < rows && part >= 0 && !join) *chunk_part_ml(p, part, row) = make_float2(m, l);
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::O_FREE + tile));
      if (part >= 0 && p.counters != nullptr && !join && !idle)
        chunk_join(p, first, last, counter, tile * 128 + q4 * 32, rows,
                   p.out + (size_t)s_seg[slot].r * p.sstride_out + (size_t)(s_seg[slot].q0 + s_seg[slot].tok0) * p.rstride_out +
                       s_seg[slot].g * gq * kHd);
      release_segment(slot);
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

// The parts of a call with few items, which many CTAs share (one request's 4000 keys: 19 CTAs per kv head): a CTA
// per row, each of its warps an eighth of the parts, joined in order. At most one item begins in a CTA and goes
// on in the next ones, as that CTA describes it. blockIdx.x is that CTA (up to eight rows), or counts the CTAs that
// left one: a grid of all of them times 256 rows would be 39 000 CTAs, nearly all without work. Scheduled behind
// the attention grid's last CTAs (programmatic launch); it reads only after that grid has completed. Latency
// bounds it, a chain of three or four loads (four rows per warp, whole items' parts in turn: one request of 64
// tokens over 30 000 keys 65 us, this 47).
constexpr int kMergeWarps = 8;
__global__ void __launch_bounds__(32 * kMergeWarps) chunk_merge_kernel(const ChunkAttnParams p, int ctas) {
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int cta = blockIdx.x;
  if (p.group_rows > 8) {
    __shared__ unsigned s_left[kMergeWarps];         // one bit per CTA: at most 256
    const unsigned left = __ballot_sync(0xffffffffu, (int)threadIdx.x < ctas && p.items[threadIdx.x].rows > 0);
    if (lane == 0) s_left[warp] = left;
    __syncthreads();
    int rank = cta, w = 0;
    for (; w < kMergeWarps && rank >= __popc(s_left[w]); ++w) rank -= __popc(s_left[w]);
    if (w == kMergeWarps) return;
    unsigned bits = s_left[w];
    for (; rank > 0; --rank) bits &= bits - 1u;
    cta = 32 * w + __ffs(bits) - 1;
  }
  const TreeItem it = p.items[cta];
  if (row >= it.rows) return;
  __shared__ float4 s_o[kMergeWarps][32];
  __shared__ float s_l[kMergeWarps];
  auto slot = [&](int c) { return c == cta ? 2 * c + 1 : 2 * c; };
  float m = -INFINITY;
  for (int c = cta + lane; c <= it.last; c += 32) m = fmaxf(m, chunk_part_ml(p, slot(c), row)->x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const int n = it.last - cta + 1, per = (n + kMergeWarps - 1) / kMergeWarps, c1 = min(cta + (warp + 1) * per, it.last + 1);
#pragma unroll 4
  for (int c = cta + warp * per; c < c1; ++c) {
    const float2 x = *chunk_part_ml(p, slot(c), row);
    const float4 v = *reinterpret_cast<const float4*>(chunk_part_o(p, slot(c), row, 4 * lane));
    if (x.y != 0.f) {                                // else the row sees no key of that part
      const float w = exp2f(x.x - m);
      l += exp2f(log2f(x.y) + (x.x - m));            // in the exponent: l is far from 1 where v's scales differ much
      o.x += w * v.x;
      o.y += w * v.y;
      o.z += w * v.z;
      o.w += w * v.w;
    }
  }
  s_o[warp][lane] = o;
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < kMergeWarps; ++w) {
    const float4 v = s_o[w][lane];
    l += s_l[w];
    o.x += v.x;
    o.y += v.y;
    o.z += v.z;
    o.w += v.w;
  }
  const float inv = 1.0f / l;                         // (0: all the row's scores are -inf, and the output is NaN)
  const int gq = p.call.gq, tok = row / gq;
  uint2 out;
  out.x = pack_bf16x2(o.x * inv, o.y * inv);
  out.y = pack_bf16x2(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(p.out + (size_t)it.r * p.sstride_out + (size_t)(it.q0 + tok) * p.rstride_out +
                            (it.g * gq + row - tok * gq) * kHd + 4 * lane) = out;
}

// Up to eight rows go to the warp-level kernel (chunk_decode.cu): one request of 4000 keys 12.4 us, 15.6 by tiles; 32
// requests of 2000 keys in 8 bits 38 us, 57 by tiles. Tiles where they stream faster, in bf16, once the call has
// an item for every SM and contexts are long: 32 requests of 2000 keys 53.9 us by warps, 50.0 by tiles, 48 of 4100 keys
// of a window 73.4 and 71.0, 32 of 1100 keys 35.3 and 34.9; but 32 of 900 keys 31.3 and 32.5, 64 of 300 keys 29.3 and
// 32.7. Up to 128 rows are one tile (every request with as many new tokens, 4 q heads per kv head; bf16, then 8 bits):
//   8 requests of 30 tokens (120 rows) over 4000 keys  50.2 and 53.9 us as one tile, 51.7 and 56.9 as two
//   8 of 16 (64 rows) over 4000                        40.7 and 44.6, 42.2 and 47.5
//   32 of 4 (16 rows) over 2000                        51.8 and 57.5, 55.1 and 69.4
// A call's bounds stand for its requests here: 64 requests of 300 keys in a call of up to 8192 keys take the tiles.
int chunk_group_rows(int max_rows, bool q8, bool many, int max_keys) {
  if (max_rows <= 8 && (q8 || !many || max_keys < 1024)) return 8;
  return max_rows <= 128 ? 128 : 256;
}

template <int MT, bool Q8>
static cudaError_t launch_chunk(const CUtensorMap& map_q, const ChunkAttnParams& p, int grid, cudaStream_t st) {
  using C = ChunkCfg<MT, Q8>;
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(chunk_attn_kernel<MT, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    // the warpgroups' register budgets (setmaxnreg) come out of the registers of the launch
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, chunk_attn_kernel<MT, Q8>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs * C::kThreads < C::kRegsAll) return cudaErrorInvalidConfiguration;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = programmatic(dim3(grid), C::kThreads, C::kSmem, st, attr);
  return cudaLaunchKernelEx(&cfg, chunk_attn_kernel<MT, Q8>, map_q, p);
}

cudaError_t launch_chunk_attention(const CUtensorMap& map_q, const ChunkAttnParams& p, int grid, cudaStream_t st) {
  const int rows = p.group_rows;
  const bool q8 = p.scales_k != nullptr;
  cudaError_t e = rows == 8    ? launch_chunk_decode(p, grid, st)
                  : rows == 128 ? (q8 ? launch_chunk<1, true>(map_q, p, grid, st) : launch_chunk<1, false>(map_q, p, grid, st))
                                : (q8 ? launch_chunk<2, true>(map_q, p, grid, st) : launch_chunk<2, false>(map_q, p, grid, st));
  if (e != cudaSuccess || p.counters != nullptr) return e;
  cudaLaunchAttribute attr[1];
  int items = grid;
  if (rows > 8) items = std::min(items, p.n_reqs * p.t * p.kv_per * ((p.call.max_query_len + p.call.tg - 1) / p.call.tg));   // fewer than SMs
  const int rows_of = std::min(p.call.max_query_len, p.call.tg) * p.call.gq;
  const cudaLaunchConfig_t cfg = programmatic(dim3(items, rows_of), 32 * kMergeWarps, 0, st, attr);
  return cudaLaunchKernelEx(&cfg, chunk_merge_kernel, p, grid);
}

}  // namespace tpl
