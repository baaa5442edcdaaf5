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
#include <atomic>

#include "gemm_tc.cuh"
#include "internal.h"
#include "tree_plan.h"

namespace tpl {

namespace {
constexpr int kHd = 128;
constexpr int kStatusShape = -2;   // TP_ERR_SHAPE
constexpr int kMaxDraft = 256;     // TP_TREE_MAX_DRAFT
}  // namespace

// One CTA per request, a thread per drafted token. By pointer jumping: a token's row starts
// as its own bit and its parent's index; each round adds the row of the token it points to
// and points to where that one points, so a chain of d ancestors takes log2(d) + 1 rounds
// (a chain of 64: 7; walking up it took 64 dependent reads). Latency bounds it: a few KB.
__global__ void __launch_bounds__(kMaxDraft)
    tree_mask_kernel(int T, int max_query_len, int words, const int* parents, const int* qsl, const int* seq_lens,
                     int* mask, int* positions, int* status) {
  constexpr int kWords = kMaxDraft / 32;
  __shared__ unsigned rows[2][kWords][kMaxDraft];
  __shared__ int up[2][kMaxDraft];                   // >= 0: the next ancestor; -1: none left; -2: a bad parent above
  const int b = blockIdx.x, i = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const int q0 = qsl[b], q1 = qsl[b + 1], len = seq_lens[b];
  if (q0 < 0 || q1 < q0 || q1 > T || q1 - q0 > max_query_len || len < q1 - q0) {   // no difference that wraps
    if (i == 0) atomicExch(status, kStatusShape);
    return;
  }
  const int n = q1 - q0, ctx = len - n;
  const int used = (n + 31) / 32;
  int to = -1;
  unsigned bits[kWords];
#pragma unroll
  for (int w = 0; w < kWords; ++w) bits[w] = 0u;
  if (i < n) {
    to = parents[q0 + i];
    if (to < -1 || to >= i) {
      to = -2;
      atomicExch(status, kStatusShape);
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w)
      if (w == i >> 5) bits[w] = 1u << (i & 31);
  }
  int buf = 0;
  for (int round = 0; round < 10; ++round) {         // 256 tokens: at most 9
    up[buf][i] = to;
#pragma unroll
    for (int w = 0; w < kWords; ++w)
      if (w < used) rows[buf][w][i] = bits[w];
    if (!__syncthreads_or(to >= 0)) break;
    if (to >= 0) {
#pragma unroll
      for (int w = 0; w < kWords; ++w)
        if (w < used) bits[w] |= rows[buf][w][to];
      to = up[buf][to];
    }
    buf ^= 1;
  }
  if (i >= n) return;
  const bool ok = to == -1;
  int depth = -1;
#pragma unroll
  for (int w = 0; w < kWords; ++w) depth += __popc(bits[w]);
#pragma unroll
  for (int w = 0; w < kWords; ++w)
    if (w < words) mask[(size_t)(q0 + i) * words + w] = ok ? (int)bits[w] : 0;
  for (int w = kWords; w < words; ++w) mask[(size_t)(q0 + i) * words + w] = 0;
  if (positions != nullptr) positions[q0 + i] = ok ? ctx + depth : -1;
}

// ---------------------------------------------------------------- attention kernel
// The queries that read one kv head of a request (its drafted tokens x the q heads of the
// group) are the rows of 128-row tensor-core tiles; its keys go by in chunks of 128, read
// once from the cache for all of them:
//   S = Q K^T  (tcgen05, 128 x 128 x 128, fp32 in tensor memory)
//   P = 2^(s c - m) as bf16, written over S (tensor memory, the A operand of P V)
//   O += P V   (tcgen05, O in tensor memory)
// with the running max m and sum l of every row in its thread's registers. Persistent, one
// CTA per SM; the chunks of all items are one line cut into equal ranges (tree_plan.h), so
// the CTAs stream the same number of keys whatever the requests' lengths.
//
// MT = 1: up to 128 rows per item; S of a chunk in one of three buffers of 128 columns; two Q
// buffers, so that the next segment's queries load while this one's are read. MT = 2: up to
// 256 rows as two tiles on the same K and V. Tensor memory holds 512 columns, 2 x 128 of them
// O: S goes by halves of a chunk (64 keys), two buffers of 64 columns per tile, so that a
// tile's next S is ready when its softmax is done with the last.
//
//   warp 0      issues S;  warp 1 issues P V (an elected lane of a converged warp);
//   warp 2      walks the CTA's range and publishes segments
//   warp 3      looks over the V rows of drafted tokens (below)
//   warps 4-7   copies: K and V rows through the block table with 16-byte cp.async into
//               128-byte-swizzled tiles (any block size: a key's row is found on its own),
//               a ring of tiles K0 V0 K1 V1 ...; Q rows of a segment
//   warps 8-    softmax, a row per thread, four warps per tile; at a segment's end O / l to
//               global memory, or the unnormalised O with (m, l) to a partial slot
//
// A row's mask applies to the chunks that hold drafted tokens alone. There, values of a drafted
// token's V that are not finite are set to zero in shared memory, so that 0 * v of a token that
// does not see the key stays 0, and the rows that do see it get the value added at the end.
// Warp 3 does that between the copy and the product (the copying threads themselves would have
// to wait for their copies, which left the ring empty at every item's end: up to 5 us of 35).
//
// Up to 128 rows HBM bounds it: a chunk is 64 KB, 1.47 us of one SM's share of the measured copy
// bandwidth, and takes 1.52 us (2 x 131072 keys, 8 drafts of 64 q heads: 167 us, 0.94). With two
// tiles shared memory does, 256 KB read by the products (Q again for each half of S) and 64 KB
// written per chunk, 1.3 us, with the chain S, softmax, P V of a tile through its two buffers:
// 1.85 us per chunk (26 drafts: 211 us, 0.75); without the exponentials or the row maximum it
// takes as long.
namespace {
constexpr int kTileBytes = 128 * 128 * 2;      // 128 rows x 128 bf16: two 64-column boxes
constexpr int kUnitSlots = 4;
constexpr float kRescaleLog2 = 8.0f;           // rescale O when the row max grows by more than this
constexpr uint32_t kIdescO = idesc_bf16_f32(128, 128) | kIdescBMnMajor;
constexpr int kTmemCols = 512;

template <int MT>
struct TreeCfg {
  static constexpr int kThreads = 256 + 128 * MT;
  static constexpr int kTiles = 5;                         // K/V ring
  static constexpr int kQBufs = MT == 1 ? 2 : 1;
  static constexpr int kSub = MT == 1 ? 128 : 64;          // keys of one S, softmax and P V
  static constexpr int kSubs = kTreeChunk / kSub;
  static constexpr int kSBufs = MT == 1 ? 3 : 2;           // S/P buffers of a tile
  static constexpr uint32_t kIdescS = idesc_bf16_f32(128, kSub);
  static constexpr int kRingOff = MT * kQBufs * kTileBytes;   // after Q
  static constexpr int kBarOff = kRingOff + kTiles * kTileBytes;
  // registers: issuers, copies, softmax
  static constexpr int kRegs0 = 80, kRegs1 = MT == 1 ? 152 : 96, kRegsS = MT == 1 ? 232 : 168;
  static constexpr int kLaunchRegs = MT == 1 ? 168 : 128;
  static_assert(128 * (kRegs0 + kRegs1 + MT * kRegsS) <= kThreads * kLaunchRegs, "register split within the launch's");
  // tensor memory: MT = 1: S/P at 0, 128, 256, O at 384; MT = 2: tile m S/P at 256 m and 256 m + 64, O at 256 m + 128
  static __device__ __forceinline__ uint32_t s_col(int tile, int buf) { return tile * 256 + (buf - tile * kSBufs) * kSub; }
  static __device__ __forceinline__ uint32_t o_col(int tile) { return MT == 1 ? 384 : tile * 256 + 128; }
  enum {
    Q_FULL = 0, Q_EMPTY = Q_FULL + kQBufs, FULL = Q_EMPTY + kQBufs, EMPTY = FULL + kTiles,
    S_FULL = EMPTY + kTiles,          // per S/P buffer of every tile
    P_READY = S_FULL + MT * kSBufs,
    S_FREE = P_READY + MT * kSBufs,   // its P V has completed
    O_FREE = S_FREE + MT * kSBufs,    // per tile
    LANDED = O_FREE + MT,             // a V tile with drafted tokens, per ring tile: to be looked over
    U_FULL = LANDED + kTiles, U_EMPTY = U_FULL + kUnitSlots,
    DONE_S = U_EMPTY + kUnitSlots, DONE_PV, NBARS
  };
  static constexpr int kMiscOff = kBarOff + 8 * NBARS;     // tensor memory address, abort flag
  static constexpr int kUnitOff = (kMiscOff + 8 + 15) / 16 * 16;
  static constexpr int kSmem = 1024 + kUnitOff + kUnitSlots * 64;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

// A segment: chunks [c0, c1) of one item. b < 0: no more.
struct __align__(16) Segment {
  int b, r, g, row0;                 // request, shard, kv head of the shard, first query row of the item
  int c0, c1, q0, n;                 // chunks; first drafted token and their number
  int len, part, rows, bad;          // tokens of the request; partial slot or -1; query rows of the item; V not finite
  int pad[4];
};
static_assert(sizeof(Segment) == 64, "unit slots");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int src_bytes, uint64_t pol) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(src_bytes),
               "l"(pol)
               : "memory");
}
// One arrival on bar once all cp.async of this thread so far have landed (counted in the barrier's own count).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Shared memory written by ordinary copies and stores, seen by this thread through a barrier,
// is ordered before the tensor core's reads that it issues next.
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// bf16 pairs of a 32-bit word whose exponent is all ones become zero; true if one was
__device__ __forceinline__ bool drop_nonfinite(uint32_t& w) {
  bool any = false;
  if ((w & 0x7f80u) == 0x7f80u) {
    w &= 0xffff0000u;
    any = true;
  }
  if ((w & 0x7f800000u) == 0x7f800000u) {
    w &= 0x0000ffffu;
    any = true;
  }
  return any;
}
}  // namespace

// Partial results of a slot: O as [16][rows][8] fp32 (pieces of eight dimensions, so that the
// 32 rows of a warp write 1 KB on end; rows written whole, 512 bytes apart, took 2.5 us for 256
// of them and held up the copies behind them), then [rows][2] (max in the exp2 domain, sum).
// part_rows is a multiple of 8 and the first slot 32-byte aligned: every piece starts on 32 bytes.
__device__ __forceinline__ float* part_o(const TreeAttnParams& p, int slot, int row, int d) {
  return p.partials + (size_t)slot * p.part_rows * (kHd + 2) + ((size_t)(d >> 3) * p.part_rows + row) * 8 + (d & 7);
}
__device__ __forceinline__ float2* part_ml(const TreeAttnParams& p, int slot, int row) {
  return reinterpret_cast<float2*>(p.partials + (size_t)slot * p.part_rows * (kHd + 2) + (size_t)p.part_rows * kHd) + row;
}

template <int MT>
__global__ void __launch_bounds__(TreeCfg<MT>::kThreads, 1) tree_attn_kernel(const TreeAttnParams p) {
  using C = TreeCfg<MT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw_addr);
  auto bar = [&](int b) { return base + C::kBarOff + 8u * b; };
  volatile uint32_t* s_tmem = reinterpret_cast<volatile uint32_t*>(base_ptr + C::kMiscOff);
  volatile int* s_abort = reinterpret_cast<volatile int*>(base_ptr + C::kMiscOff + 4);
  Segment* s_seg = reinterpret_cast<Segment*>(base_ptr + C::kUnitOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_launch_dependents();   // the merge grid may be scheduled; it waits for this one to complete
  if (warp == 0) {
    for (int b = lane; b < C::NBARS; b += 32) {
      int count = 1;
      if (b < C::Q_EMPTY || (b >= C::FULL && b < C::EMPTY)) count = 128;        // every copying thread
      if (b >= C::P_READY && b < C::S_FREE) count = 4;                          // the tile's softmax warps
      if (b >= C::S_FREE && b < C::O_FREE) count = 2;                           // the MMAs, and their issuer
      if (b >= C::O_FREE && b < C::LANDED) count = 4;
      if (b >= C::LANDED && b < C::U_FULL) count = 128;
      if (b >= C::U_EMPTY && b < C::DONE_S) count = 3 + 4 + 4 * MT;             // issuers, warp 3, copy and softmax warps
      mbar_init(bar(b), count);
    }
    if (lane == 0) *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(s_tmem)), kTmemCols);
    tmem_relinquish();
  }
  // the set-up above may overlap the grid before (programmatic launch); nothing that grid
  // wrote is read before this
  griddep_wait();
  const int gq = p.q_per / p.kv_per;                // q heads of a kv head
  constexpr int kGroupRows = 128 * MT;
  auto request = [&](int b) {
    return tree_request(p.qsl[b], p.qsl[b + 1], p.seq_lens[b], p.T, p.max_query_len, p.max_seq_len, gq, kGroupRows);
  };
  // warp 2: requests `lane`, `lane` + 32, .. of a batch of 128 (first row, drafted tokens, tokens; -1: bad
  // counts), loaded together; the first batch here, beside the set-up
  constexpr int kStrips = 4;
  int3 mine[kStrips];
  auto load_batch = [&](int b0) {
#pragma unroll
    for (int i = 0; i < kStrips; ++i) {
      mine[i] = make_int3(0, 0, 0);
      const int b = b0 + 32 * i + lane;
      if (b < p.n_reqs) {
        const TreeReq r = request(b);
        mine[i] = make_int3(r.q0, r.ok ? r.n : -1, r.len);
      }
    }
  };
  if (warp == 2) load_batch(0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
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
    return s_seg[slot].b < 0 ? -1 : slot;
  };
  auto release_segment = [&](int slot) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::U_EMPTY + slot));
  };

  if (warp < 4) {
    regs_dec<C::kRegs0>();
    if (warp == 0) {
      // ------------------------------------------------------------ S = Q K^T
      const uint64_t q_desc = smem_desc_k128(base);
      const uint64_t k_desc = smem_desc_k128(base + C::kRingOff);
      constexpr uint64_t kTileDesc = kTileBytes >> 4;
      int ring = 0;                                   // tile of the next K
      uint32_t ring_ph = 0;
      int cnt[MT] = {};                               // chunks of each tile so far
      for (int seg_no = 0;; ++seg_no) {
        const int slot = next_segment();
        if (slot < 0) break;
        const int n = s_seg[slot].c1 - s_seg[slot].c0, rows = s_seg[slot].rows;
        release_segment(slot);
        const int qb = seg_no % C::kQBufs;
        if (!wait(C::Q_FULL + qb, (seg_no / C::kQBufs) & 1)) break;
        for (int j = 0; j < n && ok; ++j) {
          if (!wait(C::FULL + ring, ring_ph)) break;
          fence_async_proxy();
#pragma unroll
          for (int h = 0; h < C::kSubs; ++h) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              if (m * 128 >= rows) break;
              const int buf = m * C::kSBufs + cnt[m] % C::kSBufs;
              if (!wait(C::S_FREE + buf, ((cnt[m] / C::kSBufs) & 1) ^ 1)) break;
              ++cnt[m];
              tc_fence_after();
              if (elect_one()) {
                const uint32_t d = tmem_base + C::s_col(m, buf);
                // half h of the chunk: 64 K rows of 128 bytes further
                const uint64_t qd = q_desc + (qb * MT + m) * kTileDesc, kd = k_desc + ring * kTileDesc + h * ((64 * 128) >> 4);
                tc_mma_bf16_c<false>(d, qd, kd, C::kIdescS);
#pragma unroll
                for (int k = 1; k < 8; ++k) {
                  const uint64_t o = (uint64_t)(((k >> 2) * (kTileBytes / 2) + (k & 3) * 32) >> 4);
                  tc_mma_bf16_c<true>(d, qd + o, kd + o, C::kIdescS);
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
        const int n = s_seg[slot].c1 - s_seg[slot].c0, rows = s_seg[slot].rows;
        release_segment(slot);
        for (int j = 0; j < n && ok; ++j) {
          if (!wait(C::FULL + ring, ring_ph)) break;
          fence_async_proxy();
#pragma unroll
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
                mbar_arrive(bar(C::S_FREE + buf));    // carries the copies' `bad` mark to the softmax
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
      const int heads = p.t * p.kv_per;
      int cost = 0;
      auto work = [&](const TreeReq& r) { return heads * tree_head(r, cost); };
      auto counted = [&](int3 m) {                    // the request of its counts (none where they are bad)
        return tree_request(m.x, m.x + max(m.y, 0), m.z, p.T, p.max_query_len, p.max_seq_len, gq, kGroupRows);
      };
      auto broadcast = [&](int3 m, int from) {
        return counted(make_int3(__shfl_sync(0xffffffffu, m.x, from), __shfl_sync(0xffffffffu, m.y, from),
                                 __shfl_sync(0xffffffffu, m.z, from)));
      };
      auto sum = [&](long long v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
      };
      // all requests' chunks and heads' places with an item cost of 0 and of 1 apart; CTA 0 reports bad counts
      long long chunks = 0, places = 0, items = 0;
      int widest = 1;
      for (int b0 = 0; b0 < p.n_reqs; b0 += 32 * kStrips) {
        if (b0 > 0) load_batch(b0);
#pragma unroll
        for (int i = 0; i < kStrips; ++i) {
          if (mine[i].y < 0 && blockIdx.x == 0) atomicExch(p.status, kStatusShape);
          const TreeReq q = counted(mine[i]);
          chunks += (long long)q.groups * q.chunks;
          places += tree_head(q, 0);
          items += q.groups;
          widest = max(widest, tree_widest(q));
        }
      }
      cost = tree_cost(heads * sum(chunks), gridDim.x);
      const long long total = heads * sum(places + cost * items);
      const long long per = tree_per(total, gridDim.x, __reduce_max_sync(0xffffffffu, widest));
      long long pos = per * blockIdx.x;
      const long long end = min(total, pos + per);
      // the request that holds the first place, and the places before it
      TreeReq r{};
      int b = 0;
      long long before = 0;
      if (pos < end) {
        bool found = false;
        for (int b0 = 0; b0 < p.n_reqs && !found; b0 += 32 * kStrips) {
          if (p.n_reqs > 32 * kStrips) load_batch(b0);
#pragma unroll
          for (int i = 0; i < kStrips; ++i) {
            if (found) break;
            const TreeReq q = counted(mine[i]);
            const long long w = work(q);
            long long pre = w;                        // the strip's places up to and with this lane's
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const long long up = __shfl_up_sync(0xffffffffu, pre, o);
              if (lane >= o) pre += up;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, before + pre > pos);
            if (hit != 0u) {
              const int f = __ffs(hit) - 1;
              b = b0 + 32 * i + f;
              before += __shfl_sync(0xffffffffu, pre - w, f);
              r = broadcast(mine[i], f);
              found = true;
            } else {
              before += __shfl_sync(0xffffffffu, pre, 31);
            }
          }
        }
      }
      // no item of this CTA is continued by others, unless a segment says so below
      if (lane == 0) p.items[blockIdx.x].rows = 0;
      __syncwarp();
      for (int u = 0;; ++u) {
        const int slot = u % kUnitSlots;
        if (!wait(C::U_EMPTY + slot, ((u / kUnitSlots) & 1) ^ 1)) break;
        Segment s;
        s.b = -1;
        while (pos < end) {
          while (pos - before >= work(r)) {            // this request is done: on to the next one with work
            before += work(r);
            for (;; b += 32) {
              const int next = b + 1 + lane;
              int3 m = make_int3(0, 0, 0);
              if (next < p.n_reqs) {
                const TreeReq q = request(next);
                m = make_int3(q.q0, q.n, q.len);
              }
              const unsigned hit = __ballot_sync(0xffffffffu, m.y > 0);
              if (hit != 0u) {
                const int f = __ffs(hit) - 1;
                b += 1 + f;
                r = broadcast(m, f);
                break;
              }
              if (b + 32 >= p.n_reqs) {                // cannot be: a place before `end` belongs to a request
                pos = end;
                r = TreeReq{};
                break;
              }
            }
            if (pos >= end) break;
          }
          if (pos >= end) break;
          const TreeSeg q = tree_segment(r, cost, pos - before, end - pos, blockIdx.x);
          pos += q.places;
          if (q.c0 == q.c1) continue;                  // no chunk begins in these places
          s.b = b;
          s.r = q.head / p.kv_per;
          s.g = q.head - s.r * p.kv_per;
          s.row0 = q.group * kGroupRows;
          s.c0 = q.c0;
          s.c1 = q.c1;
          s.q0 = r.q0;
          s.n = r.n;
          s.len = r.len;
          s.part = q.part;
          s.rows = min(kGroupRows, r.n * gq - s.row0);
          s.bad = 0;
          if (q.c0 == 0 && q.part >= 0 && lane == 0) {
            const int last = tree_last(r, q.group, before + q.begin, cost, per);
            p.items[blockIdx.x] = TreeItem{s.r, s.g, s.row0, s.rows, s.q0, last, 0, 0};
          }
          break;
        }
        if (lane == 0) {
          s_seg[slot] = s;
          mbar_arrive(bar(C::U_FULL + slot));
        }
        __syncwarp();
        if (s.b < 0) break;
      }
    } else {
      // ------------------------------------------------------------ V of drafted tokens
      int ring = 1;                                   // tile of the next V
      uint32_t phases = 0;                            // bit i: phase of LANDED + i
      for (;;) {
        const int slot = next_segment();
        if (slot < 0) break;
        const int c0 = s_seg[slot].c0, c1 = s_seg[slot].c1, len = s_seg[slot].len, ctx = len - s_seg[slot].n;
        bool bad = false;
        for (int c = c0; c < c1; ++c) {
          if ((c + 1) * kTreeChunk > ctx) {
            if (!wait(C::LANDED + ring, phases >> ring & 1u)) break;
            phases ^= 1u << ring;
            // rows of drafted tokens; a row is 8 pieces of 16 bytes in each of two boxes, in any order
            const int r1 = min(len - c * kTreeChunk, kTreeChunk), box = (lane >> 3) & 1, piece = lane & 7;
            uint8_t* v = base_ptr + C::kRingOff + ring * kTileBytes + box * (kTileBytes / 2) + piece * 16;
#pragma unroll 4
            for (int row = max(ctx - c * kTreeChunk, 0) + (lane >> 4); row < r1; row += 2) {
              uint4* q = reinterpret_cast<uint4*>(v + row * 128);
              uint4 d = *q;
              const bool x = drop_nonfinite(d.x), y = drop_nonfinite(d.y), z = drop_nonfinite(d.z), w = drop_nonfinite(d.w);
              if (x || y || z || w) {
                *q = d;
                bad = true;
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
  } else if (warp < 8) {
    // ------------------------------------------------------------ copies
    regs_dec<C::kRegs1>();
    const int w4 = warp - 4, c16 = lane & 15, half = lane >> 4;
    // this thread copies 16-byte piece c16 of rows 2 w4 + half + 8 k; lane i of the warp finds the
    // cache row of row 8 (i / 2) + 2 w4 + i % 2
    const int row_of = 2 * w4 + half, my_row = 8 * (lane >> 1) + 2 * w4 + (lane & 1);
    const uint32_t dst0 = (c16 >> 3) * (kTileBytes / 2) + row_of * 128 + (((c16 & 7) ^ (row_of & 7)) << 4);
    // the cache is read once a call by one item (evicted first) or by its groups of rows
    const uint64_t pol = p.max_query_len * gq > kGroupRows ? policy_evict_normal() : policy_evict_first();
    int ring = 0;
    uint32_t ring_ph = 0;
    auto advance = [&]() {
      if (++ring == C::kTiles) {
        ring = 0;
        ring_ph ^= 1u;
      }
    };
    // a segment's queries, once those that the buffer held are no longer read
    auto load_q = [&](const Segment& s, int seg_no) {
      const int qb = seg_no % C::kQBufs;
      if (!wait(C::Q_EMPTY + qb, ((seg_no / C::kQBufs) & 1) ^ 1)) return;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m * 128 >= s.rows) break;
        // rows past the item's keep what the buffer held: they only reach their own rows of S and O
        const __nv_bfloat16* q = p.qkv + (size_t)s.r * p.sstride_in + s.g * gq * kHd + c16 * 8;
#pragma unroll 4
        for (int k = 0; k < 16; ++k) {
          const int j = m * 128 + row_of + 8 * k;
          const int jr = s.row0 + j, tok = token_of(jr);
          if (j < s.rows)
            cp_async16(base + (qb * MT + m) * kTileBytes + dst0 + k * 1024,
                       q + (size_t)(s.q0 + tok) * p.rstride_in + (jr - tok * gq) * kHd, 16, pol);
        }
      }
      cp_async_arrive(bar(C::Q_FULL + qb));
    };
    for (int seg_no = 0;; ++seg_no) {
      const int slot = next_segment();
      if (slot < 0) break;
      const Segment s = s_seg[slot];
      const int ctx = s.len - s.n;
      const int* bt = p.block_tables + (size_t)s.b * p.max_blocks;
      auto block_of = [&](int c) -> int {            // block id of this lane's key of chunk c
        const int key = c * kTreeChunk + my_row;
        return key < s.len ? bt[key / p.block_size] : -1;
      };
      int blk = block_of(s.c0);
      // with one Q buffer the last segment's queries may still be read: the first K tile goes before
      // (and the queries' rows, 256 bytes each, start for L2: their copy is what S waits for)
      const bool q_first = C::kQBufs > 1 || seg_no == 0;
      if (q_first) {
        load_q(s, seg_no);
      } else {
        for (int j = threadIdx.x - 128; j < 2 * s.rows; j += 128) {
          const int jr = s.row0 + (j >> 1), tok = token_of(jr);
          prefetch_l2(p.qkv + (size_t)s.r * p.sstride_in + (size_t)(s.q0 + tok) * p.rstride_in +
                      (s.g * gq + jr - tok * gq) * kHd + (j & 1) * 64);
        }
      }
      for (int c = s.c0; c < s.c1 && ok; ++c) {
        const int key = c * kTreeChunk + my_row;
        int row = -1;                                // cache row of this lane's key (-1: zeros)
        if (key < s.len) {
          if (blk >= 0 && blk < p.num_blocks)
            row = (s.r * p.num_blocks + blk) * p.block_size + key % p.block_size;
          else
            atomicExch(p.status, kStatusShape);
        }
        if (c + 1 < s.c1) blk = block_of(c + 1);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          if (!wait(C::EMPTY + ring, ring_ph ^ 1)) break;
          const __nv_bfloat16* src = (kv ? p.cache_v : p.cache_k) + s.g * kHd + c16 * 8;
          const uint32_t dst = base + C::kRingOff + ring * kTileBytes + dst0;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int rw = __shfl_sync(0xffffffffu, row, 2 * k + half);
            cp_async16(dst + k * 1024, src + (size_t)max(rw, 0) * p.kv_per * kHd, rw >= 0 ? 16 : 0, pol);
          }
          cp_async_arrive(bar((kv == 1 && (c + 1) * kTreeChunk > ctx ? C::LANDED : C::FULL) + ring));
          advance();
          if (kv == 0 && c == s.c0 && !q_first) load_q(s, seg_no);
          if (!ok) break;
        }
      }
      if (!ok) break;
      release_segment(slot);
    }
    cp_async_wait_all();       // no copy into this CTA's shared memory may outlive it
  } else {
    // ------------------------------------------------------------ softmax
    regs_inc<C::kRegsS>();
    const int tile = (warp - 8) >> 2, q4 = warp & 3;
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
      const int n = s_seg[slot].n, len = s_seg[slot].len, ctx = len - n, q0 = s_seg[slot].q0;
      const bool idle = tile * 128 + q4 * 32 >= rows;  // no row of this warp
      const int jr = s_seg[slot].row0 + row, tok = row < rows ? token_of(jr) : 0;
      const int* words = p.mask + (size_t)(q0 + tok) * p.mask_words;
      float m = -INFINITY, l = 0.f;
      for (int sc = c0 * C::kSubs; sc < c1 * C::kSubs; ++sc) {
        const int buf = tile * C::kSBufs + cnt % C::kSBufs;
        if (!wait(C::S_FULL + buf, (cnt / C::kSBufs) & 1)) break;
        if (!idle) {
          tc_fence_after();
          const uint32_t sa = lane_addr + C::s_col(tile, buf);
#pragma unroll
          for (int k = 0; k < C::kSub; k += 32) tmem_ld32(sa + k, s + k);
          tc_wait_ld();
          if ((sc + 1) * C::kSub > ctx) {
            // drafted tokens (or the end) among these keys: the row's mask
#pragma unroll
            for (int w = 0; w < C::kSub / 32; ++w) {
              const unsigned bits = tree_window(words, sc * C::kSub + 32 * w, ctx, n);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(bits >> i & 1u)) s[32 * w + i] = -INFINITY;
            }
          }
          float mk[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) mk[j] = fmaxf(s[j], s[8 + j]);
#pragma unroll
          for (int k = 16; k < C::kSub; k += 16)
#pragma unroll
            for (int j = 0; j < 8; ++j) mk[j] = fmax3(mk[j], s[k + j], s[k + 8 + j]);
          const float mx = c * fmax3(fmax3(mk[0], mk[1], mk[2]), fmax3(mk[3], mk[4], mk[5]), fmaxf(mk[6], mk[7]));
          if (sc == c0 * C::kSubs) {
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
#pragma unroll
            for (int k = 0; k < 128; k += 32) {
              tmem_ld32(lane_addr + C::o_col(tile) + k, o);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] *= f;
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
            for (int j = 0; j < 32; ++j) {
              float x0, x1;
              f32x2_unpack(f32x2_fma(f32x2_pack(s[h * 64 + 2 * j], s[h * 64 + 2 * j + 1]), c2, nm2), x0, x1);
              const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
              lk[j & 3] = f32x2_add(lk[j & 3], f32x2_pack(e0, e1));
              pk[j] = pack_bf16x2(e0, e1);
            }
            tmem_st32(sa + h * 32, reinterpret_cast<const float*>(pk));
          }
          float la[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) f32x2_unpack(lk[j], la[2 * j], la[2 * j + 1]);
          l += ((la[0] + la[1]) + (la[2] + la[3])) + ((la[4] + la[5]) + (la[6] + la[7]));
          tc_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::P_READY + buf));
        ++cnt;
      }
      if (!ok) break;
      if (!wait_last_pv()) break;
      if (!idle) {
        tc_fence_after();
        const int bad = *reinterpret_cast<volatile int*>(&s_seg[slot].bad);
        const int r = s_seg[slot].r, g = s_seg[slot].g, b = s_seg[slot].b, part = s_seg[slot].part;
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        __nv_bfloat16* dst = p.out + (size_t)r * p.sstride_out + (size_t)(q0 + tok) * p.rstride_out + (g * gq + jr - tok * gq) * kHd;
#pragma unroll 1
        for (int k = 0; k < 128; k += C::kSub) {
          __syncwarp();
#pragma unroll
          for (int j = 0; j < C::kSub; j += 32) tmem_ld32(lane_addr + C::o_col(tile) + k + j, s + j);
          tc_wait_ld();
          if (bad) {
            // V values that were dropped, added to the rows that see their keys
            const int* bt = p.block_tables + (size_t)b * p.max_blocks;
            const int k0 = max(c0 * kTreeChunk, ctx), k1 = min(c1 * kTreeChunk, len);
            for (int key = k0; row < rows && key < k1; ++key) {
              if (!(tree_window(words, key & ~31, ctx, n) >> (key & 31) & 1u)) continue;
              const int blk = bt[key / p.block_size];
              if (blk < 0 || blk >= p.num_blocks) continue;
              const __nv_bfloat16* v = p.cache_v + ((size_t)(r * p.num_blocks + blk) * p.block_size + key % p.block_size) * p.kv_per * kHd + g * kHd + k;
#pragma unroll
              for (int j = 0; j < C::kSub; ++j) {
                const float x = __bfloat162float(v[j]);
                if (!(fabsf(x) < INFINITY)) s[j] += x;
              }
            }
          }
          if (row < rows) {
            if (part >= 0) {
#pragma unroll
              for (int j = 0; j < C::kSub; j += 8)
                st_global_v8(part_o(p, part, row, k + j), *reinterpret_cast<const uint32_t(*)[8]>(s + j));
            } else {
#pragma unroll
              for (int j = 0; j < C::kSub; j += 16) {
                uint32_t v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = pack_bf16x2(s[j + 2 * i] * inv, s[j + 2 * i + 1] * inv);
                if (p.out_align32) {
                  st_global_v8(dst + k + j, v);
                } else {
                  *reinterpret_cast<uint4*>(dst + k + j) = make_uint4(v[0], v[1], v[2], v[3]);
                  *reinterpret_cast<uint4*>(dst + k + j + 8) = make_uint4(v[4], v[5], v[6], v[7]);
                }
              }
            }
          }
        }
        if (row < rows && part >= 0) *part_ml(p, part, row) = make_float2(m, l);
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::O_FREE + tile));
      release_segment(slot);
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

// Joins the parts of the items that more than one CTA computed. At most one item begins in a
// CTA and goes on in the next ones: item blockIdx.x (described by that CTA), a warp per query
// row, four head dimensions per lane, the parts in the order of their keys (the same bits
// every time).
//   o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,  m = max_i m_i
// Scheduled behind the attention grid's last CTAs (programmatic launch); it reads only after
// that grid has completed.
constexpr int kMergeRows = 8;    // rows, and warps, of a CTA
__global__ void __launch_bounds__(32 * kMergeRows) tree_merge_kernel(const TreeAttnParams p) {
  griddep_wait();
  const int cta = blockIdx.x, row = blockIdx.y * kMergeRows + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const TreeItem it = p.items[cta];
  if (row >= it.rows) return;
  auto slot = [&](int c) { return c == cta ? 2 * c + 1 : 2 * c; };
  auto ml = [&](int c) { return *part_ml(p, slot(c), row); };
  float m = -INFINITY;
  for (int c = cta + lane; c <= it.last; c += 32) m = fmaxf(m, ml(c).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = cta; c <= it.last; ++c) {
    const float2 x = ml(c);
    const float4 v = *reinterpret_cast<const float4*>(part_o(p, slot(c), row, 4 * lane));
    if (x.x != -INFINITY) {                          // else the row sees no key of that part
      const float w = exp2f(x.x - m);
      l += w * x.y;
      o.x += w * v.x;
      o.y += w * v.y;
      o.z += w * v.z;
      o.w += w * v.w;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  const int gq = p.q_per / p.kv_per, jr = it.row0 + row, tok = jr / gq;
  uint2 out;
  out.x = pack_bf16x2(o.x * inv, o.y * inv);
  out.y = pack_bf16x2(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(p.out + (size_t)it.r * p.sstride_out + (size_t)(it.q0 + tok) * p.rstride_out +
                            (it.g * gq + jr - tok * gq) * kHd + 4 * lane) = out;
}

cudaError_t launch_tree_mask(int T, int n_reqs, int max_query_len, int words, const int* parents, const int* qsl,
                             const int* seq_lens, int* mask, int* positions, int* status, cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = programmatic(dim3(n_reqs), (max_query_len + 31) / 32 * 32, 0, st, attr);
  return cudaLaunchKernelEx(&cfg, tree_mask_kernel, T, max_query_len, words, parents, qsl, seq_lens, mask, positions, status);
}

// Up to 128 rows the kernel of one tile: with whole chunks per softmax and two Q buffers it is
// ahead where the cache does not bound it (48 requests on the same 4096 tokens' pages, which L2
// holds: 101 us, the kernel of two tiles 116), and little where it does (2 x 131072 keys: 167.1
// against 168.0 us; 32 requests of 256 to 4096 keys: 56.1 against 56.6).
int tree_group_rows(int max_rows) { return max_rows <= 128 ? 128 : 256; }

template <int MT>
static cudaError_t launch_tree_mt(const TreeAttnParams& p, int grid, cudaStream_t st) {
  using C = TreeCfg<MT>;
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(tree_attn_kernel<MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    // the warpgroups' register budgets (setmaxnreg) come out of the registers of the launch
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, tree_attn_kernel<MT>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs * C::kThreads < 128 * (C::kRegs0 + C::kRegs1 + MT * C::kRegsS)) return cudaErrorInvalidConfiguration;
    attr_done.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = programmatic(dim3(grid), C::kThreads, C::kSmem, st, attr);
  return cudaLaunchKernelEx(&cfg, tree_attn_kernel<MT>, p);
}

cudaError_t launch_tree_attention(const TreeAttnParams& p, int grid, cudaStream_t st) {
  const int max_rows = p.max_query_len * (p.q_per / p.kv_per);
  cudaError_t e = tree_group_rows(max_rows) == 128 ? launch_tree_mt<1>(p, grid, st) : launch_tree_mt<2>(p, grid, st);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = programmatic(dim3(grid, (p.part_rows + kMergeRows - 1) / kMergeRows), 32 * kMergeRows, 0, st, attr);
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel, p);
}

}  // namespace tpl
