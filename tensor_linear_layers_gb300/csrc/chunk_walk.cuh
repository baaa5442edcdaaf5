// A CTA's walk over its range of a call's key chunks (chunk_plan.h), and what the kernels of the
// attention of chunks share: which keys an item's tokens see, and the layout of partial results.
#pragma once
#include <cuda_runtime.h>

#include "chunk_plan.h"
#include "internal.h"

namespace tpl {

// A segment: chunks [c0, c1) of one item. b < 0: no more.
struct __align__(16) ChunkSegment {
  int b, r, g, tok0;                 // request, shard, kv head of the shard, first new token of the group
  int c0, c1, q0, ctx;               // chunks; row of the request's first new token; cached tokens
  int part, rows, bad, skip;         // partial slot or -1; query rows; V not finite; key chunks left out from sc on
  int p0, p1, pad0, pad1;            // positions of the group's first and last token
};
static_assert(sizeof(ChunkSegment) == 64, "unit slots");


constexpr int kChunkStatusShape = -2;   // TP_ERR_SHAPE

// Key chunk of chunk j of an item.
__device__ __forceinline__ int key_chunk(int j, int sc, int skip) { return j + (j >= sc ? skip : 0); }
// A key that some tokens (at positions p0 to p1) see and others do not, of those that any sees.
__device__ __forceinline__ bool chunk_partly(const ChunkCall& c, int key, int p0, int p1) {
  return key > p0 || (c.window > 0 && key <= p1 - c.window && key >= c.sinks);
}
// Whether key chunk kc has such keys.
__device__ __forceinline__ bool chunk_mixed(const ChunkCall& c, int kc, int p0, int p1) {
  const int k0 = kc * kChunkKeys, k1 = k0 + kChunkKeys - 1;
  return p1 > p0 && (k1 > p0 || (c.window > 0 && k0 <= p1 - c.window && k1 > p0 - c.window && k1 >= c.sinks));
}
// Whether any of the tokens sees the key.
__device__ __forceinline__ bool chunk_any(const ChunkCall& c, int key, int p0, int p1) {
  return key <= p1 && (c.window == 0 || key > p0 - c.window || key < c.sinks);
}
// Cache row of a key for shard r: a head's elements are at (row * kv_per + g) * 128; -1 on a bad block.
__device__ __forceinline__ int chunk_row(const ChunkAttnParams& p, int r, int blk, int key) {
  return blk >= 0 && blk < p.num_blocks ? (r * p.num_blocks + blk) * p.block_size + key % p.block_size : -1;
}

constexpr int kChunkHd = 128;
// Partial results of a slot: O as [16][rows][8] fp32 (pieces of eight dimensions, so that the
// 32 rows of a warp write 1 KB on end), then [rows][2] (max in the exp2 domain, sum).
// part_rows is a multiple of 8 and the first slot 32-byte aligned: every piece starts on 32 bytes.
__device__ __forceinline__ float* chunk_part_o(const ChunkAttnParams& p, int slot, int row, int d) {
  return p.partials + (size_t)slot * p.part_rows * (kChunkHd + 2) + ((size_t)(d >> 3) * p.part_rows + row) * 8 + (d & 7);
}
__device__ __forceinline__ float2* chunk_part_ml(const ChunkAttnParams& p, int slot, int row) {
  return reinterpret_cast<float2*>(p.partials + (size_t)slot * p.part_rows * (kChunkHd + 2) + (size_t)p.part_rows * kChunkHd) + row;
}


// One warp walks: every lane calls, with the same result.
struct ChunkWalk {
  // requests `lane`, `lane` + 32, .. of a batch of 128 (row of the first new token, new tokens, all tokens;
  // -1 new tokens: bad counts), loaded together
  static constexpr int kStrips = 4;
  int3 mine[kStrips];
  ChunkReq r;
  long long pos, end, begin, per;   // places: where the walk is, where it ends, the first of the item it is in
  int b, head, group, heads, cost;

  static __device__ __forceinline__ int3 counts(const ChunkAttnParams& p, int b) {
    const ChunkReq q = chunk_request(p.call, p.qsl[b], p.qsl[b + 1], p.seq_lens[b]);
    return make_int3(q.q0, q.ok ? q.n : -1, q.ctx + q.n);
  }
  static __device__ __forceinline__ ChunkReq request(const ChunkAttnParams& p, int3 m) {   // none where the counts are bad
    return chunk_request(p.call, m.x, m.x + max(m.y, 0), m.z);
  }
  static __device__ __forceinline__ ChunkReq broadcast(const ChunkAttnParams& p, int3 m, int from) {
    return request(p, make_int3(__shfl_sync(0xffffffffu, m.x, from), __shfl_sync(0xffffffffu, m.y, from),
                                __shfl_sync(0xffffffffu, m.z, from)));
  }
  static __device__ __forceinline__ long long sum(long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }

  __device__ __forceinline__ void load(const ChunkAttnParams& p, int b0, int lane) {
#pragma unroll
    for (int i = 0; i < kStrips; ++i) {
      const int at = b0 + 32 * i + lane;
      mine[i] = at < p.n_reqs ? counts(p, at) : make_int3(0, 0, 0);
    }
  }

  // The CTA's range and the item that holds its first place; load(0) before. CTA 0 reports bad counts.
  __device__ __forceinline__ void start(const ChunkAttnParams& p, int lane) {
    heads = p.t * p.kv_per;
    // a head's places of all requests with an item cost of 0, and its items. A batch's places are kept:
    // they are looked up again for the CTA's first request.
    long long places = 0, items = 0, kept[kStrips];
    int widest = 1;
    for (int b0 = 0; b0 < p.n_reqs; b0 += 32 * kStrips) {
      if (b0 > 0) load(p, b0, lane);
#pragma unroll
      for (int i = 0; i < kStrips; ++i) {
        if (mine[i].y < 0 && blockIdx.x == 0) atomicExch(p.status, kChunkStatusShape);
        const ChunkReq q = request(p, mine[i]);
        kept[i] = chunk_head(p.call, q, 0);
        places += kept[i];
        items += q.groups;
        widest = max(widest, chunk_widest(p.call, q));
      }
    }
    places = heads * sum(places);
    cost = chunk_cost(places, p.call.full, gridDim.x);
    const long long total = places + heads * cost * sum(items);
    per = chunk_per(total, gridDim.x, __reduce_max_sync(0xffffffffu, widest));
    pos = per * blockIdx.x;
    end = min(total, pos + per);
    r = ChunkReq{};
    b = head = group = 0;
    begin = 0;
    // no item of this CTA is continued by others, unless a segment says so below
    if (lane == 0) p.items[blockIdx.x].rows = 0;
    __syncwarp();
    if (pos >= end) return;
    // the request that holds the first place, and the places before it
    long long before = 0, head_places = 1;
    bool found = false;
    for (int b0 = 0; b0 < p.n_reqs && !found; b0 += 32 * kStrips) {
      const bool again = p.n_reqs > 32 * kStrips;
      if (again) load(p, b0, lane);
#pragma unroll
      for (int i = 0; i < kStrips; ++i) {
        if (found) break;
        const ChunkReq q = request(p, mine[i]);
        const long long one = (again ? chunk_head(p.call, q, 0) : kept[i]) + (long long)cost * q.groups, w = heads * one;
        long long pre = w;                            // the strip's places up to and with this lane's
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
          head_places = __shfl_sync(0xffffffffu, one, f);
          r = broadcast(p, mine[i], f);
          found = true;
        } else {
          before += __shfl_sync(0xffffffffu, pre, 31);
        }
      }
    }
    head = (int)((pos - before) / head_places);
    const long long at = pos - before - head * head_places;
    // the last group whose prefix is not past `at`: 32 candidates at a time
    int n = r.groups;
    while (n > 1) {
      const int step = (n + 31) / 32, g = group + lane * step;
      const bool in = g < group + n && chunk_prefix(p.call, r, g, cost) <= at;
      const int last = 31 - __clz(__ballot_sync(0xffffffffu, in));
      n = min(step, n - last * step);
      group += last * step;
    }
    begin = before + head * head_places + chunk_prefix(p.call, r, group, cost);
  }

  // What next() needs, kept elsewhere and taken up again.
  __device__ __forceinline__ void keep(ChunkWalk& at) const {
    at.r = r;
    at.pos = pos;
    at.end = end;
    at.begin = begin;
    at.per = per;
    at.b = b;
    at.head = head;
    at.group = group;
    at.heads = heads;
    at.cost = cost;
  }
  __device__ __forceinline__ void resume(const ChunkWalk& at) { at.keep(*this); }

  // The next segment (b < 0: none is left).
  __device__ __forceinline__ ChunkSegment next(const ChunkAttnParams& p, int lane) {
    ChunkSegment s;
    s.b = -1;
    while (pos < end) {
      const ChunkKeys keys = chunk_item_keys(p.call, r, group);
      const int width = chunk_width(p.call, r, group);
      const long long item = cost + (long long)keys.count * width, p1 = min(item, end - begin);
      const ChunkPart q = chunk_part(pos - begin, p1, cost, width, keys.count, blockIdx.x);
      const int it_head = head, it_group = group, it_b = b;
      const ChunkReq it = r;
      const long long it_begin = begin;
      pos = begin + p1;
      if (p1 == item && pos < end) {                   // on to the next item
        begin = pos;
        if (++group == r.groups) {
          group = 0;
          if (++head == heads) {
            head = 0;
            for (;; b += 32) {                         // the next request with new tokens
              const int next = b + 1 + lane;
              const int3 m = next < p.n_reqs ? counts(p, next) : make_int3(0, 0, 0);
              const unsigned hit = __ballot_sync(0xffffffffu, m.y > 0);
              if (hit != 0u) {
                const int f = __ffs(hit) - 1;
                b += 1 + f;
                r = broadcast(p, m, f);
                break;
              }
              if (b + 32 >= p.n_reqs) {                // cannot be: a place before `end` belongs to a request
                pos = end;
                break;
              }
            }
          }
        }
      }
      if (q.c0 == q.c1) continue;                      // no chunk begins in these places
      s.b = it_b;
      s.r = it_head / p.kv_per;
      s.g = it_head - s.r * p.kv_per;
      s.tok0 = it_group * p.call.tg;
      s.c0 = q.c0;
      s.c1 = q.c1;
      s.q0 = it.q0;
      s.ctx = it.ctx;
      s.part = q.slot;
      const int tokens = min(p.call.tg, it.n - s.tok0);
      s.rows = tokens * p.call.gq;
      s.bad = 0;
      s.skip = keys.skip;
      s.p0 = it.ctx + s.tok0;
      s.p1 = s.p0 + tokens - 1;
      s.pad0 = s.pad1 = 0;
      if (q.c0 == 0 && q.slot >= 0 && lane == 0) {
        const int last = chunk_last(it_begin, cost, width, keys.count, per);
        p.items[blockIdx.x] = TreeItem{s.r, s.g, 0, s.rows, s.q0 + s.tok0, last, 0, 0};
      }
      break;
    }
    return s;
  }
};

}  // namespace tpl
