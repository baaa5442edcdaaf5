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
  int part, rows, bad, skip;         // partial slot or -1; query rows; V not finite; keys left out from key sc of the item on
  int p0, p1, first, last;           // positions of the group's first and last token; of a part: the item's first and last CTA
};
static_assert(sizeof(ChunkSegment) == 64, "unit slots");


constexpr int kChunkStatusShape = -2;   // TP_ERR_SHAPE

// A key that some tokens (at positions p0 to p1) see and others do not, of those that any sees.
__device__ __forceinline__ bool chunk_partly(const ChunkCall& c, int key, int p0, int p1) {
  return key > p0 || (c.window > 0 && key <= p1 - c.window && key >= c.sinks);
}
// Whether chunk j of an item has such keys.
__device__ __forceinline__ bool chunk_mixed(const ChunkCall& c, int j, int sc, int skip, int p0, int p1) {
  return p1 > p0 && chunk_masked(c, j * kChunkKeys, kChunkKeys, sc, skip, p0, p1);
}
// Whether any of the tokens sees the key.
__device__ __forceinline__ bool chunk_any(const ChunkCall& c, int key, int p0, int p1) {
  return key <= p1 && (c.window == 0 || key > p0 - c.window || key < c.sinks);
}
// Page of a key: key / block_size as a product with 2^32 / block_size rounded up, too large by one at most
// (key < 2^26: the product is off by less than 2^-6).
__device__ __forceinline__ int chunk_page(const ChunkAttnParams& p, int key) {
  if (p.block_size == 1) return key;
  const int q = (int)__umulhi((unsigned)key, p.block_magic);
  return q * p.block_size > key ? q - 1 : q;
}
// Cache row of a key for shard r: a head's elements are at (row * kv_per + g) * 128; -1 on a bad block.
__device__ __forceinline__ int chunk_row(const ChunkAttnParams& p, int r, int blk, int key) {
  return blk >= 0 && blk < p.num_blocks ? (r * p.num_blocks + blk) * p.block_size + key - chunk_page(p, key) * p.block_size : -1;
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


// One warp walks: every lane calls, with the same result. The code is kept short, each function at one
// place: it runs once per CTA, and what bounds it is the fetch of its instructions (with four strips of
// requests unrolled the first segment came after 7 us of a prompt's 150). ONE: every request is one group.
template <bool ONE>
struct ChunkWalk {
  int3 first;                       // request `lane`: row of the first new token, new tokens (-1: bad counts), all tokens
  ChunkReq r;
  long long pos, end, begin, per;   // places: where the walk is, where it ends, the first of the item it is in
  int b, head, group, heads, cost;

  static __device__ __forceinline__ int3 counts(const ChunkAttnParams& p, int b) {
    if (b >= p.n_reqs) return make_int3(0, 0, 0);
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
  // sum over the lanes up to and with this one
  static __device__ __forceinline__ long long scan(long long v, int lane) {
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += up;
    }
    return v;
  }

  __device__ __forceinline__ void load(const ChunkAttnParams& p, int lane) { first = counts(p, lane); }

  // The CTA's range and the item that holds its first place; load() before. CTA 0 reports bad counts.
  __device__ __forceinline__ void start(const ChunkAttnParams& p, int lane) {
    heads = p.t * p.kv_per;
    r = ChunkReq{};
    b = head = group = cost = 0;
    begin = pos = end = 0;
    // no item of this CTA is continued by others, unless a segment says so below
    if (p.counters == nullptr && lane == 0) p.items[blockIdx.x].rows = 0;
    __syncwarp();
    // Twice over the requests, 32 at a time: a head's places of all of them with an item cost of 0, and its
    // items; then the request that holds the CTA's first place, and the places before it.
    long long places = 0, before = 0, one = 0;
    long long items = 0;
    int widest = 1;
    bool found = false;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      int3 m = first;
#pragma unroll 1
      for (int b0 = 0; b0 < p.n_reqs && !found; b0 += 32) {
        const int3 mine = m;
        if (b0 + 32 < p.n_reqs) m = counts(p, b0 + 32 + lane);       // (the next ones, early)
        const ChunkReq q = request(p, mine);
        if (pass == 0 || p.n_reqs > 32)
          one = ONE ? (q.groups > 0 ? chunk_item(p.call, q, 0, cost) : 0) : chunk_head(p.call, q, cost);
        else
          one += q.groups * (long long)cost;                         // (the first pass's, with a cost of 0)
        const long long pre = scan(heads * one, lane);               // the places up to and with this lane's
        if (pass == 0) {
          if (mine.y < 0 && blockIdx.x == 0) atomicExch(p.status, kChunkStatusShape);
          places += __shfl_sync(0xffffffffu, pre, 31);
          items += q.groups;
          widest = max(widest, chunk_widest(p.call, q));
        } else {
          const unsigned hit = __ballot_sync(0xffffffffu, before + pre > pos);
          if (hit != 0u) {
            const int f = __ffs(hit) - 1;
            b = b0 + f;
            before += __shfl_sync(0xffffffffu, pre - heads * one, f);
            one = __shfl_sync(0xffffffffu, one, f);
            r = broadcast(p, mine, f);
            found = true;
          } else {
            before += __shfl_sync(0xffffffffu, pre, 31);
          }
        }
      }
      if (pass == 0) {
        cost = chunk_cost(places, p.call.full, gridDim.x);
        const long long total = places + heads * cost * __shfl_sync(0xffffffffu, scan(items, lane), 31);
        per = chunk_per(total, gridDim.x, __reduce_max_sync(0xffffffffu, widest));
        pos = per * blockIdx.x;
        end = min(total, pos + per);
        if (pos >= end) return;
      }
    }
    // its head and the last group whose places are not all before
    long long at = pos - before;
    while (at >= 32 * one) {
      at -= 32 * one;
      head += 32;
    }
    const int h = 31 - __clz(__ballot_sync(0xffffffffu, lane * one <= at));
    head += h;
    at -= h * one;
    begin = pos - at;                                  // the head's first place; then its group's
    if constexpr (ONE) return;
    int n = r.groups;
    long long skipped = 0;
#pragma unroll 1
    while (n > 32) {                                   // 32 candidates at a time
      const int step = (n + 31) / 32, g = group + lane * step;
      const long long prefix = chunk_prefix(p.call, r, min(g, r.groups - 1), cost);
      const int last = 31 - __clz(__ballot_sync(0xffffffffu, g < group + n && prefix <= at));
      n = min(step, n - last * step);
      group += last * step;
      skipped = __shfl_sync(0xffffffffu, prefix, last);
    }
    const long long w = lane < n ? chunk_item(p.call, r, group + lane, cost) : 0;      // then 32 items' places added up
    const long long pre = skipped + scan(w, lane) - w;
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, lane < n && pre <= at));
    group += last;
    begin += __shfl_sync(0xffffffffu, pre, last);
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
#pragma unroll 1
    while (pos < end) {
      const ChunkKeys keys = chunk_item_keys(p.call, r, group);
      const int width = chunk_width(p.call, r, group), item = cost + keys.count * width, p0 = (int)(pos - begin);
      const bool whole = end - begin >= item;
      const int p1 = whole ? item : (int)(end - begin);
      const ChunkPart q = chunk_part(p0, p1, cost, width, keys.count, blockIdx.x);
      if (q.c0 < q.c1) {                               // else no chunk begins in these places
        s.b = b;
        s.r = head / p.kv_per;
        s.g = head - s.r * p.kv_per;
        s.tok0 = group * p.call.tg;
        s.c0 = q.c0;
        s.c1 = q.c1;
        s.q0 = r.q0;
        s.ctx = r.ctx;
        s.part = q.slot;
        const int tokens = min(p.call.tg, r.n - s.tok0);
        s.rows = tokens * p.call.gq;
        s.bad = 0;
        s.skip = keys.skip;
        s.p0 = r.ctx + s.tok0;
        s.p1 = s.p0 + tokens - 1;
        s.first = s.last = blockIdx.x;
        if (q.slot >= 0) {
          s.first = chunk_holder(begin, cost, width, 0, per);
          s.last = chunk_holder(begin, cost, width, keys.count - 1, per);
          if (p.counters == nullptr && q.c0 == 0 && lane == 0) p.items[blockIdx.x] = TreeItem{s.r, s.g, 0, s.rows, s.q0 + s.tok0, s.last, 0, 0};
        }
      }
      pos = begin + p1;
      if (whole && pos < end) {                        // on to the next item
        begin = pos;
        if (++group == r.groups) {
          group = 0;
          if (++head == heads) {
            head = 0;
#pragma unroll 1
            for (;; b += 32) {                         // the next request with new tokens
              const int3 m = counts(p, b + 1 + lane);
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
      if (s.b >= 0) break;
    }
    return s;
  }
};

}  // namespace tpl
