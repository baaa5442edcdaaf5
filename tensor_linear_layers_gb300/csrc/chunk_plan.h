// Work split of the attention of chunks of new tokens, shared by its kernel and a host test.
//
// Request b has t * kv_per * groups items: a kv head of a shard and a group of up to `tg` whole
// tokens, whose tg * gq query rows (gq: q heads of the kv head) fill one or two tiles of 128. The
// tokens of group G are those from tg * G on, the first at position p0 and the last at p1. The keys that
// the item goes through, in order, are
//   the first `sinks` tokens                  [0, sc),   sc = sinks up to a multiple of 16   (with a window)
//   and those of its window up to its end     [lo, p1],  lo = p0 - window + 1 down to a multiple of 16
// (or all of [0, p1] where these meet): key x of the item is key x, or x + skip from x = sc on, skip =
// max(0, lo - sc). They go by in chunks of 128, so that a window of 1024 and a few sinks take nine chunks,
// not the ten or eleven that they touch; 16 keys in a row stay one after another in their pages.
//
// Items lie on a line, requests in order, head by head and group by group. A chunk takes
// 2 + tiles places, an item `cost` more before its first chunk for what it costs besides them.
// CTA c of the grid takes the chunks whose first place is in [c * per, (c + 1) * per), so the CTAs
// have the same work whatever the lengths, windows and numbers of new tokens. No CTA has fewer places than the
// call's widest chunk: inside an item every CTA then holds some chunk's first place and writes
// its slot. An item that crosses a boundary is computed in parts: CTA c writes the part that
// continues an item begun by an earlier CTA to slot 2 c, the part that begins one it does not
// finish to slot 2 c + 1; they are joined in order.
#pragma once

#include <algorithm>

#ifndef TPL_HD
#ifdef __CUDACC__
#define TPL_HD __host__ __device__ __forceinline__
#else
#define TPL_HD inline
#endif
#endif

namespace tpl {

constexpr int kChunkKeys = 128;
// Places that an item costs besides its chunks: the drain of its products and its output. Measured at two row
// tiles as some 3.5 us against 1.65 us of a chunk, 4 places (a prompt of 4096 tokens: 145 us without this cost, 126
// with 6 to 10 places, 128 with 13 or 16).
TPL_HD int chunk_item_cost(int full) { return full == 4 ? 10 : 4; }

// a / b of places (a >= 0, b > 0): in 32 bits where they fit, a quarter of the instructions
TPL_HD long long chunk_div(long long a, long long b) {
  return ((a | b) >> 31) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// sum of floor((a i + b) / m) over i = 0 .. n - 1; n a + b < 2^31, all >= 0, m > 0: by Euclid's
// steps on (a, m), each of which exchanges the axes of the lattice points under the line
TPL_HD long long chunk_floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  long long s = 0;
  if (n == 0) return 0;
  for (;;) {
    const unsigned qa = m == (unsigned)kChunkKeys ? a / kChunkKeys : a / m, qb = m == (unsigned)kChunkKeys ? b / kChunkKeys : b / m;
    s += (long long)qa * ((long long)n * (n - 1LL) / 2) + (long long)qb * n;
    a -= qa * m;
    b -= qb * m;
    const unsigned top = a * n + b;
    if (top < m) return s;
    n = m == (unsigned)kChunkKeys ? top / kChunkKeys : top / m;
    b = top - n * m;
    const unsigned x = a;
    a = m;
    m = x;
  }
}

// What the groups of a call have in common.
struct ChunkCall {
  int T, max_query_len, max_seq_len;
  int gq, tg;                       // q heads of a kv head; whole tokens of a group
  int window, sinks;                // 0: none
  int full;                         // places of a chunk of a full group: 2 + its tiles
};
// rows_per_group: 8, 128 or 256, at least gq
TPL_HD int chunk_group_tokens(int gq, int rows_per_group) { return rows_per_group / gq; }

struct ChunkReq {
  int q0, n, ctx, groups;
  int last;                         // places of a chunk of the last group
  bool ok;                          // the counts fit the call
};
TPL_HD ChunkReq chunk_request(const ChunkCall& c, int q0, int q1, int len) {
  ChunkReq r;
  r.q0 = q0;
  r.ok = q0 >= 0 && q1 >= q0 && q1 <= c.T && q1 - q0 <= c.max_query_len && len >= q1 - q0 && len <= c.max_seq_len;
  r.n = r.ok ? q1 - q0 : 0;
  r.ctx = r.ok ? len - r.n : 0;
  r.groups = (r.n + c.tg - 1) / c.tg;
  r.last = 2 + ((r.n - (r.groups - 1) * c.tg) * c.gq + 127) / 128;
  return r;
}

// The keys of one item.
constexpr int kChunkUnit = 16;      // keys that stay together
struct ChunkKeys {
  int count, sc, skip;              // chunks of the item; its key x >= sc is key x + skip
};
TPL_HD int chunk_sinks(const ChunkCall& c) {
  return c.window > 0 ? (c.sinks + kChunkUnit - 1) / kChunkUnit * kChunkUnit : 0;
}
TPL_HD int chunk_key(int x, int sc, int skip) { return x + (x >= sc ? skip : 0); }
TPL_HD ChunkKeys chunk_keys(const ChunkCall& c, int p0, int p1) {
  ChunkKeys k;
  k.sc = chunk_sinks(c);
  const int lo = c.window > 0 && p0 >= c.window ? (p0 - c.window + 1) / kChunkUnit * kChunkUnit : 0;
  k.skip = lo > k.sc ? lo - k.sc : 0;
  k.count = (p1 - k.skip) / kChunkKeys + 1;
  return k;
}
TPL_HD ChunkKeys chunk_item_keys(const ChunkCall& c, const ChunkReq& r, int group) {
  const int t0 = group * c.tg, t1 = t0 + c.tg < r.n ? t0 + c.tg : r.n;
  return chunk_keys(c, r.ctx + t0, r.ctx + t1 - 1);
}
TPL_HD int chunk_width(const ChunkCall& c, const ChunkReq& r, int group) { return group < r.groups - 1 ? c.full : r.last; }
// Places of one item.
TPL_HD long long chunk_item(const ChunkCall& c, const ChunkReq& r, int group, int cost) {
  return cost + (long long)chunk_item_keys(c, r, group).count * chunk_width(c, r, group);
}
// Places of a head's first m items, all of them full groups (m < groups).
TPL_HD long long chunk_prefix(const ChunkCall& c, const ChunkReq& r, int m, int cost) {
  if (m <= 0) return 0;
  // the first g0 groups skip nothing: their chunks are quotients of a line by 128
  long long g0 = m;
  const int sc = chunk_sinks(c);
  if (c.window > 0) {
    const long long at = (long long)sc + kChunkUnit + c.window - 1 - r.ctx;   // from a = p0 - window + 1 = sc + 16 on
    g0 = at > 0 ? (at + c.tg - 1) / c.tg : 0;
    if (g0 > m) g0 = m;
  }
  long long n = m + chunk_floor_sum((unsigned)g0, kChunkKeys, c.tg, r.ctx + c.tg - 1);
  if (g0 < m) {
    // the others go through sc + window + tg - 1 keys and a mod 16 more
    const int rest = (int)(m - g0), keys = c.window + c.tg - 2 + sc, edge = kChunkKeys - keys % kChunkKeys;
    n += (long long)rest * (keys / kChunkKeys);
    if (edge < kChunkUnit) {                         // one chunk more where a mod 16 >= edge
      const int a = (int)(r.ctx + g0 * c.tg - c.window + 1);
      n += chunk_floor_sum(rest, kChunkUnit, c.tg, a + kChunkUnit - edge) - chunk_floor_sum(rest, kChunkUnit, c.tg, a);
    }
  }
  return (long long)m * cost + n * c.full;
}
// Places of all items of one head.
TPL_HD long long chunk_head(const ChunkCall& c, const ChunkReq& r, int cost) {
  return r.groups > 0 ? chunk_prefix(c, r, r.groups - 1, cost) + chunk_item(c, r, r.groups - 1, cost) : 0;
}
TPL_HD int chunk_widest(const ChunkCall& c, const ChunkReq& r) { return r.groups > 1 ? c.full : r.groups > 0 ? r.last : 0; }

// Few chunks per CTA: they are spread over as many CTAs as there are, so an item costs nothing besides them (one
// request of 4000 keys 12.4 us, 12.8 with a cost).
TPL_HD int chunk_cost(long long places, int full, int grid) { return places >= 4LL * full * grid ? chunk_item_cost(full) : 0; }
TPL_HD long long chunk_per(long long total, int grid, int widest) {
  const long long even = chunk_div(total + grid - 1, grid);
  return even > widest ? even : widest;
}

// Part of the item whose places are [0, cost + count * width): those from p0 on that lie before p1.
struct ChunkPart {
  int c0, c1;                       // the item's chunks that begin there
  int slot;                         // slot of the partial result, or -1: the item is whole
};
// (an item has under 2^23 places: 2^19 chunks of up to four)
TPL_HD int chunk_before(int place, int cost, int width) {   // chunks that begin before a place of their item
  const unsigned x = place > cost ? (unsigned)(place - cost + width - 1) : 0u;
  return (int)(width == 4 ? x / 4u : width == 3 ? x / 3u : x / (unsigned)width);
}
TPL_HD ChunkPart chunk_part(int p0, int p1, int cost, int width, int count, int cta) {
  ChunkPart s;
  s.c0 = chunk_before(p0, cost, width);
  s.c1 = chunk_before(p1, cost, width);
  s.slot = s.c0 > 0 ? 2 * cta : s.c1 < count ? 2 * cta + 1 : -1;
  return s;
}
// The CTA that holds chunk j of an item whose first place is `begin`.
TPL_HD int chunk_holder(long long begin, int cost, int width, int j, long long per) {
  return (int)chunk_div(begin + cost + (long long)j * width, per);
}

// CTAs of the grid: as many as run at once, no more than a call of these bounds has chunks.
inline int chunk_grid(int nsm, int n_reqs, int heads, int max_query_len, int tg, int max_seq_len) {
  const double groups = (max_query_len + tg - 1) / tg;
  const double chunks = (double)n_reqs * heads * groups * ((max_seq_len + kChunkKeys - 1) / kChunkKeys);
  return chunks < nsm ? (int)chunks : nsm;
}

// Visibility of the 32 keys from `key` on to a token at position pos, as bits.
TPL_HD unsigned chunk_low(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }
TPL_HD unsigned chunk_sees(int key, int pos, int window, int sinks) {
  unsigned bits = chunk_low(pos - key + 1);
  if (window > 0) bits &= ~chunk_low(pos - window + 1 - key) | chunk_low(sinks - key);
  return bits;
}

// The same for keys x to x + 31 of an item (x a multiple of 16).
TPL_HD unsigned chunk_item_sees(int x, int sc, int skip, int pos, int window, int sinks) {
  unsigned bits = chunk_sees(x + skip, pos, window, sinks);
  if (skip > 0 && x < sc) {          // the sinks, long past, and what fills their last unit
    const unsigned first = chunk_low(sc - x);
    bits = (bits & ~first) | (chunk_low(sinks - x) & first);
  }
  return bits;
}
// Whether keys x to x + n - 1 of an item may be seen by some of its tokens and not by others, or by none.
TPL_HD bool chunk_masked(const ChunkCall& c, int x, int n, int sc, int skip, int p0, int p1) {
  return x + n - 1 + skip > p0 || (c.window > 0 && x + n > c.sinks && ((skip > 0 && x < sc) || x + skip <= p1 - c.window));
}

}  // namespace tpl
