// Work split of the tree attention, shared by its kernels and a host test.
//
// Request b has t * kv_per * groups items: a kv head of a shard and a group of query rows,
// up to 128 or 256 of them in one or two tiles of 128. Every item takes its chunks of 128 keys,
// ceil(L / 128). Items lie on a line, head by head and group by group, requests in order. A
// chunk takes 2 + tiles places (the second tile's products and softmax against the copies,
// which both share: 1.6 us against 1.2 us), and an item kTreeItemCost more before its first
// chunk for what it costs besides them (its queries, the first products, its output). CTA c
// of the grid takes the chunks whose first place is in [c * per, (c + 1) * per), so the CTAs
// have the same work whatever the lengths (32 requests of 256 to 4096 keys: 56.1 us, 59.8 with
// chunks alone counted). A CTA has at least the places of the call's widest chunk: with fewer,
// a CTA inside an item could hold no chunk's first place, and so leave its slot unwritten for
// the merge, which reads the slots of all CTAs from an item's first to its last. Where there is little work (fewer than four chunks per CTA) an item
// costs nothing besides its chunks: they are spread over as many CTAs as there are (one request
// of 508 keys: 13.0 us, 13.7 with the cost). An item that crosses a boundary is computed in parts: CTA c writes the part that
// continues an item begun by an earlier CTA to slot 2 c, the part that begins one it does not
// finish to slot 2 c + 1, and the merge kernel joins them in chunk order.
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

constexpr int kTreeChunk = 128;   // keys of one chunk

constexpr int kTreeItemCost = 4;  // places
constexpr int kTreeWidest = 4;    // places of the widest chunk there is (two tiles of rows)

// CTAs of the grid: one per SM, no more than a call of these bounds has chunks. heads: kv heads over
// all shards; max_rows: query rows of one of them; rows_per_group: those of one item.
inline int tree_grid(int nsm, int n_reqs, int heads, int max_rows, int rows_per_group, int max_seq_len) {
  const long long groups = (max_rows + rows_per_group - 1) / rows_per_group;
  const long long chunks = (long long)n_reqs * heads * groups * ((max_seq_len + kTreeChunk - 1) / kTreeChunk);
  return (int)std::min<long long>(nsm, chunks);
}

struct TreeReq {
  int q0, n, len, chunks, groups;
  int full, last;                 // places of a chunk in a full group and in the last one
  bool ok;                        // the counts fit the call (a request without drafts does too, and has no work)
};
// rows_per_group: query rows (tokens x q heads of one kv head) of one item.
TPL_HD TreeReq tree_request(int q0, int q1, int len, int T, int max_query_len, int max_seq_len, int gq,
                            int rows_per_group) {
  TreeReq r;
  r.q0 = q0;
  r.len = len;
  r.ok = q0 >= 0 && q1 >= q0 && q1 <= T && q1 - q0 <= max_query_len && len >= q1 - q0 && len <= max_seq_len;
  r.n = r.ok ? q1 - q0 : 0;
  r.chunks = r.n > 0 ? (len + kTreeChunk - 1) / kTreeChunk : 0;
  r.groups = r.n > 0 ? (r.n * gq + rows_per_group - 1) / rows_per_group : 0;
  r.full = 2 + rows_per_group / 128;
  r.last = 2 + (r.n * gq - (r.groups - 1) * rows_per_group + 127) / 128;
  return r;
}

// Places of one head's items. cost: kTreeItemCost, or 0.
TPL_HD long long tree_head(const TreeReq& r, int cost) {
  return r.groups > 0 ? (long long)(r.groups - 1) * (cost + r.chunks * r.full) + cost + r.chunks * r.last : 0;
}

// Places of the widest chunk of a request (0: no work).
TPL_HD int tree_widest(const TreeReq& r) { return r.groups > 1 ? r.full : r.groups > 0 ? r.last : 0; }

// What an item costs besides its chunks, and the places per CTA.
TPL_HD int tree_cost(long long chunks, int grid) { return chunks >= 4LL * grid ? kTreeItemCost : 0; }
// widest: the most places that a chunk of any request takes (tree_widest). Where all chunks take as
// many, each still has a CTA of its own when there are CTAs enough; held to the widest chunk there
// is, chunks of three places would go two to some CTAs.
TPL_HD long long tree_per(long long total, int grid, int widest = kTreeWidest) {
  const long long even = (total + grid - 1) / grid;
  return even > widest ? even : widest;
}

struct TreeSeg {
  int head, group;
  long long places;               // taken from the line
  int c0, c1;                     // the item's chunks [c0, c1); none where no chunk begins in the places
  int part;                       // slot of the partial result, or -1: the item is whole
  long long begin;                // the item's first place in its request
};
// The segment of CTA cta that starts at place `at` of its request, `left` places before the CTA's end.
TPL_HD TreeSeg tree_segment(const TreeReq& r, int cost, long long at, long long left, int cta) {
  TreeSeg s;
  const long long head = tree_head(r, cost);
  const int item_full = cost + r.chunks * r.full;
  s.head = (int)(at / head);
  const int in = (int)(at - s.head * head);
  s.group = in / item_full < r.groups - 1 ? in / item_full : r.groups - 1;
  const int p0 = in - s.group * item_full, w = s.group < r.groups - 1 ? r.full : r.last;
  s.begin = s.head * head + (long long)s.group * item_full;
  const int item = cost + r.chunks * w;
  s.places = item - p0 < left ? item - p0 : left;
  const int p1 = p0 + (int)s.places;
  s.c0 = p0 > cost ? (p0 - cost + w - 1) / w : 0;
  s.c1 = p1 > cost ? (p1 - cost + w - 1) / w : 0;
  s.part = s.c0 > 0 ? 2 * cta : s.c1 < r.chunks ? 2 * cta + 1 : -1;
  return s;
}

// The CTAs that hold the first and the last chunk of the item of group `group` that begins at place `begin` of the line.
TPL_HD int tree_first(long long begin, int cost, long long per) { return (int)((begin + cost) / per); }
TPL_HD int tree_last(const TreeReq& r, int group, long long begin, int cost, long long per) {
  return (int)((begin + cost + (long long)(r.chunks - 1) * (group < r.groups - 1 ? r.full : r.last)) / per);
}

// Visibility of the 32 keys from position key on, as bits, to a drafted token with mask row
// `words`: cached positions (before ctx) always, the n drafted ones by their bits, none after.
template <class Words>
TPL_HD unsigned tree_window(const Words& words, int key, int ctx, int n) {
  const int rel = key - ctx;      // draft index of the first key
  if (rel <= -32) return 0xffffffffu;
  if (rel >= n) return 0u;
  const int w = rel < 0 ? 0 : rel >> 5, sh = rel < 0 ? 0 : rel & 31;
  unsigned bits = (unsigned)words[w] >> sh;
  if (sh != 0 && 32 * (w + 1) < n) bits |= (unsigned)words[w + 1] << (32 - sh);
  const int have = n - (rel < 0 ? 0 : rel);   // drafts from that one on
  if (have < 32) bits &= (1u << have) - 1u;
  if (rel < 0) bits = (bits << -rel) | ((1u << -rel) - 1u);
  return bits;
}

}  // namespace tpl
