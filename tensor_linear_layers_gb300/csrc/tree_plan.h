// Work split of the tree attention, shared by its kernels and a host test.
//
// Request b has units(b) = t * kv_per * groups items (a kv head of a shard and a group of query
// rows), each of chunks(b) = ceil(L / 128) chunks of 128 keys. An item takes its chunks' places
// on a line, after kTreeItemCost more for what it costs besides them (its queries, the first
// products, its output); items and requests follow each other in order. CTA c of the grid
// takes places [c * per, (c + 1) * per), so the CTAs have the same work whatever the lengths.
// An item that crosses a boundary is computed in parts: CTA c writes the part that continues
// an item begun by an earlier CTA to slot 2 c, the part that begins one it does not finish to
// slot 2 c + 1, and the merge kernel joins them in chunk order.
#pragma once

#ifdef __CUDACC__
#define TPL_HD __host__ __device__ __forceinline__
#else
#define TPL_HD inline
#endif

namespace tpl {

constexpr int kTreeChunk = 128;   // keys of one chunk

struct TreeReq {
  int q0, n, len, chunks, groups;
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
  return r;
}

// Places of an item.
constexpr int kTreeItemCost = 1;
TPL_HD long long tree_item(int chunks) { return chunks > 0 ? chunks + kTreeItemCost : 0; }

// Places per CTA.
TPL_HD long long tree_per(long long total, int grid) { return total > 0 ? (total + grid - 1) / grid : 1; }

struct TreeSeg {
  long long unit;                 // item within the request
  long long places;               // taken from the line
  int c0, c1;                     // its chunks [c0, c1); none where the places are the item's first ones alone
  int part;                       // slot of the partial result, or -1: the item is whole
};
// The segment of CTA cta that starts at place `at` of its request, `left` places before the CTA's end.
TPL_HD TreeSeg tree_segment(long long at, int chunks, long long left, int cta) {
  TreeSeg s;
  const long long item = tree_item(chunks);
  s.unit = at / item;
  const int p0 = (int)(at - s.unit * item);
  s.places = item - p0 < left ? item - p0 : left;
  const int p1 = p0 + (int)s.places;
  s.c0 = p0 > kTreeItemCost ? p0 - kTreeItemCost : 0;
  s.c1 = p1 > kTreeItemCost ? p1 - kTreeItemCost : 0;
  s.part = s.c0 > 0 ? 2 * cta : s.c1 < chunks ? 2 * cta + 1 : -1;
  return s;
}

// The CTAs that hold the first and the last chunk of the item that begins at place `begin`.
TPL_HD int tree_first(long long begin, long long per) { return (int)((begin + kTreeItemCost) / per); }
TPL_HD int tree_last(long long begin, int chunks, long long per) { return (int)((begin + kTreeItemCost + chunks - 1) / per); }

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
