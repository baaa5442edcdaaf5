// The tree attention's walk over its line of chunks, and the slots that its merge reads, for
// tests/test_tree_split.py: what warp 2 of every CTA and the merge kernel do, on tree_plan.h.
#include <map>
#include <set>
#include <tuple>
#include <vector>

#include "../tensor_linear_layers_gb300/csrc/tree_plan.h"

extern "C" {
// out: chunks of all items, slots the merge reads, of these not written by this call (or by another
// item), chunks computed twice or never, CTAs with work, most chunks of a CTA. Returns the grid.
int split(int nsm, int heads, int gq, int rows, int max_q, int max_len, int reqs, const int* n, const int* len, int* out) {
  using Item = std::tuple<int, int, int>;   // request, head, group
  const int grid = tpl::tree_grid(nsm, reqs, heads, max_q * gq, rows, max_len);
  std::vector<tpl::TreeReq> req;
  long long chunks = 0, places = 0, items = 0;
  int widest = 1;
  for (int b = 0; b < reqs; ++b) {
    req.push_back(tpl::tree_request(0, n[b], len[b], n[b], max_q, max_len, gq, rows));
    const tpl::TreeReq& q = req.back();
    if (!q.ok) return -1;
    chunks += (long long)q.groups * q.chunks;
    places += tpl::tree_head(q, 0);
    items += q.groups;
    if (tpl::tree_widest(q) > widest) widest = tpl::tree_widest(q);
  }
  const int cost = tpl::tree_cost(heads * chunks, grid);
  const long long total = heads * (places + cost * items), per = tpl::tree_per(total, grid, widest);
  std::map<int, Item> slots;
  std::map<int, std::pair<Item, int>> unfinished;   // of a CTA: its item and the last CTA with a part of it
  std::set<std::tuple<Item, int>> seen;
  int doubled = 0, busy = 0, most = 0;
  for (int cta = 0; cta < grid; ++cta) {
    long long pos = per * cta, before = 0;
    const long long end = total < pos + per ? total : pos + per;
    int b = 0, mine = 0;
    while (pos < end) {
      while (pos - before >= heads * tpl::tree_head(req[b], cost)) before += heads * tpl::tree_head(req[b++], cost);
      const tpl::TreeSeg s = tpl::tree_segment(req[b], cost, pos - before, end - pos, cta);
      pos += s.places;
      if (s.c0 == s.c1) continue;
      const Item item(b, s.head, s.group);
      for (int c = s.c0; c < s.c1; ++c) doubled += seen.insert({item, c}).second ? 0 : 1;
      mine += s.c1 - s.c0;
      if (s.part >= 0) slots[s.part] = item;
      if (s.part >= 0 && s.c0 == 0)
        unfinished[cta] = {item, tpl::tree_last(req[b], s.group, before + s.begin, cost, per)};
    }
    busy += mine > 0;
    most = mine > most ? mine : most;
  }
  int reads = 0, holes = 0;
  for (const auto& u : unfinished)
    for (int c = u.first; c <= u.second.second; ++c) {
      const auto it = slots.find(c == u.first ? 2 * c + 1 : 2 * c);
      ++reads;
      holes += it == slots.end() || it->second != u.second.first;
    }
  out[0] = (int)(heads * chunks);
  out[1] = reads;
  out[2] = holes;
  out[3] = doubled + (int)(heads * chunks - (long long)seen.size());
  out[4] = busy;
  out[5] = most;
  return grid;
}
}
