// The chunk attention's work split on the host: the kernel's walk over a CTA's range, and what the
// merge then reads.
#include <cstdint>
#include <map>
#include <set>
#include <tuple>
#include <vector>

#include "../tensor_linear_layers_gb300/csrc/chunk_plan.h"

using namespace tpl;

extern "C" {

long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) { return chunk_floor_sum(n, m, a, b); }

unsigned sees(int key, int pos, int window, int sinks) { return chunk_sees(key, pos, window, sinks); }

// Keys that an item goes through, in order; returns their number (whole chunks).
int item_keys(int p0, int p1, int window, int sinks, int* out) {
  ChunkCall c{};
  c.window = window;
  c.sinks = sinks;
  const ChunkKeys k = chunk_keys(c, p0, p1);
  for (int x = 0; x < k.count * kChunkKeys; ++x) out[x] = chunk_key(x, k.sc, k.skip);
  return k.count * kChunkKeys;
}

// Bits of the item's keys x to x + 31 to a token, and whether x to x + n - 1 are taken through the masks.
unsigned item_sees(int p0, int p1, int window, int sinks, int x, int pos) {
  ChunkCall c{};
  c.window = window;
  c.sinks = sinks;
  const ChunkKeys k = chunk_keys(c, p0, p1);
  return chunk_item_sees(x, k.sc, k.skip, pos, window, sinks);
}
int item_masked(int p0, int p1, int window, int sinks, int x, int n) {
  ChunkCall c{};
  c.window = window;
  c.sinks = sinks;
  const ChunkKeys k = chunk_keys(c, p0, p1);
  return chunk_masked(c, x, n, k.sc, k.skip, p0, p1);
}

// Head prefixes of a request in closed form against the sum of its items; 0 where all agree.
int prefixes(int n, int ctx, int gq, int rows, int window, int sinks, int cost) {
  ChunkCall c{1 << 24, n, ctx + n, gq, chunk_group_tokens(gq, rows), window, sinks, 2 + (rows + 127) / 128};
  const ChunkReq r = chunk_request(c, 0, n, ctx + n);
  long long at = 0;
  for (int g = 0; g < r.groups; ++g) {
    if (chunk_prefix(c, r, g, cost) != at) return g + 1;
    at += chunk_item(c, r, g, cost);
  }
  return chunk_head(c, r, cost) == at ? 0 : -1;
}

// out: chunks in all, slots the merge reads, slots it reads that this call did not write for that
// item, chunks computed twice or never, CTAs with work, most chunks of a CTA. Returns the grid.
int split(int nsm, int heads, int gq, int rows, int max_q, int max_len, int window, int sinks, int n_reqs, const int* n,
          const int* lens, int* out) {
  int T = 0;
  for (int b = 0; b < n_reqs; ++b) T += n[b];
  ChunkCall c{T, max_q, max_len, gq, chunk_group_tokens(gq, rows), window, sinks, 2 + (rows + 127) / 128};
  std::vector<ChunkReq> reqs;
  int q0 = 0, widest = 1;
  long long places = 0, items = 0;
  for (int b = 0; b < n_reqs; ++b) {
    reqs.push_back(chunk_request(c, q0, q0 + n[b], lens[b]));
    q0 += n[b];
    places += heads * chunk_head(c, reqs[b], 0);
    items += (long long)heads * reqs[b].groups;
    widest = std::max(widest, chunk_widest(c, reqs[b]));
  }
  const int grid = chunk_grid(nsm, n_reqs, heads, max_q, c.tg, max_len);
  const int cost = chunk_cost(places, c.full, grid);
  const long long total = places + cost * items, per = chunk_per(total, grid, widest);
  using Item = std::tuple<int, int, int>;
  std::map<int, Item> slots;
  std::set<std::tuple<int, int, int, int>> done;
  int wrong = 0, busy = 0, most = 0;
  struct Join {
    Item item;
    int cta, last;
  };
  std::vector<Join> joins;
  std::map<Item, std::pair<int, int>> named;
  for (int cta = 0; cta < grid; ++cta) {
    long long pos = per * cta;
    const long long end = std::min(total, pos + per);
    int mine = 0;
    if (pos < end) {
      long long before = 0;
      int b = 0;
      while (before + heads * chunk_head(c, reqs[b], cost) <= pos) before += heads * chunk_head(c, reqs[b++], cost);
      const long long one = chunk_head(c, reqs[b], cost);
      int head = (int)((pos - before) / one);
      const long long at = pos - before - head * one;
      int lo = 0, m = reqs[b].groups;
      while (m > 32) {
        const int step = (m + 31) / 32;
        int last = 0;
        for (int l = 0; l < 32; ++l)
          if (lo + l * step < lo + m && chunk_prefix(c, reqs[b], lo + l * step, cost) <= at) last = l;
        m = std::min(step, m - last * step);
        lo += last * step;
      }
      long long begin = before + head * one + chunk_prefix(c, reqs[b], lo, cost);
      int group = lo;
      for (; group < lo + m - 1 && begin + chunk_item(c, reqs[b], group, cost) <= pos; ++group)
        begin += chunk_item(c, reqs[b], group, cost);
      while (pos < end) {
        const ChunkReq& r = reqs[b];
        const int count = chunk_item_keys(c, r, group).count, width = chunk_width(c, r, group);
        const long long item = cost + (long long)count * width, p1 = std::min(item, end - begin);
        const ChunkPart q = chunk_part((int)(pos - begin), (int)p1, cost, width, count, cta);
        const Item it{b, head, group};
        for (int k = q.c0; k < q.c1; ++k) {
          if (!done.insert({b, head, group, k}).second) ++wrong;
          ++mine;
        }
        if (q.c0 < q.c1 && q.slot >= 0) {
          slots[q.slot] = it;
          // every part names the same CTAs, the first of which begins the item
          const int first = chunk_holder(begin, cost, width, 0, per), last = chunk_holder(begin, cost, width, count - 1, per);
          if (q.c0 == 0) joins.push_back({it, cta, last});
          wrong += (q.c0 == 0) != (cta == first) || (q.c1 == count) != (cta == last) || first == last;
          const auto known = named.insert({it, {first, last}});
          wrong += known.first->second != std::make_pair(first, last);
        }
        pos = begin + p1;
        if (p1 == item && pos < end) {
          begin = pos;
          if (++group == r.groups) {
            group = 0;
            if (++head == heads) {
              head = 0;
              do ++b;
              while (b < n_reqs && reqs[b].groups == 0);
              if (b == n_reqs) break;
            }
          }
        }
      }
    }
    busy += mine > 0;
    most = std::max(most, mine);
  }
  int all = 0;
  for (int b = 0; b < n_reqs; ++b)
    for (int g = 0; g < reqs[b].groups; ++g) all += heads * chunk_item_keys(c, reqs[b], g).count;
  wrong += all - (int)done.size();
  int reads = 0, holes = 0;
  for (const Join& j : joins)
    for (int x = j.cta; x <= j.last; ++x, ++reads) {
      const auto at = slots.find(x == j.cta ? 2 * x + 1 : 2 * x);
      if (at == slots.end() || at->second != j.item) ++holes;
    }
  // every item that was cut is joined
  std::set<Item> joined;
  for (const Join& j : joins) joined.insert(j.item);
  for (const auto& s : slots) holes += joined.count(s.second) == 0;
  out[0] = all;
  out[1] = reads;
  out[2] = holes;
  out[3] = wrong;
  out[4] = busy;
  out[5] = most;
  return grid;
}
}
