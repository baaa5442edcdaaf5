// Host build of the tree attention's work split, for tests/test_tree_plan.py.
#include "../tensor_linear_layers_gb300/csrc/tree_plan.h"

extern "C" {
static tpl::TreeReq g_req;
// sets the request that the calls below go by
int plan_request(int q0, int q1, int len, int T, int max_q, int max_len, int gq, int rows, int* out) {
  g_req = tpl::tree_request(q0, q1, len, T, max_q, max_len, gq, rows);
  out[0] = g_req.n;
  out[1] = g_req.chunks;
  out[2] = g_req.groups;
  return g_req.ok ? 1 : 0;
}
int plan_cost(long long chunks, int grid) { return tpl::tree_cost(chunks, grid); }
long long plan_head(int cost) { return tpl::tree_head(g_req, cost); }
long long plan_per(long long total, int grid) { return tpl::tree_per(total, grid); }
void plan_segment(int cost, long long at, long long left, int cta, long long* out) {
  const tpl::TreeSeg s = tpl::tree_segment(g_req, cost, at, left, cta);
  out[0] = s.head;
  out[1] = s.group;
  out[2] = s.c0;
  out[3] = s.c1;
  out[4] = s.part;
  out[5] = s.places;
  out[6] = s.begin;
}
void plan_parts(int group, long long begin, int cost, long long per, int* out) {
  out[0] = tpl::tree_first(begin, cost, per);
  out[1] = tpl::tree_last(g_req, group, begin, cost, per);
}
unsigned plan_window(const int* words, int key, int ctx, int n) { return tpl::tree_window(words, key, ctx, n); }
}
