// Host build of the tree attention's work split, for tests/test_tree_plan.py.
#include "../tensor_linear_layers_gb300/csrc/tree_plan.h"

extern "C" {
int plan_request(int q0, int q1, int len, int T, int max_q, int max_len, int gq, int rows, int* out) {
  const tpl::TreeReq r = tpl::tree_request(q0, q1, len, T, max_q, max_len, gq, rows);
  out[0] = r.n;
  out[1] = r.chunks;
  out[2] = r.groups;
  return r.ok ? 1 : 0;
}
long long plan_item(int chunks) { return tpl::tree_item(chunks); }
long long plan_per(long long total, int grid) { return tpl::tree_per(total, grid); }
void plan_segment(long long at, int chunks, long long left, int cta, long long* out) {
  const tpl::TreeSeg s = tpl::tree_segment(at, chunks, left, cta);
  out[0] = s.unit;
  out[1] = s.c0;
  out[2] = s.c1;
  out[3] = s.part;
  out[4] = s.places;
}
void plan_parts(long long begin, int chunks, long long per, int* out) {
  out[0] = tpl::tree_first(begin, per);
  out[1] = tpl::tree_last(begin, chunks, per);
}
unsigned plan_window(const int* words, int key, int ctx, int n) { return tpl::tree_window(words, key, ctx, n); }
}
