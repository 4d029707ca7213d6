// Host-side probe of the row operators' plans, run without a GPU by
// tests/test_rows_plan.py. Reads commands from stdin, one result per line:
//   p <mode> <q_rows> <len>   -> splits and whether the next kernel is let go early
//   c <rows>                  -> whether a cross attention goes a token a unit
//   t <rows> <groups> <keys>  -> query tokens of a row tile; keys 0: the expected length
// for the handle that the arguments describe:
//   rows_probe <batch> <H_q> <H_kv> <d> <dtype> <max_pages> <page> <SMs> <active[1..16]>
#include <stdio.h>
#include <stdlib.h>

#include "rows_plan.cuh"

using namespace fastocr;

int main(int argc, char** argv) {
  if (argc != 9 + kMaxSplits) return 2;
  auto arg = [&](int i) { return atoi(argv[i]); };
  fastocr_handle h;
  memset(&h, 0, sizeof(h));
  h.dims.batch = arg(1);
  h.dims.num_q_heads = arg(2);
  h.dims.num_kv_heads = arg(3);
  h.dims.head_dim = arg(4);
  h.dims.dtype = arg(5);
  h.dims.max_pages_per_seq = arg(6);
  h.dims.page_size = arg(7);
  h.dims.num_layers = 1;
  h.log2_page = ilog2_exact(arg(7));
  h.num_sms = arg(8);
  for (int c = 1; c <= kMaxSplits; ++c) h.active[c] = arg(8 + c);
  h.max_splits = kMaxSplits;
  for (int v = 0; v < kNumVariants; ++v) h.max_splits_v[v] = kMaxSplits;
  char cmd[4];
  while (scanf("%3s", cmd) == 1) {
    if (cmd[0] == 'p') {
      int mode, q_rows;
      long len;
      if (scanf("%d %d %ld", &mode, &q_rows, &len) != 3) return 2;
      Params p;
      memset(&p, 0, sizeof(p));
      p.q_rows = q_rows;
      plan_launch(&h, mode, len, p);
      printf("%d %d\n", p.splits, (int)p.pdl_early);
    } else if (cmd[0] == 'c') {
      long rows;
      if (scanf("%ld", &rows) != 1) return 2;
      printf("%d\n", (int)cross_by_token(&h, rows));
    } else if (cmd[0] == 't') {
      long rows, groups, keys;
      if (scanf("%ld %ld %ld", &rows, &groups, &keys) != 3) return 2;
      printf("%d\n", choose_tile_tokens(&h, rows, groups, keys > 0 ? keys : expected_tokens(&h)));
    } else {
      return 2;
    }
  }
  return 0;
}
