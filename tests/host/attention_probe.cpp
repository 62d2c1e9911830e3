// Host-side probe of what the attention kernels' workgroups work out about
// their rows and steps. Reads lines of
//   rows <new tokens> <length> <group> <window> <row0> <tile rows>
// and prints the positions and first tokens seen of that row tile, and the
// steps that the few-row kernel counts for the sequence; and lines of
//   length <length> <table width> <page size>
// and prints the length that the kernels take; and lines of
//   start <first row> <row after the last> <tokens>
// and prints the first row and the number of rows that they take. Runs on the CPU only; calls no
// HIP runtime function.
#include <cstdio>
#include <cstring>

#include "attention.hpp"

using namespace qlinear;

int main() {
  char what[16];
  while (scanf("%15s", what) == 1) {
    if (!strcmp(what, "rows")) {
      attn::Work w = {};
      AttentionArgs a = {};
      attn::Plan plan = {};
      int group, row0, tile_rows;
      if (scanf("%d %d %d %d %d %d", &w.n, &w.len, &group, &a.window, &row0, &tile_rows) != 6) return 1;
      plan.rows = 16;
      plan.max_rows = INT32_MAX;
      const attn::Item it = attn::few_item(a, plan, group, w);
      attn::row_tile(a, group, row0, tile_rows, w);
      printf("%d %d %d %d %d %d\n", w.p_min, w.p_max, w.lo_min, w.lo_max, it.first_step, it.steps);
    } else if (!strcmp(what, "length")) {
      int len, width, page;
      if (scanf("%d %d %d", &len, &width, &page) != 3) return 1;
      printf("%d\n", attn::bounded_length(len, width, page));
    } else if (!strcmp(what, "start")) {
      attn::Work w = {};
      int q0, q1, tokens;
      if (scanf("%d %d %d", &q0, &q1, &tokens) != 3) return 1;
      attn::bounded_rows(q0, q1, tokens, w);
      printf("%d %d\n", w.q0, w.n);
    } else {
      return 1;
    }
  }
  return 0;
}
