// Host-side probe of what attention calls with sinks or shared prefixes take of
// their workspace. Reads lines of
//   <head_dim> <bits> <kv_heads> <tokens> <q_heads> <batch> <max_q_len> <max_kv_len> <window> <sinks>
//   <groups> <max_shared_len>
// (groups 0: sinks) and prints the bytes that such a call needs and the bytes that
// the workspace query answers; and after the word `rows`, lines of
//   rows <tokens> <sequences> <groups> <q_start, sequences + 1 numbers>
//   <shared_start, groups + 1 numbers> <shared_len, groups numbers> <kv_len, sequences numbers>
// and prints first row, rows, length, first own token, row of the block table and
// kind of the groups and then of the sequences. Runs on the CPU only; launches nothing.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "attention_views.hip"

namespace qlinear {
QLINEAR_VIEW_LAUNCHER(launch_view_few_64) { return hipSuccess; }
QLINEAR_VIEW_LAUNCHER(launch_view_few_128) { return hipSuccess; }
QLINEAR_VIEW_LAUNCHER(launch_view_few_256) { return hipSuccess; }
QLINEAR_VIEW_LAUNCHER(launch_view_chunk_64) { return hipSuccess; }
QLINEAR_VIEW_LAUNCHER(launch_view_chunk_128) { return hipSuccess; }
QLINEAR_VIEW_LAUNCHER(launch_view_chunk_256) { return hipSuccess; }
}  // namespace qlinear

using namespace qlinear;

static std::vector<int> numbers(int n) {
  std::vector<int> v(n);
  for (int& x : v)
    if (scanf("%d", &x) != 1) x = 0;
  return v;
}

int main() {
  char what[16];
  while (scanf("%15s", what) == 1) {
    qlinear_kv_cache c = {};
    ViewArgs a = {};
    if (!strcmp(what, "rows")) {
      int sequences;
      if (scanf("%d %d %d", &a.tokens, &sequences, &a.groups) != 3) return 1;
      const auto q_start = numbers(sequences + 1), start = numbers(a.groups + 1), len = numbers(a.groups),
                 kv = numbers(sequences);
      a.q_start = q_start.data();
      a.shared_start = start.data();
      a.shared_len = len.data();
      a.kv_len = kv.data();
      a.batch = a.groups + sequences;
      a.table_width = 1000;
      c.page_size = 16;
      for (int b = 0; b < a.batch; ++b) {
        attn::Work w = {};
        attn::sequence(a, c, b, w);
        printf("%d %d %d %d %d %d ", w.q0, w.n, w.len, w.low, w.row, (int)w.all);
      }
      printf("\n");
      continue;
    }
    c.head_dim = atoi(what);
    if (scanf("%d %d %d %d %d %d %d %d %d %d %d", &c.bits, &c.kv_heads, &a.tokens, &a.q_heads, &a.batch, &a.max_q_len,
              &a.max_kv_len, &a.window, &a.sinks, &a.groups, &a.max_shared_len) != 11)
      return 1;
    a.batch += a.groups;
    if (a.groups)
      printf("%zu %zu\n", shared_attention_workspace_need(c, a), shared_attention_workspace_bytes(c, a));
    else
      printf("%zu %zu\n", sinks_attention_workspace_need(c, a), sinks_attention_workspace_bytes(c, a));
  }
  return 0;
}
