// Host-side probe of what a paged attention call takes of its workspace. Reads
// lines of
//   <head_dim> <bits> <kv_heads> <tokens> <q_heads> <batch> <max_q_len> <max_kv_len> <window>
// and prints the bytes that such a call needs and the bytes that the workspace
// query answers. Runs on the CPU only; launches nothing.
#include <cstdio>

#include "paged_attention.hip"

namespace qlinear {
#define NO_LAUNCH(name)                                                                                     \
  hipError_t name(const qlinear_kv_cache&, const AttentionArgs&, const attn::Plan&, const attn::Partials&, \
                  hipStream_t) {                                                                            \
    return hipSuccess;                                                                                      \
  }
NO_LAUNCH(launch_attention_few_64)
NO_LAUNCH(launch_attention_few_128)
NO_LAUNCH(launch_attention_few_256)
NO_LAUNCH(launch_attention_chunk_64)
NO_LAUNCH(launch_attention_chunk_128)
NO_LAUNCH(launch_attention_chunk_256)
}  // namespace qlinear

int main() {
  qlinear_kv_cache c = {};
  qlinear::AttentionArgs a = {};
  while (scanf("%d %d %d %d %d %d %d %d %d", &c.head_dim, &c.bits, &c.kv_heads, &a.tokens, &a.q_heads, &a.batch,
               &a.max_q_len, &a.max_kv_len, &a.window) == 9)
    printf("%zu %zu\n", qlinear::paged_attention_workspace_need(c, a), qlinear::paged_attention_workspace_bytes(c, a));
  return 0;
}
