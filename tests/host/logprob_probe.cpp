// Host-side probe of the log probabilities' launch plan. Reads lines of
//   <rows> <vocab> <bits of a logit> <top>
// and prints the workspace that such a call takes, the larger of that for rows
// that start at multiples of 16 bytes and for others, and what a query of these
// sizes answers. Runs on the CPU only; calls no HIP runtime function.
#include <cstdio>

#include "logprob.hip"

using namespace qlinear;

int main() {
  LogprobArgs a = {};
  int bits;
  while (scanf("%d %d %d %d", &a.rows, &a.vocab, &bits, &a.top) == 4) {
    a.f32 = bits == 32;
    a.logits = nullptr;
    a.stride = 1 << 20;
    const size_t whole = logprob_workspace_need(a);
    a.logits = (const void*)4;
    const size_t other = logprob_workspace_need(a);
    printf("%zu %zu\n", whole > other ? whole : other, logprob_workspace_bytes(a));
  }
  return 0;
}
