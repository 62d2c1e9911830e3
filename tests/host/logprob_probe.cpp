// Host-side probe of the log probabilities' launch plan. Reads lines of
//   <rows> <vocab> <bits of a logit> <top>
// and prints the workspace that such a call takes, and what a query of these
// sizes answers. Runs on the CPU only; calls no HIP runtime function.
#include <cstdio>

#include "logprob.hip"

using namespace qlinear;

int main() {
  LogprobArgs a = {};
  int bits;
  while (scanf("%d %d %d %d", &a.rows, &a.vocab, &bits, &a.top) == 4) {
    a.f32 = bits == 32;
    printf("%zu %zu\n", logprob_workspace_need(a), logprob_workspace_bytes(a));
  }
  return 0;
}
