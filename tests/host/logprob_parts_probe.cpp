// Host-side probe of how the log probabilities' rows are cut. Reads lines of
//   <rows> <vocab> <bits of a logit>
// and prints the parts of a row where all rows start at multiples of 16 bytes,
// those where they do not, and the most parts that the join reads. Runs on the
// CPU only; calls no HIP runtime function.
#include <cstdio>

#include "logprob.hip"

using namespace qlinear;

int main() {
  int rows, vocab, bits;
  while (scanf("%d %d %d", &rows, &vocab, &bits) == 3)
    printf("%d %d %d\n", make_plan(rows, vocab, bits == 32, true).parts, make_plan(rows, vocab, bits == 32, false).parts,
           kJoinTurns * kThreads);
  return 0;
}
