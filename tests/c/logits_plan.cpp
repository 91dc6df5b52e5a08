// The launch shapes of the adjusted logits (gated_delta_rule_59_amd/csrc/kda_logits_plan.h), compiled with g++
// and run on the CPU: reads lines of N R V, prints each one's steps, blocks and splits.
#include <cstdio>

#include "kda_logits_plan.h"

int main() {
  int N, R, V;
  while (std::scanf("%d %d %d", &N, &R, &V) == 3) {
    const int steps = kda::logits_steps(N, R, V);
    const long long blocks = kda::logits_blocks(V, steps);
    std::printf("%d %lld %d\n", steps, blocks, kda::logits_splits(N, R, blocks));
  }
  return 0;
}
