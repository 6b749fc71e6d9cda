// Asks csrc/plan.h for the plan of block-scaled products: lines of rows, experts, N, blocks
// of K, two weights, SMs and forced tile; prints the row tile and the split of K.
#include <cstdio>

#include "plan.h"

int main() {
  long long rows;
  int experts, N, kblocks, two, sms, forced;
  while (std::scanf("%lld %d %d %d %d %d %d", &rows, &experts, &N, &kblocks, &two, &sms, &forced) == 7) {
    const g3::plan::BlocksChoice c = g3::plan::blocks_choice(rows, experts, N, kblocks, two != 0, sms, forced);
    std::printf("%d %d\n", c.nt, c.split);
  }
  return 0;
}
