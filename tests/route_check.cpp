// Asks csrc/plan.h for the plan of a routing call: lines of tokens, experts and SMs; prints warps,
// blocks, tokens a block and whether one block orders the slots.
#include <cstdio>

#include "plan.h"

int main() {
  int tokens, experts, sms;
  while (std::scanf("%d %d %d", &tokens, &experts, &sms) == 3) {
    const g3::plan::RoutePlan p = g3::plan::route_plan(tokens, experts, sms);
    std::printf("%d %d %d %d\n", p.warps, p.blocks, p.chunk, p.few ? 1 : 0);
  }
  return 0;
}
