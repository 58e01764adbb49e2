// What the planner chooses for 8-bit products, one a line on the standard input (256 compute units):
//   <quantizes its input: 0, 1> <experts, 0 for the dense product> <M> <N> <K>
// Prints "<rows> <columns of a tile> <split of the contraction> <three stages: 0, 1>", rows 0 where no tiles are staged.
#include <cstdio>
#include <iostream>

#include "plan.hpp"

using namespace fp8bq;

int main() {
  int linear;
  int64_t E, M, N, K;
  while (std::cin >> linear >> E >> M >> N >> K) {
    const MxPlan p = plan_int8(linear != 0, E, M, N, K, 256);
    std::printf("%d %d %d %d\n", p.skinny ? 0 : tile_rows(p.shape), p.skinny ? 0 : tile_cols(p.shape), p.split_k, p.deep ? 1 : 0);
  }
  return 0;
}
