// What the planner chooses for the sizes on the standard input, one product a line (256 compute units):
//   grouped <op: 0 fprop, 1 dgrad, 2 wgrad> <experts> <tokens, padded for wgrad> <N> <K> <with a workspace: 0, 1>
//   mx <quantizes its input: 0, 1> <experts, 0 for the dense product> <M> <N> <K>
//   stores <output: 0 BF16, 1 FP32, 2 FP32 added to it> <bytes of the output, of the operands> <rows crowded: 0, 1>
// Prints "<rows> <columns of a tile> <sets of partial sums>" and "<rows> <columns> <split of the contraction>" (rows 0
// where no tiles are staged); and 1 where the output's full tiles are stored past the caches, else 0.
#include <cstdio>
#include <iostream>
#include <string>

#include "plan.hpp"

using namespace fp8bq;

int main() {
  std::string what;
  while (std::cin >> what) {
    if (what == "grouped") {
      int op, split;
      int64_t E, T, N, K;
      if (!(std::cin >> op >> E >> T >> N >> K >> split)) return 1;
      const GemmPlan p = plan_grouped(op, E, T, N, K, 256, split != 0);
      std::printf("%d %d %d\n", p.tile_m, p.tile_n, p.group_split.sets);
    } else if (what == "stores") {
      int out_t;
      int crowded;
      double out, operands;
      if (!(std::cin >> out_t >> out >> operands >> crowded)) return 1;
      std::printf("%d\n", stores_past_caches(out_t, out, operands, crowded != 0) ? 1 : 0);
    } else {
      int linear;
      int64_t E, M, N, K;
      if (what != "mx" || !(std::cin >> linear >> E >> M >> N >> K)) return 1;
      const MxPlan p = plan_mx(linear != 0, E, M, N, K, 256);
      std::printf("%d %d %d\n", p.skinny ? 0 : tile_rows(p.shape), p.skinny ? 0 : tile_cols(p.shape), p.split_k);
    }
  }
  return 0;
}
