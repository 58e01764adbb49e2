// Plan of an orthogonalization (ortho.hip): tile shapes, splits and the workspace's layout (pure host C++).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace fp8bq {

struct OrthoProduct {
  int shape = 0;
  int split = 1;
  bool deep = false;  // 64 x 64 tiles that are all on the card at once: a ring of three stages
  int64_t tiles_m = 0, tiles_n = 0, tiles = 0;  // tiles: of one matrix (those on and above the diagonal for A and A^2)
  int64_t grid = 0;
};

struct OrthoPlan {
  int64_t batch, R, C, m, n, mp, np;  // m, n: the shorter and the longer side; mp, np: padded to whole stages
  OrthoProduct gram, poly, update;
  int norm_blocks;                    // of a matrix
  // byte offsets in the workspace: factors of each matrix's steps; first halves of X and, at at_low, its second ones; X^T, A and the polynomial hold both
  size_t at_norms, at_factor, at_x, at_xt[2], at_low, at_gram, at_poly, at_parts;
  size_t ws;
};

// batch >= 1, 1 <= R, C <= kMaxOrthoSide, batch <= kMaxOrthoBatch; *fits false where the workspace or a launch's work
// units would pass what is addressable.
constexpr int64_t kMaxOrthoSide = (int64_t)1 << 20, kMaxOrthoBatch = 4096;
constexpr int kMaxOrthoSteps = 64;
OrthoPlan plan_ortho(int64_t batch, int64_t R, int64_t C, int cu_count, bool* fits);

}  // namespace fp8bq
