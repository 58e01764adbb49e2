// Plan of an orthogonalization (pure host C++).
#include "ortho_plan.hpp"

#include "plan.hpp"

namespace fp8bq {

static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
static size_t up256(double n) { return ((size_t)n + 255) & ~(size_t)255; }

// Time of one 128-byte stage for a full round of resident work units, us (as the MXFP4 product's, whose loop it is).
static double stage_us(int shape) {
  return shape == k256x256 ? 2.1 : shape == k256x192 ? 1.65 : shape == k64x64 ? 0.98 : 1.33;
}
constexpr int kMaxOrthoSplit = 16, kOrthoTerms = 3;

// rows x cols outputs (triangle: a symmetric rows x rows result) of nkb stages for each term, for each of the batch.
static OrthoProduct plan_product(int64_t rows, int64_t cols, int64_t nkb, int64_t batch, bool triangle, int64_t cus) {
  OrthoProduct best;
  double best_us = 0.0;
  const int shapes[4] = {k256x256, k128x128, k64x64, k256x192};
  for (int i = 0; i < (triangle ? 3 : 4); ++i) {  // (a symmetric result has square tiles)
    const int s = shapes[i];
    OrthoProduct p;
    p.shape = s;
    p.tiles_m = cdiv(rows, tile_rows(s));
    p.tiles_n = cdiv(cols, tile_cols(s));
    p.tiles = triangle ? p.tiles_m * (p.tiles_m + 1) / 2 : p.tiles_m * p.tiles_n;
    const int64_t slots = cus * blocks_per_cu(s);
    for (int split = 1; split <= (triangle ? kMaxOrthoSplit : 1); ++split) {
      if (split > 1 && nkb / split < 4) break;  // (also of the one term that the first step may have)
      const double units = (double)p.tiles * (double)split * (double)batch;
      const double rounds = units / (double)slots, full = (double)(int64_t)rounds, frac = rounds - full;
      double us = (full + (frac > 0.0 ? 0.5 * (1.0 + frac) : 0.0)) * ((double)(kOrthoTerms * nkb) / split + 1.0) * stage_us(s);
      if (split > 1) us += 5.0 + 8.0 * units * (double)(tile_rows(s) * tile_cols(s)) / 5.0e6;
      if ((i == 0 && split == 1) || us < best_us * (split > 1 ? 0.97 : 1.0)) {
        best_us = us;
        best = p;
        best.split = split;
      }
    }
  }
  const int64_t slots = cus * blocks_per_cu(best.shape);
  const int64_t g = slots >= 8 ? slots - slots % 8 : slots;
  const int64_t units = best.tiles * best.split * batch;
  best.grid = units < g ? units : g;
  best.deep = best.shape == k64x64 && units <= kDeepPerCu * cus;
  return best;
}

OrthoPlan plan_ortho(int64_t batch, int64_t R, int64_t C, int cu_count, bool* fits) {
  OrthoPlan p{};
  const int64_t cus = cu_count > 0 ? cu_count : 256;
  p.batch = batch;
  p.R = R;
  p.C = C;
  p.m = R < C ? R : C;
  p.n = R < C ? C : R;
  p.mp = cdiv(p.m, 64) * 64;
  p.np = cdiv(p.n, 64) * 64;
  // buffers and partial sums stay below 2^46 bytes, a launch's work units below 2^31
  const double elements = (double)batch * (double)p.np * (double)p.mp;
  *fits = elements * 24.0 < 7.0e13 && elements / 4096.0 * kMaxOrthoSplit * 8.0 < 2147483647.0;
  if (!*fits) return p;
  p.gram = plan_product(p.m, p.m, p.np / 64, batch, true, cus);
  p.poly = plan_product(p.m, p.m, p.mp / 64, batch, true, cus);
  p.update = plan_product(p.n, p.m, p.mp / 64, batch, false, cus);
  const int64_t blocks = cdiv(R * C, 16384), most = cdiv(2048, batch);
  p.norm_blocks = (int)(blocks < most ? blocks : most);
  size_t at = 0;
  auto take = [&](double bytes) {
    const size_t here = at;
    at += up256(bytes);
    return here;
  };
  const double b = (double)batch, m = (double)p.m, n = (double)p.n, mp = (double)p.mp, np = (double)p.np;
  p.at_norms = take(b * p.norm_blocks * 8.0);
  p.at_factor = take(b * kMaxOrthoSteps * 8.0);
  p.at_x = take(b * m * np * 2.0);
  p.at_xt[0] = take(b * n * mp * 4.0);
  p.at_xt[1] = take(b * n * mp * 4.0);
  p.at_low = take(b * m * np * 2.0);
  p.at_gram = take(b * m * mp * 4.0);
  p.at_poly = take(b * m * mp * 4.0);
  auto parts = [&](const OrthoProduct& q) {
    return q.split > 1 ? (double)(q.tiles * q.split) * b * (double)(tile_rows(q.shape) * tile_cols(q.shape)) * 4.0 : 0.0;
  };
  const double a = parts(p.gram), c = parts(p.poly);
  p.at_parts = take(a > c ? a : c);
  p.ws = at;
  return p;
}

}  // namespace fp8bq
