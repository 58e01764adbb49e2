// Tile / launch planner (pure host C++).
#include "plan.hpp"

#include <cstdlib>

namespace fp8bq {

// FP8BQ_GEMM_TILE=<0..4> forces a tile shape (a TileShape value; tuning aid; the grouped and the MXFP4 products have the
// shapes 0, 3 and 4 only and ignore the others); read once.
static int forced_shape() {
  static const int v = [] {
    const char* e = std::getenv("FP8BQ_GEMM_TILE");
    const int x = e ? std::atoi(e) : -1;
    return (x >= 0 && x <= 4) ? x : -1;
  }();
  return v;
}

static bool forced_planned_shape() {
  return forced_shape() == k128x128 || forced_shape() == k256x256 || forced_shape() == k64x64;
}

static int64_t cdiv(int64_t a, int64_t b) { return a / b + (a % b != 0 ? 1 : 0); }  // a >= 0, b > 0

// Time of one contraction block for one round of resident work units, in microseconds, measured
// on MI355X: two 128x128 workgroups per CU take ~1.2 us per block, one 256x256 workgroup ~2.05 us
// (4x the work for 1.7x the time: half the operand traffic per flop), four 64x64 workgroups ~0.94 us
// (half the work of two 128x128 ones for 0.8 of the time: that tile pays off only where the larger
// ones leave compute units idle, i.e. few output rows).
static double block_us(int shape) { return shape == k256x256 ? 2.05 : shape == k64x64 ? 0.94 : 1.2; }

// Cost model in microseconds: rounds of resident units x blocks per unit x block time, plus, for a
// split, a pass that writes and re-reads split x rows x cols FP32 partials and writes the output
// (~5 TB/s effective) and costs a fixed ~6 us as a launch of its own (measured: a 512-token fprop
// split in two took 18.9 us where 1024 tokens unsplit took 15.8).  Splitting pays off only when
// the tiles alone leave workgroup slots idle.
// A last round that fills only a fraction f of the slots runs faster than a full one (less
// contention for memory and power): it is charged (1 + f) / 2 of a round, as measured on MI355X
// (a half-full last round of 256x256 tiles took ~0.74 of a full one).
static double split_cost(int64_t rows, int64_t cols, int64_t nkb, int64_t slots, int shape, int s) {
  const int64_t tiles = cdiv(rows, tile_rows(shape)) * cdiv(cols, tile_cols(shape));
  const int64_t units = tiles * s;
  const int64_t full = units / slots;
  const double frac = (double)(units - full * slots) / (double)slots;
  const double rounds = (double)full + (frac > 0.0 ? 0.5 * (1.0 + frac) : 0.0);
  const double gemm_us = rounds * ((double)nkb / s) * block_us(shape);
  const double red_us = s > 1 ? 6.0 + (8.0 * s + 4.0) * (double)rows * (double)cols / 5.0e6 : 0.0;
  return gemm_us + red_us;
}

static int best_split(int64_t rows, int64_t cols, int64_t nkb, int64_t slots, int shape, double* cost) {
  int best = 1;
  double best_us = 0.0;
  for (int s = 1; s <= kMaxSplit; ++s) {
    if (s > 1 && nkb / s < 4) break;  // keep at least 4 blocks per unit
    const double us = split_cost(rows, cols, nkb, slots, shape, s);
    if (s == 1 || us < best_us * 0.97) {
      best = s;
      best_us = us;
    }
  }
  if (cost) *cost = best_us;
  return best;
}

GemmPlan plan_gemm(int op, int64_t M, int64_t N, int64_t K, int cu_count) {
  GemmPlan p;
  // Output shape and contraction length in the kernel's TN frame.
  int64_t rows, cols, contraction;
  if (op == kOpFprop || op == kOpTensor) {
    rows = M; cols = N; contraction = K;
  } else if (op == kOpDgrad || op == kOpDgradWt) {
    rows = M; cols = K; contraction = N;
  } else {
    rows = N; cols = K; contraction = M;
  }
  const int64_t cus = cu_count > 0 ? cu_count : 256;
  const int64_t nkb = contraction / 128;
  // one launch addresses its work units with 32 bits: at most 2^31 - 1 units of any tile shape and
  // split; sizes beyond that (far past any device memory) get an empty plan that the caller refuses
  const int64_t kMaxTiles128 = ((int64_t)1 << 28) - 1;
  const int64_t t128m = rows > 0 ? cdiv(rows, 128) : 0, t128n = cols > 0 ? cdiv(cols, 128) : 0;
  if (t128m > kMaxTiles128 || t128n > kMaxTiles128 || (t128n > 0 && t128m > kMaxTiles128 / t128n) ||
      nkb > ((int64_t)1 << 31) - 1 ||
      (op == kOpDgrad && (double)N * (double)K >= 4.611686018427388e18)) {
    p.fits = false;
    return p;
  }
  const bool work = rows > 0 && cols > 0 && nkb > 0;
  if (forced_shape() >= 0) {
    p.shape = forced_shape();
  } else if (work) {
    // the fastest tile shape under the cost model (ties go to the larger tile)
    double c64 = 0.0, c128 = 0.0, c256 = 0.0;
    best_split(rows, cols, nkb, cus * blocks_per_cu(k64x64), k64x64, &c64);
    best_split(rows, cols, nkb, cus * blocks_per_cu(k128x128), k128x128, &c128);
    best_split(rows, cols, nkb, cus * blocks_per_cu(k256x256), k256x256, &c256);
    p.shape = c256 <= c128 ? k256x256 : k128x128;
    if (c64 < (p.shape == k256x256 ? c256 : c128)) p.shape = k64x64;
  } else {
    p.shape = k128x128;
  }
  p.tile_m = tile_rows(p.shape);
  p.tile_n = tile_cols(p.shape);
  const int64_t slots = cus * blocks_per_cu(p.shape);
  p.tiles_m = cdiv(rows, p.tile_m);
  p.tiles_n = cdiv(cols, p.tile_n);
  p.split_k = work ? best_split(rows, cols, nkb, slots, p.shape, nullptr) : 1;
  // (a split is only chosen for few tiles; this keeps the unit count in 31 bits whatever the tile)
  if (p.split_k > 1 && p.tiles_m * p.tiles_n > (((int64_t)1 << 31) - 1) / p.split_k) p.split_k = 1;
  p.units = p.tiles_m * p.tiles_n * p.split_k;
  // persistent grid: one workgroup per slot (a multiple of 8, so each workgroup stays on one XCD's
  // range of tiles), or one per unit when there are fewer units
  int64_t g = slots >= 8 ? slots - slots % 8 : slots;  // (a device with fewer than 8 CUs: all of them)
  p.grid = p.units < g ? p.units : g;
  p.ws_gemm = p.split_k > 1 ? (size_t)p.split_k * (size_t)rows * (size_t)cols * 4 : 0;
  p.ws_transpose = (op == kOpDgrad) ? (size_t)N * (size_t)K : 0;
  // round the transpose buffer up so the partial sums that follow it stay 256-byte aligned
  p.ws_transpose = (p.ws_transpose + 255) & ~(size_t)255;
  return p;
}

// Stored past the caches, an output neither pushes what is in them out nor has to be written back from the L2 when the
// kernel ends; kept, it is there for whatever reads it next, and the caches spread its lines over the memory channels:
// where rows lie a multiple of 8 KB apart, the rows of a tile share a few channels, and stores past the caches wait for
// those.  us of one product after the other, and in turn with the quantizer of three inputs, each kept / past:
//   BF16 rows of a multiple of 8 KB (MXFP4: 16 KB), output and operands within the 256 MB cache: kept
//     8192 x 8192 x 2048 (134 MB)     124 / 133    137 / 143     (rows 512 bytes longer 124 / 123, 137 / 136)
//     8192 x 4096 x 2048 (67 MB)      63 / 68      74 / 79       16384 x 4096 x 2048 (134 MB)  123 / 126   149 / 144
//     wgrad 2048 x 8192 x 8192        136 / 146    152 / 156     MXFP4 8192 x 8192 x 2048      74 / 84     85 / 92
//   the same with less output (48 MB): past
//     wgrad 2048 x 4096 x 4096        38 / 37      47 / 46       MXFP4 2048 x 8192 x 2048      22 / 22     29 / 29
//   or more than the cache: past
//     16384 x 8192 x 2048 (268 MB)    248 / 247    295 / 268     (12288 x 8192 x 2048, 201 MB    180 / 187   207 / 203)
//   other BF16 rows: past
//     16384 x 2048 x 2048 (67 MB)     65 / 65      87 / 82       32768 x 2048 x 2048 (134 MB)  122 / 124   173 / 167
//     MXFP4 16384 x 3328 x 2048       70 / 69      89 / 85       16384 x 11264 x 2048 (369 MB) 350 / 308
//     (a decoder block's step, six of whose outputs have 67 or 84 MB, 2562 / 2529)
//   MXFP4 rows of 8 KB: past (16384 x 4096 x 2048 72 / 80 and 93 / 97, but through the linear layer 104 / 96)
//   grouped weight gradients, whose rows' tiles are dealt out otherwise: past whatever the rows
//     8 experts of 2048 x 4096        93 / 85      125 / 107     8 experts of 1024 x 8192      46 / 42     57 / 54
//   below 6 MB: kept (512 x 2048 x 2048 with the quantizer that reads it 12.6 / 13.4; 4 MB 15.4 / 15.8; 8 MB 21.4 / 21.3)
// FP32, alone and with a copy to BF16 that reads it: 17 MB 13.2 / 12.4 and 20.9 / 20.1, 67 MB 28.9 / 28.5 and 44.1 / 43.8:
// past; 268 MB 99 / 109 and 183 / 187, 279 / 279 and 351 / 367: kept; 369 MB 748 / 728 and 848 / 827, 738 MB 297 / 241
// and 507 / 466: past.  Added to the output, whose lines the addition has just read: 268 MB 182 / 183, 1476 MB
// 818 / 827: kept.
bool stores_past_caches(int out_t, double out, double operands, bool crowded) {
  if (out_t == 2 || out < 6e6) return false;
  if (out_t == 1) return out < 100e6 || out > 320e6;
  return !crowded || out < 48e6 || out + operands > 215e6;
}

// Blocks of 128 tokens that the longest expert has to be able to have before the grouped wgrad may split it.  The pass that
// adds up the chunks costs 3 us, also where the counts then split nothing (8 experts, 30000 tokens, 512 x 512, even:
// 30 and 33 us).  Uneven experts gain more (us, whole and split; 32 experts of 2048 x 1408, 32768 tokens): 25% (62%) of
// the tokens on one of the 32 experts 198 / 166 (313 / 169), 62% on one of the 8 experts 105 / 32, the same at 8000
// tokens on 4 experts of 1024 x 1024 35 / 32; at 4096 tokens nothing.
constexpr int64_t kMinSplitBlocks = 48;

// Splitting of the grouped wgrad's long experts with tiles of shape s: up to two sets of partial sums for every
// expert's worth of tiles that the workgroups hold at once, none where one expert's tiles fill them or
// where its contraction cannot be long.  A set is written and read back at about 5 TB/s.
static GroupSplit group_split(bool may, int64_t E, int64_t padded, int64_t N, int64_t K, int64_t slots, int s) {
  const double tiles = (double)cdiv(N, tile_rows(s)) * (double)cdiv(K, tile_cols(s));
  const int64_t longest = (padded - 127 * E) / 128 + 1;  // (padded holds all tokens and up to 127 rows an expert)
  GroupSplit g = {0, (float)tiles, (float)slots, (float)blocks_per_cu(s),
                  (float)(8.0 * (double)N * (double)K / 5.0e6 / block_us(s)), (float)(3.0 / block_us(s))};
  if (!may || longest <= kMinSplitBlocks || tiles >= (double)slots) return g;
  const double sets = 2.0 * (double)slots / tiles + 1.0;
  g.sets = sets < (double)kMaxSets ? (int)sets : kMaxSets;
  return g;
}

GemmPlan plan_grouped(int op, int64_t E, int64_t T, int64_t N, int64_t K, int cu_count, bool may_split) {
  GemmPlan p;
  const int64_t cus = cu_count > 0 ? cu_count : 256;
  const int64_t used = T < E ? (T > 0 ? T : 1) : E;
  const int64_t share = cdiv(T, used);
  const int64_t cols = op == kOpFprop ? N : K;
  const int64_t nkb = (op == kOpFprop ? K : N) / 128;
  const int shapes[3] = {k256x256, k128x128, k64x64};
  double best = 0.0;
  for (int i = 0; i < 3; ++i) {
    const int s = shapes[i];
    const double slots = (double)(cus * blocks_per_cu(s));
    double us;
    if (op == kOpWgrad) {
      // what the kernel will find, if the shares are equal
      const GroupSplit g = group_split(may_split, E, T, N, K, (int64_t)slots, s);
      us = 3.0e38;
      for (int l = g.sets > 0 ? 0 : 63; l < 64; ++l) {
        const int n = (int)cdiv(share, 128);
        const float len = chunk_candidate(l);
        if ((float)n / len > (float)kMaxSets) continue;
        ChunkSums even(n, len);
        even.add(n, len, 1.0f / len, (int)used);
        const double t = (double)chunk_time(even, g) * block_us(s);
        us = t < us ? t : us;
      }
    } else {
      // ragged shares end half a tile short on average (a quarter with 256 rows, whose last tile may be a short one)
      double tiles_m = (double)share / tile_rows(s) + (s == k256x256 ? 0.25 : 0.5);
      tiles_m = tiles_m < 1.0 ? 1.0 : tiles_m;
      const double units = (double)used * tiles_m * (double)cdiv(cols, tile_cols(s));
      const double full = (double)(int64_t)(units / slots);
      const double frac = units / slots - full;
      us = (full + (frac > 0.0 ? 0.5 * (1.0 + frac) : 0.0)) * (double)nkb * block_us(s);
    }
    if (i == 0 || us < best) {
      best = us;
      p.shape = s;
    }
  }
  if (forced_planned_shape()) p.shape = forced_shape();
  p.tile_m = tile_rows(p.shape);
  p.tile_n = tile_cols(p.shape);
  p.tiles_n = cdiv(cols, p.tile_n);
  p.tiles_m = op == kOpWgrad ? cdiv(N, p.tile_m) : T / p.tile_m + used;  // upper bound over the experts
  const int64_t slots = cus * blocks_per_cu(p.shape);
  const int64_t g = slots >= 8 ? slots - slots % 8 : slots;
  if (op == kOpWgrad) {
    p.group_split = group_split(may_split, E, T, N, K, g, p.shape);
    const size_t sets = (size_t)p.group_split.sets;
    p.ws_gemm = sets > 0 ? kSplitListBytes + sets * (size_t)N * (size_t)K * 4 : 0;
  }
  const double units = (double)p.tiles_m * (double)p.tiles_n * (op == kOpWgrad ? (double)(E + p.group_split.sets) : 1.0);
  if (units >= 2147483647.0) {
    p.fits = false;
    return p;
  }
  p.units = (int64_t)units;
  p.grid = p.units < g ? p.units : g;
  return p;
}

// Time of one 256-long stage for one full round of resident MXFP4 work units, in microseconds, measured on
// MI355X (8192 x 8192 x 8192 with each tile: 275, 340 and 500 us).
static double mx_stage_us(int shape) { return shape == k256x256 ? 2.1 : shape == k64x64 ? 0.98 : 1.33; }

MxPlan plan_mx(bool linear, int64_t E, int64_t M, int64_t N, int64_t K, int cu_count) {
  MxPlan p;
  const int64_t cus = cu_count > 0 ? cu_count : 256;
  const int64_t used = E == 0 ? 1 : (M < E ? (M > 0 ? M : 1) : E);
  p.rows = cdiv(M, used);
  // Few rows on few column tiles: the kernel without LDS staging.  From codes (us, one row and K = 2048; the
  // tiled kernel second): N = 4096 3.6 / 6.5, 11264 4.7 / 6.5, 22528 6.4 / 7.1, 45056 11.5 / 10.1.
  const int64_t tiles = used * cdiv(N, 16);
  p.skinny = M <= 16 && tiles <= 1536;
  if (p.skinny) {
    // Every tile quantizes its rows itself while that costs less than a quantizer launch (us, fused and not):
    // 16 rows, 11264 x 2048 9.4 / 10.5, 16384 x 2048 11.6 / 10.5; 8 rows, 16384 x 2048 9.1 / 9.9, 22528 x 2048
    // 12.2 / 11.5; 16 rows, 2048 x 11264 15.7 / 12.8; 8 rows, 2048 x 11264 11.4 / 12.4.
    const int64_t steps = tiles * cdiv(K, 128);
    p.fused = linear && steps <= 300000 / (p.rows + 8) && p.rows * K <= 131072;
    p.split_k = 8;
    while (p.split_k > 1 && p.split_k > cdiv(K, 256)) p.split_k /= 2;
    const int64_t groups = E == 0 ? 1 : used;
    const int64_t units = groups * cdiv(N, 8 / p.split_k * 16);
    p.grid = units < 16 * cus ? units : 16 * cus;
    return p;
  }
  const int64_t nkb = cdiv(K, 256);
  const int shapes[3] = {k256x256, k128x128, k64x64};
  double best = 0.0;
  for (int i = 0; i < 3; ++i) {
    const int s = shapes[i];
    const int64_t slots = cus * blocks_per_cu(s);
    const double tiles = (double)used * (double)cdiv(p.rows, tile_rows(s)) * (double)cdiv(N, tile_cols(s));
    for (int split = 1; split <= (E == 0 ? kMaxSplit : 1); ++split) {
      if (split > 1 && nkb / split < 4) break;
      const double rounds = tiles * split / (double)slots;
      const double full = (double)(int64_t)rounds, frac = rounds - full;
      double us = (full + (frac > 0.0 ? 0.5 * (1.0 + frac) : 0.0)) * ((double)nkb / split + 1.0) * mx_stage_us(s);
      if (split > 1) us += 6.0 + (8.0 * split + 4.0) * (double)M * (double)N / 5.0e6;
      if ((i == 0 && split == 1) || us < best * (split > 1 ? 0.97 : 1.0)) {
        best = us;
        p.shape = s;
        p.split_k = split;
      }
    }
  }
  if (forced_planned_shape()) p.shape = forced_shape();
  p.tiles_n = cdiv(N, tile_cols(p.shape));
  p.tiles_m = E == 0 ? cdiv(M, tile_rows(p.shape)) : M / tile_rows(p.shape) + used;
  const int64_t units = p.tiles_m * p.tiles_n * p.split_k;  // (sizes are limited by the validation)
  const int64_t slots = cus * blocks_per_cu(p.shape);
  const int64_t g = slots >= 8 ? slots - slots % 8 : slots;
  p.grid = units < g ? units : g;
  p.ws = p.split_k > 1 ? (size_t)p.split_k * (size_t)M * (size_t)(cdiv(N, 4) * 4) * 4 : 0;
  return p;
}

}  // namespace fp8bq
