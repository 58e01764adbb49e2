// Tile / launch planner for the scaled FP8 GEMMs (pure host C++, no HIP calls).
//
// Given the product (fprop, dgrad, wgrad), its sizes and the device's compute-unit count, picks the
// split of the contraction across workgroups, the persistent grid, and the workspace it needs.
// Deterministic for equal inputs.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace fp8bq {

enum SbMode : int { kSbBlock128 = 0, kSbColumn = 1 };
// kOpDgradWt: dgrad on weight codes already transposed (W^T [K, N]): the dgrad kernel, no transpose.
// kOpTensor: Y[M, N] = sa sb A[M, K] B[N, K]^T with one scale per operand (per-tensor scaling): the
// fprop kernel with broadcast scales, planned as fprop.
enum Op : int { kOpFprop = 0, kOpDgrad = 1, kOpWgrad = 2, kOpDgradWt = 3, kOpTensor = 4 };

// Workgroup tile shapes (output rows x columns of one work unit):
//   k128x128: 4 waves of 64x64, two workgroups per CU;
//   k128x256 / k256x128: 8 waves of 64x64, one workgroup per CU (tuning shapes, never planned);
//   k256x256: 8 waves of 128x64, one workgroup per CU;
//   k64x64: 4 waves of 16x64, four workgroups per CU (few output rows: 4x the tiles of 128x128).
enum TileShape : int { k128x128 = 0, k128x256 = 1, k256x128 = 2, k256x256 = 3, k64x64 = 4 };
inline int tile_rows(int shape) {
  return shape == k64x64 ? 64 : (shape == k256x128 || shape == k256x256) ? 256 : 128;
}
inline int tile_cols(int shape) {
  return shape == k64x64 ? 64 : (shape == k128x256 || shape == k256x256) ? 256 : 128;
}
inline int blocks_per_cu(int shape) { return shape == k64x64 ? 4 : shape == k128x128 ? 2 : 1; }
constexpr int kMaxSplit = 8;

// Splitting of long experts in a product grouped by expert that contracts over the tokens (wgrad).  The counts are
// on the device, so the kernel chooses there how long a chunk of the contraction may be; the host gives it what
// it needs for that: sets of partial sums [N, K] that the workspace holds (0: no splitting), output tiles an
// expert, workgroups (in all and on a compute unit), and in units of one block's time what writing and adding up
// one set costs and what the pass that adds them costs besides.  The kernel leaves its choice in the workspace for
// the pass that adds the sets up: two kernels that computed it apart might round differently.
constexpr int kMaxSets = 64;
constexpr size_t kSplitListBytes = 256;  // in front of the sets: count and entries of the split experts (half the sets)
struct GroupSplit {
  int sets;
  float tiles, slots, per_cu, set_cost, sum_cost;
};
#if defined(__HIPCC__)
#define FP8BQ_HOST_DEVICE __host__ __device__
#else
#define FP8BQ_HOST_DEVICE
#endif
// Lengths of chunk to choose from, in blocks: 4 x 1.15^i, and one that splits nothing.
FP8BQ_HOST_DEVICE inline float chunk_candidate(int i) {
  return i == 63 ? 1e9f : 4.0f * __builtin_exp2f(0.2f * (float)i);
}
// Chunks of n > 0 blocks, none much longer than s = 1 / inv (n of them at most).
FP8BQ_HOST_DEVICE inline int chunks_of(int n, float s, float inv) {
  return (float)n <= s ? 1 : (int)__builtin_ceilf((float)n * inv);
}
// The chunks of all experts, by length against the longest: over a half, over a quarter, and the others.
struct ChunkSums {
  float top;  // the longest chunk
  int sets = 0;
  int units[3] = {0, 0, 0}, blocks[3] = {0, 0, 0};
  // longest: the most blocks of an expert
  FP8BQ_HOST_DEVICE ChunkSums(int longest, float s) : top((float)longest < s ? (float)longest : s) {}
  FP8BQ_HOST_DEVICE void add(int n, float s, float inv, int experts = 1) {
    if (n <= 0) return;
    const int c = chunks_of(n, s, inv);
    sets += c > 1 ? experts * c : 0;
    const float total = (float)c * top;  // the chunks' blocks if each were the longest
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const bool in = i == 0 ? 2.0f * (float)n > total : i == 1 ? 2.0f * (float)n <= total && 4.0f * (float)n > total
                                                                : 4.0f * (float)n <= total;
      units[i] += in ? experts * c : 0;
      blocks[i] += in ? experts * n : 0;
    }
  }
};
// Blocks of time of a product with those chunks, longest first on the workgroups in turn: everyone's share of the blocks
// (each chunk with a block's time for its first loads and its output), half a chunk for the last round, and what the
// longest chunk has more than the first round's average; at least the longest chunk; and the sets.  A block takes
// half the time where a compute unit has one workgroup instead of as many as it holds (128 x 128 tiles 0.69 and
// 1.2 us, 64 x 64 0.49 and 0.94).  Splitting has to be worth 3%.
FP8BQ_HOST_DEVICE inline float chunk_time(const ChunkSums& c, const GroupSplit& g) {
  if (c.sets > g.sets) return 3.0e38f;
  const int count = c.units[0] + c.units[1] + c.units[2], blocks = c.blocks[0] + c.blocks[1] + c.blocks[2];
  const float units = (float)count * g.tiles;
  float left = g.slots, first = 0.0f;  // the first round's workgroups and blocks
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const float u = (float)c.units[i] * g.tiles, take = u < left ? u : left;
    first += c.units[i] > 0 ? take * (float)c.blocks[i] / (float)c.units[i] : 0.0f;
    left -= take;
  }
  float t = (float)(blocks + count) * g.tiles / g.slots;
  if (units > g.slots) {
    const float over = c.top - first / g.slots;
    t += 0.5f * (float)blocks / (float)count + (over > 0.0f ? over : 0.0f);
  }
  const float on_cu = __builtin_ceilf(units * g.per_cu / g.slots);
  const float rate = g.per_cu > 1.0f && on_cu < g.per_cu ? 0.5f + 0.5f * (on_cu - 1.0f) / (g.per_cu - 1.0f) : 1.0f;
  const float longest = rate * (c.top + 1.0f);
  t = t > longest ? t : longest;
  return c.sets == 0 ? 0.97f * t : t + (float)c.sets * g.set_cost + g.sum_cost;
}

struct GemmPlan {
  int shape = k128x128;
  int tile_m = 128;
  int tile_n = 128;
  int split_k = 1;    // contraction split across work units (FP32 partials reduced afterwards)
  int64_t tiles_m = 0, tiles_n = 0;
  int64_t units = 0;  // tiles x split
  int64_t grid = 0;   // persistent workgroups launched
  size_t ws_gemm = 0;       // workspace for split partial sums
  size_t ws_transpose = 0;  // workspace for dgrad's transposed weight codes
  GroupSplit group_split = {};
  // false when the product is too large for one launch (more than 2^28 - 1 output tiles of
  // 128x128, or a dgrad transpose buffer past 2^62 bytes); the plan is then empty
  bool fits = true;
  size_t ws_total() const { return ws_transpose + ws_gemm; }
};

// M, N, K follow the C-ABI meaning for each op (fprop: Y[M,N] = X[M,K] W[N,K]^T; dgrad: dX[M,K] =
// dY[M,N] W[N,K]; wgrad: dW[N,K] = dY[M,N]^T X[M,K]).
GemmPlan plan_gemm(int op, int64_t M, int64_t N, int64_t K, int cu_count);

// Whether a product with that many bytes of output and of operands stores its full output tiles past the caches.  out_t:
// 0 BF16, 1 FP32, 2 FP32 added to the output; crowded: the output's rows lie a multiple of 8 KB (MXFP4: 16 KB) apart.
bool stores_past_caches(int out_t, double out, double operands, bool crowded);

// Plan of a product grouped by expert: tile shape and persistent grid.  op is kOpFprop, kOpDgrad or
// kOpWgrad; T tokens on E experts; N, K as in plan_gemm.  The tokens of each expert are known on the device
// only, so the shape is chosen for equal shares and the grid covers the most tiles any shares can give.
// Without may_split no expert's contraction is split (no workspace).
GemmPlan plan_grouped(int op, int64_t E, int64_t T, int64_t N, int64_t K, int cu_count, bool may_split = true);

// Rows that hold T tokens with every expert's padded to whole 128-token blocks, whatever their shares.
inline int64_t grouped_padded_rows(int64_t T, int64_t E) { return (T + 127 * (E < T ? E : T)) / 128 * 128; }

// Plan of an MXFP4 product (E == 0: dense; else M tokens grouped on E experts).  linear: A comes unquantized.
struct MxPlan {
  bool fused = false;  // A is quantized in the product's kernel (only with linear)
  bool skinny = true;  // few rows: the streaming kernel; else LDS tiles of the shape below
  int64_t rows = 0;    // rows one product is expected to have
  int shape = k128x128;
  int split_k = 1;     // skinny: waves of a workgroup that split the contraction; else as in GemmPlan
  int64_t tiles_m = 0, tiles_n = 0;
  int64_t grid = 0;
  size_t ws = 0;       // workspace of the product itself
};
MxPlan plan_mx(bool linear, int64_t E, int64_t M, int64_t N, int64_t K, int cu_count);

}  // namespace fp8bq
