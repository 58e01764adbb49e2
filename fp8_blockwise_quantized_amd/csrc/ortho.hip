// Orthogonalization of an update by Newton-Schulz products, a batch of matrices [R, C] of one size.
//
// Mathematics.  With m = min(R, C), n = max(R, C) and X the m x n one of G and its transpose, X <- X / (|X|_F + eps), then
// in every step A = X X^T, X <- a X + (b A + c A^2) X: each singular value s becomes a s + b s^3 + c s^5, and the singular
// vectors stay.  Three products a step, A and A^2 symmetric: only their upper triangle of tiles is computed, and a tile
// is written twice.
//
// Rounding.  A step amplifies what it is given: an error of X in directions where X is small by a, one of A by up to b + 2 c A.
// With A and P held in 11 bits and products of 11-bit operands the result was off by 3 10^-4 (low rank) to 7 10^-3 of its norm
// (few rows, equal singular values), where its own rounding to BF16 is 1.7 10^-3; every one of these roundings alone is worth
// 2 10^-4 to 6 10^-3.  So X, A and P are each the sum of two 16-bit floats (22 bits), and a product of two such sums takes
// three of the four products (first halves; first by second; second by first), with FP32 accumulation: off by 5 10^-6 or less for
// random, low-rank and orthogonal matrices, as FP32 products are, at three times the matrix instructions.  A BF16 input fits
// the first half, so the first step has one term in A and two in the update.
//
// Scaling.  Halves hold 6 10^-8 .. 65504; X is held as 2^12 X, A and the polynomial as 2^8 A: an entry of A may be the
// square of a singular value, so that singular values up to 15.99 fit both.  What is held is X / u, where the unit u of
// each matrix and step is known from |G|, eps and the coefficients alone (ortho_factors): the first X is G times the power
// of two that brings its own norm to 1/2 .. 1 (exact), and while X can be at most S < 1, it is held in units of the power of
// two above S.  So a G far below eps, whose X is tiny, keeps its bits; from S = 1 on the unit is one.
//
// Layout.  X (rows along n) serves A's product, X^T (rows along m) the update's: X^T_new = X^T P is a product
// of rows again.  The update writes both: a patch of accumulators is transposed in registers, eight lanes exchanging
// 8 x 8 values, so that either goes out in 16-byte stores.  Second halves lie beside the first ones, in matrices of their own.
// Rows are padded with zeros to whole stages of 64 halves.
//
// Bound, where the tiles fill the card, by row_gemm.hpp's loop and in the update by its epilogue as well, 12 bytes an element
// read and written.  A lone matrix's A and A^2 have few tiles and long contractions, which are split, the parts being added
// up by a second kernel with the same epilogue.  Measured, five steps (us): 32 of 1408 x 2048 8900 (a step: A 524, P 407,
// update 967, 0.8 to 1.03 PFLOP/s of what is computed; before them norm 39 and first X 90, 6.1 TB/s), 11264 x 2048 FP32 2630
// (142 + 18, 35 + 15, 322; 24 and 59), 8 of 512 x 384 191 (17 launches that wait for each other, 6 to 16 each).
#include <cmath>

#include "launch.hpp"
#include "ortho_plan.hpp"
#include "quant_common.hpp"
#include "row_gemm.hpp"

namespace fp8bq {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));

constexpr float kScaleX = 4096.0f, kScaleA = 256.0f;

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, v2h));
}
__device__ __forceinline__ void unpack_f16x2(uint32_t w, float& lo, float& hi) {
  const v2h v = __builtin_bit_cast(v2h, w);
  lo = (float)v.x;
  hi = (float)v.y;
}

// 8 x 8 values of 16 bits held by eight neighbouring lanes, one row (four pairs) a lane, transposed: first within pairs
// of lanes, then pairs of values between lanes 2 and 4 apart.
__device__ __forceinline__ void transpose8(u32x4& d, int lane) {
  const uint32_t sel = (lane & 1) ? 0x03020706u : 0x05040100u;
#pragma unroll
  for (int k = 0; k < 4; ++k) d[k] = __builtin_amdgcn_perm(dpp_read<kDppXor1>(d[k]), d[k], sel);
  const bool b1 = (lane & 2) != 0;
#pragma unroll
  for (int k = 0; k < 4; k += 2) {
    const uint32_t got = dpp_read<kDppXor2>(b1 ? d[k] : d[k + 1]);
    d[k] = b1 ? got : d[k];
    d[k + 1] = b1 ? d[k + 1] : got;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t p = d[k], q = d[k + 2];
    d[k + 2] = (uint32_t)__builtin_amdgcn_update_dpp((int)q, (int)p, 0x104, 0xF, 0x5, false);  // row_shl:4
    d[k] = (uint32_t)__builtin_amdgcn_update_dpp((int)p, (int)q, 0x114, 0xF, 0xA, false);      // row_shr:4
  }
}

// Sums of squares: parts[batch][block], in 64 bits (gradients may be as small as their squares are not in FP32).
template <typename TIn>
__global__ __launch_bounds__(256) void ortho_norm_kernel(const TIn* __restrict__ g, int64_t R, int64_t C, int64_t ldg,
                                                         int64_t bstride, int wide, double* __restrict__ parts) {
  __shared__ double red[4];
  const TIn* gb = g + (int64_t)blockIdx.y * bstride;
  double sum = 0.0;
  if (wide) {
    const int64_t chunks = C / 8, total = R * chunks;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
      const int64_t r = i / chunks, c = i - r * chunks;
      float v[8];
      Load8<TIn>::run(gb + r * ldg + 8 * c, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = __builtin_fma((double)v[k], (double)v[k], sum);
    }
  } else {
    const int64_t total = R * C;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
      const int64_t r = i / C, c = i - r * C;
      double v;
      if constexpr (sizeof(TIn) == 2) v = (double)bf16lo(gb[r * ldg + c]);
      else v = (double)gb[r * ldg + c];
      sum = __builtin_fma(v, v, sum);
    }
  }
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) sum += __shfl_xor(sum, s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) parts[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// The coefficients' magnitudes, from which the units are found.
struct OrthoSteps {
  int steps;
  float a[kMaxOrthoSteps], b[kMaxOrthoSteps], c[kMaxOrthoSteps];
};
// What a matrix's epilogues multiply with: of step k factor[2 k] for A (u_k^2) and factor[2 k + 1] for the update (u_k / u_k+1;
// in the last step u_k, as the result is in units of one).  norm = |G|; u_0 = 2^ex / (norm + eps).
__device__ __forceinline__ void ortho_factors(const OrthoSteps& s, double norm, int ex, double eps, float* factor) {
  double u = norm > 0.0 ? __builtin_ldexp(1.0, ex) / (norm + eps) : 1.0;
  double most = norm / (norm + eps);  // no singular value of X is larger (nor its norm)
  for (int k = 0; k < s.steps; ++k) {
    const double q = most * most;
    most *= (double)s.a[k] + q * ((double)s.b[k] + q * (double)s.c[k]);
    most = most < 16.0 ? most : 16.0;
    const double above = __builtin_ldexp(1.0, __builtin_amdgcn_frexp_exp(most));
    // (2^-120: quotients of units stay finite, and a smaller result is zero in BF16)
    const double next = k == s.steps - 1 || !(most > 0.0) || above > 1.0 ? 1.0 : above < 0x1p-120 ? 0x1p-120 : above;
    factor[2 * k] = (float)(u * u);
    factor[2 * k + 1] = (float)(u / next);
    u = next;
  }
}

// The first X in both layouts, from tiles of 64 x 64 of G, and the factors.  tall: G is X^T.
struct OrthoBuffers {
  uint16_t *x, *x_low;    // [batch][m][np] first and second halves (second: FP32 input; BF16 fits the first)
  uint16_t *xt, *xt_low;  // [batch][n][mp]
  int64_t m, n, mp, np;
};
template <typename TIn>
__global__ __launch_bounds__(256) void ortho_begin_kernel(const TIn* __restrict__ g, int64_t R, int64_t C, int64_t ldg,
                                                          int64_t bstride, const double* __restrict__ parts, int nparts,
                                                          double eps, OrthoBuffers b, int tall, int wide, OrthoSteps steps,
                                                          float* __restrict__ factor) {
  __shared__ __attribute__((aligned(16))) uint16_t tile[64][72];
  __shared__ __attribute__((aligned(16))) uint16_t low[sizeof(TIn) == 4 ? 64 : 1][72];
  const int t = threadIdx.x, batch = blockIdx.z;
  const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
  const TIn* gb = g + (int64_t)batch * bstride;
  const int row = t >> 3, c = 8 * (t & 7);  // eight columns of rows row and row + 32, on their way while the norm is taken
  float v[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t r = r0 + row + 32 * h;
    if (wide && r < R && c0 + c < C) {
      Load8<TIn>::run(gb + r * ldg + c0 + c, v[h]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[h][i] = 0.0f;
        if (r < R && c0 + c + i < C) {
          if constexpr (sizeof(TIn) == 2) v[h][i] = bf16lo(gb[r * ldg + c0 + c + i]);
          else v[h][i] = gb[r * ldg + c0 + c + i];
        }
      }
    }
  }
  double sum = 0.0;  // (every wave alike, in a fixed order)
  for (int i = t & 63; i < nparts; i += 64) sum += parts[(int64_t)batch * nparts + i];
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) sum += __shfl_xor(sum, s);
  const double norm = __builtin_sqrt(sum);
  const bool finite = norm < __builtin_inf();
  // norm = fr 2^ex, 1/2 <= fr < 1: held is G 2^(12 - ex)
  const int ex = finite ? __builtin_amdgcn_frexp_exp(norm) : 0;
  if (t == 0 && blockIdx.x == 0 && blockIdx.y == 0) {
    float* f = factor + (int64_t)batch * (2 * kMaxOrthoSteps);
    if (finite) {
      ortho_factors(steps, norm, ex, eps, f);
    } else {
      for (int k = 0; k < 2 * steps.steps; ++k) f[k] = __builtin_nanf("");
    }
  }
  // (buffers are padded to whole tiles of 64 along their rows; rows past the matrix are not there)
  // straight: rows of G; turned: its columns
  const int64_t of_x = (int64_t)batch * b.m * b.np, of_xt = (int64_t)batch * b.n * b.mp;
  uint16_t* straight = tall ? b.xt + of_xt : b.x + of_x;
  uint16_t* straight_low = tall ? b.xt_low + of_xt : b.x_low + of_x;
  uint16_t* turned = tall ? b.x + of_x : b.xt + of_xt;
  uint16_t* turned_low = tall ? b.x_low + of_x : b.xt_low + of_xt;
  const int64_t lds = tall ? b.mp : b.np, ldt = tall ? b.np : b.mp;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t r = r0 + row + 32 * h;
    u32x4 hi, lo = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a0 = __builtin_ldexpf(v[h][2 * i], 12 - ex), a1 = __builtin_ldexpf(v[h][2 * i + 1], 12 - ex);
      hi[i] = pack_f16x2(a0, a1);
      if constexpr (sizeof(TIn) == 4) {
        float h0, h1;
        unpack_f16x2(hi[i], h0, h1);
        lo[i] = pack_f16x2(a0 - h0, a1 - h1);
      }
    }
    *reinterpret_cast<u32x4*>(&tile[row + 32 * h][c]) = hi;
    if constexpr (sizeof(TIn) == 4) *reinterpret_cast<u32x4*>(&low[row + 32 * h][c]) = lo;
    if (r < R) {
      *reinterpret_cast<u32x4*>(straight + r * lds + c0 + c) = hi;
      if constexpr (sizeof(TIn) == 4) *reinterpret_cast<u32x4*>(straight_low + r * lds + c0 + c) = lo;
    }
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = row + 32 * h;  // column of G; rows c .. c + 7
    if (c0 + i >= C) continue;
    u32x4 hi, lo;
#pragma unroll
    for (int k = 0; k < 4; ++k) hi[k] = tile[c + 2 * k][i] | (uint32_t)tile[c + 2 * k + 1][i] << 16;
    *reinterpret_cast<u32x4*>(turned + (c0 + i) * ldt + r0 + c) = hi;
    if constexpr (sizeof(TIn) == 4) {
#pragma unroll
      for (int k = 0; k < 4; ++k) lo[k] = low[c + 2 * k][i] | (uint32_t)low[c + 2 * k + 1][i] << 16;
      *reinterpret_cast<u32x4*>(turned_low + (c0 + i) * ldt + r0 + c) = lo;
    }
  }
}

// What is done with a row of patches of a finished tile.
enum OrthoStep : int { kOrthoGram = 0, kOrthoPoly = 1, kOrthoUpdate = 2, kOrthoLast = 3, kOrthoLastWide = 4 };
struct OrthoEnd {
  float a, b, c;          // the step's coefficients
  const float* factor;    // Gram, update: the step's factor of the first matrix
  const uint16_t *old, *old_low;  // polynomial: A; update: X^T as it was (second halves null: zeros)
  uint16_t *to, *to_low;          // Gram, polynomial: [batch][m][mp]; update: X^T
  uint16_t *x, *x_low;            // update: X
  uint16_t* out;          // last: BF16 result [batch], rows ldo apart
  int64_t ldo, obatch;
  int vec;                // 16-byte stores into it are possible
  int64_t m, n, mp, np;
};

// Rows [0, rows) x columns [0, width) of 16-bit values: eight columns from col on, as far as they are there (all eight
// where the buffer is padded: width a multiple of 64).
__device__ __forceinline__ void put8(uint16_t* row, int64_t col, int64_t width, bool vec, const u32x4& d) {
  if (col >= width) return;
  if (vec && col + 8 <= width) {
    *reinterpret_cast<u32x4*>(row + col) = d;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (col + k < width) row[col + k] = (uint16_t)(d[k >> 1] >> (16 * (k & 1)));
  }
}

// A lane's two 16-byte chunks of a patch row (columns 0 .. 7 and 16 .. 23 of its half): lanes l and l + 16 swap one, so that an
// access takes 64 contiguous bytes of 16 rows and not 32 of 32 rows (2% of 11264 x 2048 with one term).  The swap undoes itself: it stands behind loads and
// ahead of stores, and chunk q then lies at row m - (l & 16) + 16 q, column n0 + (l & 16).
__device__ __forceinline__ void swap_chunks(u32x4 (&d)[2]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const auto p = __builtin_amdgcn_permlane16_swap(d[0][k], d[1][k], false, false);
    d[0][k] = p[0];
    d[1][k] = p[1];
  }
}
__device__ __forceinline__ int64_t swapped_at(int64_t m, int64_t n0, int64_t ld, int lane) {
  return (m - (lane & 16)) * ld + n0 + (lane & 16);
}

// What a patch's end reads: A (polynomial), or X^T as it was and its second half (update).  Whole tiles: as loaded, chunks
// still swapped.
struct OrthoOld {
  u32x4 hi[2], lo[2];
};
template <int STEP>
__device__ __forceinline__ void ortho_load(const OrthoEnd& e, const RowPlace& p, int64_t m, int64_t n0, OrthoOld& o) {
  if constexpr (STEP == kOrthoGram) return;
  const int64_t rows = STEP == kOrthoPoly ? e.m : e.n;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    o.hi[q] = o.lo[q] = (u32x4){0, 0, 0, 0};
    if (!p.whole && (m >= p.mlim || n0 + 16 * q >= e.mp)) continue;
    const int64_t at = p.batch * rows * e.mp + (p.whole ? swapped_at(m, n0, e.mp, p.lane) + 16 * q * e.mp : m * e.mp + n0 + 16 * q);
    o.hi[q] = *reinterpret_cast<const u32x4*>(e.old + at);
    if (e.old_low) o.lo[q] = *reinterpret_cast<const u32x4*>(e.old_low + at);
  }
}

// Both chunks of a row of a matrix (rows ld apart) of which `width` columns are there.
__device__ __forceinline__ void put_chunks(uint16_t* o, int64_t ld, int64_t width, bool vec, const RowPlace& p, int64_t m,
                                           int64_t n0, const u32x4 (&d)[2]) {
  if (p.whole && vec) {
    u32x4 w[2] = {d[0], d[1]};
    swap_chunks(w);
    uint16_t* at = o + swapped_at(m, n0, ld, p.lane);
    *reinterpret_cast<u32x4*>(at) = w[0];
    *reinterpret_cast<u32x4*>(at + 16 * ld) = w[1];
  } else if (m < p.mlim) {
    put8(o + m * ld, n0, width, vec, d[0]);
    put8(o + m * ld, n0 + 16, width, vec, d[1]);
  }
}
// Their transposes: eight rows of the patch in a row of a matrix whose rows are the patch's columns.
__device__ __forceinline__ void put_turned(uint16_t* o, int64_t ld, int64_t width, bool vec, const RowPlace& p, int64_t m,
                                           int64_t n0, const u32x4 (&d)[2]) {
  const int turn = p.lane & 7;  // the lane's column among the eight after the turn
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    u32x4 w = d[q];
    transpose8(w, p.lane);
    const int64_t n = n0 + 16 * q + turn;
    if (n < p.nlim) put8(o + n * ld, m - turn, width, vec, w);
  }
}

// STEP of one patch: v[8 q + i] is row m, column n0 + 16 q + i of the product.
template <int STEP>
__device__ __forceinline__ void ortho_patch(const OrthoEnd& e, const v16f& v, const RowPlace& p, int64_t m, int64_t n0, float f,
                                            OrthoOld& old) {
  if (STEP != kOrthoGram && p.whole) {
    swap_chunks(old.hi);
    if (e.old_low) swap_chunks(old.lo);
  }
  u32x4 d[2], l[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = v[8 * q + i];
    if constexpr (STEP == kOrthoGram) {
      const float s = f * (kScaleA / (kScaleX * kScaleX));
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= s;
    } else if constexpr (STEP == kOrthoPoly) {
      const float s = e.c * (1.0f / kScaleA);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float h0, h1, l0, l1;
        unpack_f16x2(old.hi[q][i], h0, h1);
        unpack_f16x2(old.lo[q][i], l0, l1);
        y[2 * i] = __builtin_fmaf(e.b, h0 + l0, s * y[2 * i]);
        y[2 * i + 1] = __builtin_fmaf(e.b, h1 + l1, s * y[2 * i + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float h0, h1, l0, l1;
        unpack_f16x2(old.hi[q][i], h0, h1);
        unpack_f16x2(old.lo[q][i], l0, l1);
        y[2 * i] = f * __builtin_fmaf(e.a, h0 + l0, y[2 * i] * (1.0f / kScaleA));
        y[2 * i + 1] = f * __builtin_fmaf(e.a, h1 + l1, y[2 * i + 1] * (1.0f / kScaleA));
      }
    }
    if (!p.whole) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = m < p.mlim && n0 + 16 * q + i < p.nlim ? y[i] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (STEP == kOrthoLast || STEP == kOrthoLastWide) {
        d[q][i] = pack_bf16x2(y[2 * i] * (1.0f / kScaleX), y[2 * i + 1] * (1.0f / kScaleX));
      } else {
        d[q][i] = pack_f16x2(y[2 * i], y[2 * i + 1]);
        float h0, h1;
        unpack_f16x2(d[q][i], h0, h1);
        l[q][i] = pack_f16x2(y[2 * i] - h0, y[2 * i + 1] - h1);
      }
    }
  }
  if constexpr (STEP == kOrthoGram || STEP == kOrthoPoly) {
    const int64_t at = p.batch * e.m * e.mp;
    put_chunks(e.to + at, e.mp, e.mp, true, p, m, n0, d);
    put_chunks(e.to_low + at, e.mp, e.mp, true, p, m, n0, l);
    if (p.mirror) {
      put_turned(e.to + at, e.mp, e.mp, true, p, m, n0, d);
      put_turned(e.to_low + at, e.mp, e.mp, true, p, m, n0, l);
    }
  } else if constexpr (STEP == kOrthoUpdate) {
    const int64_t at = p.batch * e.n * e.mp, of_x = p.batch * e.m * e.np;
    put_chunks(e.to + at, e.mp, e.mp, true, p, m, n0, d);
    put_chunks(e.to_low + at, e.mp, e.mp, true, p, m, n0, l);
    put_turned(e.x + of_x, e.np, e.np, true, p, m, n0, d);
    put_turned(e.x_low + of_x, e.np, e.np, true, p, m, n0, l);
  } else {
    uint16_t* o = e.out + p.batch * e.obatch;
    if constexpr (STEP == kOrthoLast) put_chunks(o, e.ldo, e.m, e.vec != 0, p, m, n0, d);
    else put_turned(o, e.ldo, e.n, e.vec != 0, p, m, n0, d);
  }
}

// MI x NI patches; what a patch reads is asked for two patches ahead (with one term 11264 x 2048 1222 -> 1190 us, 16 of
// 1024 x 1024 751 -> 702).
template <int STEP, int MI, int NI>
__device__ __forceinline__ void ortho_patches(const OrthoEnd& e, const v16f (&v)[MI][NI], const RowPlace& p) {
  constexpr int P = MI * NI, kAhead = 2;
  const float f = STEP == kOrthoPoly ? 1.0f : e.factor[p.batch * (2 * kMaxOrthoSteps)];
  OrthoOld old[kAhead + 1];
#pragma unroll
  for (int u = 0; u < (P < kAhead ? P : kAhead); ++u) ortho_load<STEP>(e, p, p.m + 32 * (u / NI), p.n + 32 * (u % NI), old[u]);
#pragma unroll
  for (int u = 0; u < P; ++u) {
    const int w = u + kAhead;
    if (w < P) ortho_load<STEP>(e, p, p.m + 32 * (w / NI), p.n + 32 * (w % NI), old[w % (kAhead + 1)]);
    __builtin_amdgcn_sched_barrier(0);
    ortho_patch<STEP>(e, v[u / NI][u % NI], p, p.m + 32 * (u / NI), p.n + 32 * (u % NI), f, old[u % (kAhead + 1)]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <int STEP>
constexpr int ortho_units() { return STEP == kOrthoGram || STEP == kOrthoPoly ? kUnitsTriangle : kUnitsFull; }

template <int BM, int BN, int WGM, int WGN, int NST, int STEP>
__global__ __launch_bounds__(WGM* WGN * 64, (RowTile<BM, BN, WGM * WGN, NST>::kMinWaves)) void ortho_gemm_kernel(
    RowDesc d, OrthoEnd e, uint32_t tiles_m, uint32_t tiles_n, int batches) {
  using Tile = RowTile<BM, BN, WGM * WGN, NST>;
  constexpr int MI = BM / WGM / 32, NI = BN / WGN / 32;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[Tile::kRing];
  auto end = [&](const v16f (&acc)[MI][NI], const RowPlace& p) {
    ortho_patches<STEP, MI, NI>(e, acc, p);
  };
  row_gemm_units<kRowsF16, BM, BN, WGM, WGN, NST, ortho_units<STEP>()>(d, tiles_m, tiles_n, 1, batches, nullptr, smem, end);
}

// Split contractions: a part's sums as the lanes hold them, parts[part][batch][tile][wave][patch][quarter][lane] of four
// floats; and the kernel that adds them up, one row of a wave's patches to a wave.
template <int BM, int BN, int WGM, int WGN, int NST>
__global__ __launch_bounds__(WGM* WGN * 64, (RowTile<BM, BN, WGM * WGN, NST>::kMinWaves)) void ortho_part_kernel(
    RowDesc d, v4f* __restrict__ parts, uint32_t tiles, int nsplit, int batches) {
  using Tile = RowTile<BM, BN, WGM * WGN, NST>;
  constexpr int MI = BM / WGM / 32, NI = BN / WGN / 32;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[Tile::kRing];
  const int64_t T = (int64_t)tiles * (tiles + 1) / 2;
  auto end = [&](const v16f (&acc)[MI][NI], const RowPlace& p) {
    v4f* o = parts + (((int64_t)p.split * batches + p.batch) * T + p.tile) * (BM * BN / 4) + p.wave * (MI * NI * 4 * 64) + p.lane;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          o[((i * NI + j) * 4 + r) * 64] = (v4f){acc[i][j][4 * r], acc[i][j][4 * r + 1], acc[i][j][4 * r + 2], acc[i][j][4 * r + 3]};
  };
  row_gemm_units<kRowsF16, BM, BN, WGM, WGN, NST, kUnitsTriangle>(d, tiles, tiles, nsplit, batches, nullptr, smem, end);
}
template <int BM, int BN, int WGM, int WGN, int STEP>
__global__ __launch_bounds__(256) void ortho_sum_kernel(OrthoEnd e, const v4f* __restrict__ parts, uint32_t tiles, int nsplit,
                                                        int batches) {
  constexpr int NW = WGM * WGN, MI = BM / WGM / 32, NI = BN / WGN / 32;
  const uint32_t T = tiles * (tiles + 1) / 2;
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  if (unit >= (int64_t)T * batches * (NW * MI)) return;
  const int i = (int)(unit % MI), wave = (int)(unit / MI % NW);
  const int64_t bt = unit / (MI * NW);
  const uint32_t w = (uint32_t)(bt % T);
  v16f v[1][NI];
  const v4f* at = parts + bt * (BM * BN / 4) + ((wave * MI + i) * NI) * (4 * 64) + lane;
  const int64_t step = (int64_t)T * batches * (BM * BN / 4);
#pragma unroll
  for (int j = 0; j < NI; ++j)
#pragma unroll
    for (int x = 0; x < 16; ++x) v[0][j][x] = 0.0f;
#pragma unroll 2
  for (int k = 0; k < nsplit; ++k, at += step) {  // (in the order of the parts; a part's loads are in flight together)
    v4f s[NI * 4];
#pragma unroll
    for (int q = 0; q < NI * 4; ++q) s[q] = at[q * 64];
#pragma unroll
    for (int q = 0; q < NI * 4; ++q)
#pragma unroll
      for (int x = 0; x < 4; ++x) v[0][q / 4][4 * (q % 4) + x] += s[q][x];
  }
  uint32_t tm, tn;
  row_tile<kUnitsTriangle>(w, tiles, tiles, tm, tn);
  RowPlace p;
  p.m0 = (int64_t)tm * BM;
  p.n0 = (int64_t)tn * BN;
  p.mlim = p.nlim = e.m;
  p.m = p.m0 + wave / WGN * (BM / WGM) + (lane & 31);
  p.n = p.n0 + wave % WGN * (BN / WGN) + 8 * (lane >> 5);
  p.ccol = 0;
  p.split = 0;
  p.batch = (int)(bt / T);
  p.lane = lane;
  p.tile = w;
  p.wave = wave;
  p.whole = p.m0 + BM <= p.mlim && p.n0 + BN <= p.nlim;
  p.mirror = tm != tn;
  p.m += 32 * i;
  ortho_patches<STEP, 1, NI>(e, v, p);
}

template <int BM, int BN, int WGM, int WGN, int NST, int STEP>
static hipError_t launch_product_tile(const RowDesc& d, const OrthoEnd& e, const OrthoProduct& p, int batches, void* parts,
                                      hipStream_t st) {
  const dim3 block(WGM * WGN * 64);
  if constexpr (ortho_units<STEP>() == kUnitsTriangle) {
    if (p.split > 1) {
      hipLaunchKernelGGL((ortho_part_kernel<BM, BN, WGM, WGN, NST>), dim3((unsigned)p.grid), block, 0, st, d, (v4f*)parts,
                         (uint32_t)p.tiles_m, p.split, batches);
      const hipError_t r = hipGetLastError();
      if (r != hipSuccess) return r;
      const int64_t units = p.tiles * batches * (WGM * WGN * (BM / WGM / 32));
      hipLaunchKernelGGL((ortho_sum_kernel<BM, BN, WGM, WGN, STEP>), dim3((unsigned)((units + 3) / 4)), dim3(256), 0, st, e,
                         (const v4f*)parts, (uint32_t)p.tiles_m, p.split, batches);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((ortho_gemm_kernel<BM, BN, WGM, WGN, NST, STEP>), dim3((unsigned)p.grid), block, 0, st, d, e,
                     (uint32_t)p.tiles_m, (uint32_t)p.tiles_n, batches);
  return hipGetLastError();
}
template <int STEP>
static hipError_t launch_product(const RowDesc& d, const OrthoEnd& e, const OrthoProduct& p, int batches, void* parts,
                                 hipStream_t st) {
  switch (p.shape) {
    case k256x256: return launch_product_tile<256, 256, 2, 4, 2, STEP>(d, e, p, batches, parts, st);
    case k256x192:
      if constexpr (ortho_units<STEP>() == kUnitsFull) return launch_product_tile<256, 192, 4, 2, 2, STEP>(d, e, p, batches, parts, st);
      return hipErrorInvalidValue;  // (never planned for a symmetric result)
    case k64x64:
      return p.deep ? launch_product_tile<64, 64, 2, 2, 3, STEP>(d, e, p, batches, parts, st)
                    : launch_product_tile<64, 64, 2, 2, 2, STEP>(d, e, p, batches, parts, st);
    default: return launch_product_tile<128, 128, 2, 2, 2, STEP>(d, e, p, batches, parts, st);
  }
}

#define FP8BQ_TRY(call)                      \
  do {                                       \
    const hipError_t err = (call);           \
    if (err != hipSuccess) return err;       \
  } while (0)

hipError_t launch_ortho(const void* g, int gt, int64_t ldg, int64_t gbatch, const OrthoPlan& p, int steps, const double* coef,
                        double eps, void* out, int64_t ldo, int64_t obatch, void* ws, hipStream_t st) {
  const bool tall = p.R >= p.C;
  uint8_t* w = (uint8_t*)ws;
  double* norms = (double*)(w + p.at_norms);
  float* factor = (float*)(w + p.at_factor);
  const int es = gt == 0 ? 2 : 4, B = (int)p.batch;
  // (of X^T, A and the polynomial the second halves lie behind the first ones of all matrices)
  const int64_t to_low_xt = p.batch * p.n * p.mp, to_low_sym = p.batch * p.m * p.mp;
  uint16_t* x = (uint16_t*)(w + p.at_x);
  uint16_t* x_low = (uint16_t*)(w + p.at_low);
  uint16_t* xt[2] = {(uint16_t*)(w + p.at_xt[0]), (uint16_t*)(w + p.at_xt[1])};
  uint16_t* gram = (uint16_t*)(w + p.at_gram);
  uint16_t* poly = (uint16_t*)(w + p.at_poly);
  void* parts = w + p.at_parts;
  const int wide = p.C % 8 == 0 && ((uintptr_t)g & 15) == 0 && ldg * es % 16 == 0 && (gbatch * es % 16 == 0 || B == 1);

  const dim3 ngrid((unsigned)p.norm_blocks, (unsigned)B);
  const dim3 bgrid((unsigned)((p.C + 63) / 64), (unsigned)((p.R + 63) / 64), (unsigned)B);
  OrthoSteps how{};
  how.steps = steps;
  for (int k = 0; k < steps; ++k) {
    how.a[k] = (float)std::fabs(coef[3 * k]);
    how.b[k] = (float)std::fabs(coef[3 * k + 1]);
    how.c[k] = (float)std::fabs(coef[3 * k + 2]);
  }
  const OrthoBuffers b{x, x_low, xt[0], xt[0] + to_low_xt, p.m, p.n, p.mp, p.np};
  if (gt == 0) {
    hipLaunchKernelGGL(ortho_norm_kernel<uint16_t>, ngrid, dim3(256), 0, st, (const uint16_t*)g, p.R, p.C, ldg, gbatch, wide, norms);
    FP8BQ_TRY(hipGetLastError());
    hipLaunchKernelGGL(ortho_begin_kernel<uint16_t>, bgrid, dim3(256), 0, st, (const uint16_t*)g, p.R, p.C, ldg, gbatch, norms,
                       p.norm_blocks, eps, b, (int)tall, wide, how, factor);
  } else {
    hipLaunchKernelGGL(ortho_norm_kernel<float>, ngrid, dim3(256), 0, st, (const float*)g, p.R, p.C, ldg, gbatch, wide, norms);
    FP8BQ_TRY(hipGetLastError());
    hipLaunchKernelGGL(ortho_begin_kernel<float>, bgrid, dim3(256), 0, st, (const float*)g, p.R, p.C, ldg, gbatch, norms,
                       p.norm_blocks, eps, b, (int)tall, wide, how, factor);
  }
  FP8BQ_TRY(hipGetLastError());

  for (int k = 0; k < steps; ++k) {
    const bool first = k == 0, last = k == steps - 1;
    OrthoEnd e{};
    e.a = (float)coef[3 * k];
    e.b = (float)coef[3 * k + 1];
    e.c = (float)coef[3 * k + 2];
    e.factor = factor + 2 * k;
    const bool low = !(first && gt == 0);  // X has second halves
    e.x = x;
    e.x_low = x_low;
    e.out = (uint16_t*)out;
    e.ldo = ldo;
    e.obatch = obatch;
    e.vec = ((uintptr_t)out & 15) == 0 && ldo % 8 == 0 && (obatch % 8 == 0 || B == 1);
    e.m = p.m;
    e.n = p.n;
    e.mp = p.mp;
    e.np = p.np;
    RowDesc d{};
    d.a = d.b = (const uint8_t*)x;  // A = X X^T
    d.lda = d.ldb = 2 * p.np;
    d.M = d.N = p.m;
    d.K = 2 * p.np;
    d.abatch = d.bbatch = 2 * p.m * p.np;
    d.alow = d.blow = 2 * (x_low - x);
    d.terms = low ? 3 : 1;
    e.to = gram;
    e.to_low = gram + to_low_sym;
    FP8BQ_TRY(launch_product<kOrthoGram>(d, e, p.gram, B, parts, st));
    d.a = d.b = (const uint8_t*)gram;  // P
    d.lda = d.ldb = 2 * p.mp;
    d.K = 2 * p.mp;
    d.abatch = d.bbatch = 2 * p.m * p.mp;
    d.alow = d.blow = 2 * to_low_sym;
    d.terms = 3;
    e.old = gram;
    e.old_low = gram + to_low_sym;
    e.to = poly;
    e.to_low = poly + to_low_sym;
    FP8BQ_TRY(launch_product<kOrthoPoly>(d, e, p.poly, B, parts, st));
    e.factor = factor + 2 * k + 1;
    d.a = (const uint8_t*)xt[k & 1];  // X^T P
    d.lda = 2 * p.mp;
    d.b = (const uint8_t*)poly;
    d.M = p.n;
    d.abatch = 2 * p.n * p.mp;
    d.alow = 2 * to_low_xt;
    d.terms = low ? 3 : 2;
    e.old = xt[k & 1];
    e.old_low = low ? xt[k & 1] + to_low_xt : nullptr;
    e.to = xt[(k & 1) ^ 1];
    e.to_low = e.to + to_low_xt;
    if (!last)
      FP8BQ_TRY(launch_product<kOrthoUpdate>(d, e, p.update, B, nullptr, st));
    else if (tall)
      FP8BQ_TRY(launch_product<kOrthoLast>(d, e, p.update, B, nullptr, st));
    else
      FP8BQ_TRY(launch_product<kOrthoLastWide>(d, e, p.update, B, nullptr, st));
  }
  return hipSuccess;
}

}  // namespace fp8bq
