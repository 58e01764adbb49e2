/*
 * fp8bq_mx.h -- the linear layer in microscaled 4-bit floating point (MXFP4) for AMD Instinct MI355X
 * (gfx950), dense and grouped by expert.
 *
 * Format (OCP Microscaling, MXFP4): blocks of 32 values along the contraction; E2M1 codes (1 sign, 2 exponent,
 * 1 mantissa bits: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte, the even element in the low
 * half; one E8M0 scale byte b per block, 2^(b - 127), 255 = NaN.
 *
 * Quantization rule, per block:
 *   e = max(floor(log2(max |x|)) - 2, -127),  b = e + 127;   code = E2M1 of x 2^-e, nearest, ties to even, values
 *   past 6 to 6 (the sign of a value that rounds to zero is kept).
 *   A block of zeros has b = 0.  A block that holds a NaN or an infinity has b = 255 and unspecified codes, and
 *   every product over it is NaN.
 * The codes and scales are a deterministic function of the input.
 *
 * Layouts.  Codes q [R, K / 2] bytes, row stride ldq in BYTES, a multiple of 16.  Scales: the bytes of four
 * consecutive blocks (128 values) form one 32-bit word, block j in byte j (little-endian); the words of a 128-long
 * stretch are contiguous over the rows: word (k / 128, r) is s[(k / 128) * lds + r], lds >= R in WORDS, any
 * value.  When K % 128 != 0 the last word's bytes past K / 32 are written as zeros and never used.
 *
 * Conventions, alignment, errors and stream order as in fp8bq.h (inputs need not be finite here).  Output
 * matrices may have any leading dimension >= N.
 */
#ifndef FP8BQ_MX_H_
#define FP8BQ_MX_H_

#include "fp8bq.h"
#include "fp8bq_grouped.h" /* FP8BQ_MAX_EXPERTS, the meaning of offsets */

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Quantizer.  Row outputs (blocks of 32 consecutive elements of a row), column outputs (blocks of 32
 * consecutive rows of a column, transposed: the operands of the products that contract over the rows), or
 * both from one read; a pair that is not wanted is NULL.
 *   x   [R, C] input (BF16 or FP32), row stride ldx; C % 8 == 0, and C % 32 == 0 with row outputs.
 *   q   [R, C / 2] codes (ldq),  s  [ceil(C / 128)][R] scale words (lds).
 *   qt  [C, 16 ceil(R / 32)] bytes (ldqt): code of x[r, c] in byte r / 2 of row c; the rows that fill up the last
 *       block count as zeros.   st  [ceil(R / 128)][C] scale words (ldst).
 */
int fp8bq_quantize_mxfp4(const void* x, fp8bq_in xt, int64_t R, int64_t C, int64_t ldx, uint8_t* q, int64_t ldq,
                         uint32_t* s, int64_t lds, uint8_t* qt, int64_t ldqt, uint32_t* st, int64_t ldst,
                         void* stream);

/*
 * Product of two MXFP4 operands, both contiguous along the contraction:
 *   C [M, N] = A [M, K] . B [N, K]^T,  FP32 accumulation.
 * fprop: A = rows of X, B = rows of W;  dgrad: A = rows of dY, B = columns of W;  wgrad: A = columns of dY,
 * B = columns of X, K = the tokens rounded up to 32.
 *   M, N >= 0, any; K % 32 == 0 (K == 0: zeros, or C unchanged when accumulating).
 *   ct  FP8BQ_OUT_BF16, FP8BQ_OUT_F32 or FP8BQ_OUT_F32_ACCUM (C = fp32(C + A B^T)).
 *   ws  at least fp8bq_gemm_mxfp4_workspace_size(M, N, K) bytes (may be NULL when that is 0).
 */
size_t fp8bq_gemm_mxfp4_workspace_size(int64_t M, int64_t N, int64_t K);
int fp8bq_gemm_mxfp4(int64_t M, int64_t N, int64_t K, const uint8_t* qa, int64_t ldqa, const uint32_t* sa,
                     int64_t ldsa, const uint8_t* qb, int64_t ldqb, const uint32_t* sb, int64_t ldsb, void* c,
                     fp8bq_out ct, int64_t ldc, void* ws, size_t ws_bytes, void* stream);

/*
 * Linear layer with 4-bit weights: Y [M, N] = Q(X [M, K]) . W [N, K]^T, X quantized by the rule above inside the
 * call.  The result is that of fp8bq_quantize_mxfp4 followed by fp8bq_gemm_mxfp4 up to the order of the FP32 sum.
 *   x   [M, K] BF16 or FP32, row stride ldx.   y  [M, N] BF16 or FP32.
 *   ws  at least fp8bq_linear_mxfp4_workspace_size(M, N, K) bytes (0 for a few tokens: the codes of X then
 *       never leave the registers).
 */
size_t fp8bq_linear_mxfp4_workspace_size(int64_t M, int64_t N, int64_t K);
int fp8bq_linear_mxfp4(int64_t M, int64_t N, int64_t K, const void* x, fp8bq_in xt, int64_t ldx, const uint8_t* qw,
                       int64_t ldqw, const uint32_t* sw, int64_t ldsw, void* y, fp8bq_out yt, int64_t ldy, void* ws,
                       size_t ws_bytes, void* stream);

/*
 * The two grouped by expert (offsets [E + 1], stacked weights and untouched rows as in fp8bq_grouped.h):
 *   Y_e [n_e, N] = X_e [n_e, K] . W_e [N, K]^T for the rows of every expert e.
 *   qa/sa  codes of X [T, K] (row outputs);  x  X itself.   qw  [E N, K / 2];  sw  [ceil(K / 128)][E N] words.
 *   y  [T, N] BF16 or FP32.
 *   K % 32 == 0, K >= 32; N any; E N < 2^30.
 */
size_t fp8bq_grouped_gemm_mxfp4_workspace_size(int64_t E, int64_t T, int64_t N, int64_t K);
int fp8bq_grouped_gemm_mxfp4(int64_t E, int64_t T, int64_t N, int64_t K, const int64_t* offsets, const uint8_t* qa,
                             int64_t ldqa, const uint32_t* sa, int64_t ldsa, const uint8_t* qw, int64_t ldqw,
                             const uint32_t* sw, int64_t ldsw, void* y, fp8bq_out yt, int64_t ldy, void* ws,
                             size_t ws_bytes, void* stream);
size_t fp8bq_grouped_linear_mxfp4_workspace_size(int64_t E, int64_t T, int64_t N, int64_t K);
int fp8bq_grouped_linear_mxfp4(int64_t E, int64_t T, int64_t N, int64_t K, const int64_t* offsets, const void* x,
                               fp8bq_in xt, int64_t ldx, const uint8_t* qw, int64_t ldqw, const uint32_t* sw,
                               int64_t ldsw, void* y, fp8bq_out yt, int64_t ldy, void* ws, size_t ws_bytes,
                               void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BQ_MX_H_ */
