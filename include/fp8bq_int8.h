/*
 * fp8bq_int8.h -- the linear layer in 8-bit integers, with one scale for each token and one for each output channel,
 * for AMD Instinct MI355X (gfx950), dense and grouped by expert.
 *
 * Quantization rule, per row of an operand (a token of X, an output channel of W):
 *   s = max(fp32(max |x| / 127), fp32(1e-12));   q = fp32(x / s) to the nearest integer, ties to even;   value = q s.
 * Both divisions are IEEE.  A row that holds a NaN or an infinity has the scale NaN and unspecified codes, and every
 * product over it is NaN.  Codes (int8, -127 .. 127) and scales (FP32) are a deterministic function of the input.
 *
 * Products: C[m, n] = sa[m] sb[n] sum_k qa[m, k] qb[n, k].  The sum is exact (32-bit integers: K < 2^17; codes of -128
 * are allowed) and is rounded when it becomes FP32, at each scale and to the output's type; with FP32 scales the same
 * codes give the same result whatever the sizes around them.
 *
 * Layouts.  Codes [R, K] bytes, row stride a multiple of 16; K % 16 == 0.  Scales [R] FP32, contiguous.  Output
 * matrices may have any leading dimension >= N.  Conventions, alignment, errors and stream order as in fp8bq.h (inputs
 * need not be finite here); R and C of the quantizers, M and N are below 2^30, and 255 times the leading dimension of
 * codes plus K is below 2^31.  The quantizers are no-ops without rows or without columns: scales over no elements, by the
 * rule 1e-12, are the caller's to set.
 */
#ifndef FP8BQ_INT8_H_
#define FP8BQ_INT8_H_

#include "fp8bq.h"
#include "fp8bq_grouped.h" /* FP8BQ_MAX_EXPERTS, the meaning of offsets */

#ifdef __cplusplus
extern "C" {
#endif

/* Rows: x [R, C] (BF16 or FP32, row stride ldx; C % 16 == 0) -> q [R, C] (ldq), s [R]. */
int fp8bq_quantize_int8(const void* x, fp8bq_in xt, int64_t R, int64_t C, int64_t ldx, int8_t* q, int64_t ldq, float* s,
                        void* stream);

/*
 * Columns, transposed: the operands of the products that contract over the rows.  x [R, C] (C % 8 == 0) ->
 *   qt [C, 16 ceil(R / 16)] (ldqt): code of x[r, c] in byte r of row c, zeros from R on;   st [C].
 *   ws  at least fp8bq_quantize_int8_t_workspace_size(R, C) bytes.
 */
size_t fp8bq_quantize_int8_t_workspace_size(int64_t R, int64_t C);
int fp8bq_quantize_int8_t(const void* x, fp8bq_in xt, int64_t R, int64_t C, int64_t ldx, int8_t* qt, int64_t ldqt,
                          float* st, void* ws, size_t ws_bytes, void* stream);

/*
 * C [M, N] = A [M, K] . B [N, K]^T.
 * fprop: A = rows of X, B = rows of W;  dgrad: A = rows of dY, B = columns of W;  wgrad: A = columns of dY,
 * B = columns of X, K = the tokens rounded up to 16.
 *   M, N >= 0, any; 0 <= K < 2^17 (K == 0: zeros, or C unchanged when accumulating).
 *   ct  FP8BQ_OUT_BF16, FP8BQ_OUT_F32 or FP8BQ_OUT_F32_ACCUM (C = fp32(C + A B^T): longer contractions in parts).
 *   ws  at least fp8bq_gemm_int8_workspace_size(M, N, K) bytes (may be NULL when that is 0).
 */
size_t fp8bq_gemm_int8_workspace_size(int64_t M, int64_t N, int64_t K);
int fp8bq_gemm_int8(int64_t M, int64_t N, int64_t K, const int8_t* qa, int64_t ldqa, const float* sa, const int8_t* qb,
                    int64_t ldqb, const float* sb, void* c, fp8bq_out ct, int64_t ldc, void* ws, size_t ws_bytes,
                    void* stream);

/*
 * Linear layer with 8-bit weights: Y [M, N] = Q(X [M, K]) . W [N, K]^T, X quantized by the rule above inside the call;
 * the result is that of fp8bq_quantize_int8 followed by fp8bq_gemm_int8, bit for bit.
 *   x   [M, K] BF16 or FP32, row stride ldx.   y  [M, N] BF16 or FP32.
 *   ws  at least fp8bq_linear_int8_workspace_size(M, N, K) bytes (0 for a few tokens).
 */
size_t fp8bq_linear_int8_workspace_size(int64_t M, int64_t N, int64_t K);
int fp8bq_linear_int8(int64_t M, int64_t N, int64_t K, const void* x, fp8bq_in xt, int64_t ldx, const int8_t* qw,
                      int64_t ldqw, const float* sw, void* y, fp8bq_out yt, int64_t ldy, void* ws, size_t ws_bytes,
                      void* stream);

/*
 * The two grouped by expert (offsets [E + 1], stacked weights and untouched rows as in fp8bq_grouped.h):
 *   Y_e [n_e, N] = X_e [n_e, K] . W_e [N, K]^T for the rows of every expert e.
 *   qa/sa  codes of X [T, K];  x  X itself.   qw  [E N, K];  sw  [E N].   y  [T, N] BF16 or FP32.
 *   K >= 16; N any; E N < 2^30.
 */
size_t fp8bq_grouped_gemm_int8_workspace_size(int64_t E, int64_t T, int64_t N, int64_t K);
int fp8bq_grouped_gemm_int8(int64_t E, int64_t T, int64_t N, int64_t K, const int64_t* offsets, const int8_t* qa,
                            int64_t ldqa, const float* sa, const int8_t* qw, int64_t ldqw, const float* sw, void* y,
                            fp8bq_out yt, int64_t ldy, void* ws, size_t ws_bytes, void* stream);
size_t fp8bq_grouped_linear_int8_workspace_size(int64_t E, int64_t T, int64_t N, int64_t K);
int fp8bq_grouped_linear_int8(int64_t E, int64_t T, int64_t N, int64_t K, const int64_t* offsets, const void* x,
                              fp8bq_in xt, int64_t ldx, const int8_t* qw, int64_t ldqw, const float* sw, void* y,
                              fp8bq_out yt, int64_t ldy, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BQ_INT8_H_ */
