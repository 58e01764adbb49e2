/*
 * fp8bq_ortho.h -- orthogonalization of updates by Newton-Schulz products, for AMD Instinct MI355X (gfx950): what an
 * optimizer puts in a matrix's gradient's (or momentum's) place before fp8bq_hyperball_step.
 *
 * For each matrix G [R, C] of a batch: X = G / (|G|_F + eps), then in every step
 *   A = X X^T,   X <- a X + (b A + c A^2) X     (R <= C; otherwise with X^T X from the right),
 * which takes each singular value s to a s + b s^3 + c s^5 and keeps the singular vectors.  The result is X in BF16.
 *
 * Accuracy.  X, A and the polynomial are held in 22 bits, and their products taken of these, sums in FP32: the result is off
 * by 2^-14 of its norm or less besides its own rounding to BF16, for matrices of full and of low rank, of equal singular
 * values and of a few rows alike, and however far |G| is below eps (up to twelve steps of 3.4445, -4.7750, 2.0315).
 * Until the last step singular values have to stay below 15.9, and in every step those of the polynomial b A + c A^2 below
 * 255 (16-bit floats hold no more); past that the result is not finite.  A matrix of zeros gives zeros; one with a NaN or
 * an infinity gives NaN in all of its places and leaves the others of the batch alone.
 *
 * Conventions, errors and stream order as in fp8bq.h, except that g and out need their element's alignment only and may
 * have any leading dimension >= C and any batch stride from (R - 1) ld + C on: one matrix behind the other, not between its
 * rows.  Deterministic.
 */
#ifndef FP8BQ_ORTHO_H_
#define FP8BQ_ORTHO_H_

#include "fp8bq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FP8BQ_MAX_ORTHO_STEPS 64

/*
 *   g    [B] matrices [R, C] (BF16 or FP32), row stride ldg, gstride elements from one to the next.
 *   coefficients  HOST memory, 3 steps doubles: a, b, c of each step (read during the call); finite.
 *   1 <= steps <= FP8BQ_MAX_ORTHO_STEPS;  eps > 0, finite.
 *   out  [B] matrices [R, C], BF16 (ldo, ostride).
 *   ws   at least fp8bq_orthogonalize_workspace_size(B, R, C) bytes (at most 20 an element of the matrices with both sides
 *        rounded up to 64, and the partial sums of a split contraction where few matrices leave the card idle).
 *   B <= 4096; R, C <= 2^20.
 */
size_t fp8bq_orthogonalize_workspace_size(int64_t B, int64_t R, int64_t C);
int fp8bq_orthogonalize(const void* g, fp8bq_in gt, int64_t B, int64_t R, int64_t C, int64_t ldg, int64_t gstride, int32_t steps,
                        const double* coefficients, double eps, void* out, int64_t ldo, int64_t ostride, void* ws,
                        size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BQ_ORTHO_H_ */
