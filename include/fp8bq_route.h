/*
 * fp8bq_route.h -- routing of tokens to experts and the rows that go with it, for AMD Instinct MI355X (gfx950): what
 * stands before and behind the products of fp8bq_grouped.h, fp8bq_mx.h and fp8bq_int8.h.
 *
 *   fp8bq_route_experts            logits [T, E] -> experts [T, k] and weights [T, k]
 *   fp8bq_route_experts_backward   the weights' gradient -> the logits'
 *   fp8bq_expert_rows              experts [T, k] -> offsets [E + 1], the row of each choice, the choice of each row
 *   fp8bq_gather_rows              x [T, H] -> rows [T k, H] sorted by expert (its gradient is fp8bq_combine_rows)
 *   fp8bq_combine_rows             y [T k, H] -> sums [T, H] over each token's choices
 *   fp8bq_combine_rows_backward    the sums' gradient -> y's and the weights'
 *
 * Conventions, errors and stream order as in fp8bq.h.  experts, rows, slots, weights, bias and offsets are contiguous;
 * their addresses are multiples of their element's size.  Logits may have any leading dimension and their element's
 * alignment.  Inputs need not be finite here.  1 <= E <= FP8BQ_MAX_EXPERTS, 1 <= k <= FP8BQ_MAX_CHOICES and T k < 2^31.
 * T == 0 (or H == 0) is a successful no-op, except that fp8bq_expert_rows then writes offsets of zero.  (So dweights of
 * rows without elements, whose sums are zero, are the caller's to clear.)
 * Everything is deterministic: sums run in a fixed order, ties go to the lowest index.
 */
#ifndef FP8BQ_ROUTE_H_
#define FP8BQ_ROUTE_H_

#include "fp8bq.h"
#include "fp8bq_grouped.h" /* FP8BQ_MAX_EXPERTS, the meaning of offsets */

#ifdef __cplusplus
extern "C" {
#endif

#define FP8BQ_MAX_CHOICES 64
#define FP8BQ_MAX_EXPERT_GROUPS 64

typedef enum { FP8BQ_SCORE_SOFTMAX = 0, FP8BQ_SCORE_SIGMOID = 1 } fp8bq_score;

/*
 * A token's experts.  s = softmax or sigmoid of its logits, c = s + bias.  The experts form `groups` groups of E / groups
 * neighbours; a group scores the sum of its best group_best (1 or 2) c, and the top_groups groups with the largest
 * scores stay.  Of their experts the k with the largest c are chosen, largest first.
 * weight = scale s, or with renormalize scale s / (sum of the chosen s), zero where that sum is zero.
 *   Scores and sums are computed in 64 bits.  c and groups' scores that agree in their first 43 bits count as equal, and
 *   the lower index comes first.  Without a bias and with group_best 1 the logits themselves are compared.
 *   A logit of -infinity has the score zero (a switched-off expert, chosen only when nothing else is left); a row of
 *   nothing else gives weights of zero.  A NaN is chosen like -infinity; with softmax, a NaN or +infinity makes the row's
 *   weights NaN where they depend on it.  The chosen experts are always k different indices.
 *   bias NULL or [E].  groups divides E, groups <= FP8BQ_MAX_EXPERT_GROUPS, k <= top_groups E / groups,
 *   group_best <= E / groups; scale finite.  (With groups == top_groups every group stays.)
 */
int fp8bq_route_experts(const void* logits, fp8bq_in xt, int64_t T, int64_t E, int64_t ldx, int64_t k, fp8bq_score score,
                        const float* bias, int64_t groups, int64_t top_groups, int64_t group_best, int renormalize,
                        double scale, int32_t* experts, float* weights, void* stream);

/*
 * dlogits [T, E] (of the logits' type, row stride lddx) from dweights [T, k], for the experts that were chosen with the
 * same score, renormalize and scale.  The choice itself (and with it the bias) has no gradient.  Experts outside
 * 0 .. E-1 are passed over; a token's experts have to differ.
 */
int fp8bq_route_experts_backward(const float* dweights, const void* logits, fp8bq_in xt, int64_t T, int64_t E, int64_t ldx,
                                 int64_t k, fp8bq_score score, int renormalize, double scale, const int32_t* experts,
                                 void* dlogits, int64_t lddx, void* stream);

/*
 * The stable sort of the n choices experts[i] by expert (choice i = t k + j is token t's j-th); choices outside
 * 0 .. E-1 (a dropped choice, a padded token: -1) have no row.
 *   offsets [E + 1]  expert e has the rows offsets[e] .. offsets[e+1]-1.
 *   rows [n]   row of choice i, or -1.        slots [n]  choice of row r, or -1 from offsets[E] on.
 *   ws  at least fp8bq_expert_rows_workspace_size(n, E) bytes (may be NULL when that is 0).
 */
size_t fp8bq_expert_rows_workspace_size(int64_t n, int64_t E);
int fp8bq_expert_rows(const int32_t* experts, int64_t n, int64_t E, int64_t* offsets, int32_t* rows, int32_t* slots, void* ws,
                      size_t ws_bytes, void* stream);

/* out[r] = x[slots[r] / k] for the T k rows r, zeros where slots[r] is negative (or past the tokens).  H % 8 == 0;
 * out has x's type. */
int fp8bq_gather_rows(const void* x, fp8bq_in xt, int64_t T, int64_t H, int64_t ldx, const int32_t* slots, int64_t k,
                      void* out, int64_t ldo, void* stream);

/* out[t] = sum_j weights[t, j] y[rows[t, j]] over the choices that have a row, in FP32 in the order of j; weights NULL:
 * ones.  y [T k, H] and out [T, H] BF16 or FP32 each; H % 8 == 0. */
int fp8bq_combine_rows(const void* y, fp8bq_in yt, int64_t T, int64_t k, int64_t H, int64_t ldy, const int32_t* rows,
                       const float* weights, void* out, fp8bq_out ot, int64_t ldo, void* stream);

/* dy[rows[t, j]] = weights[t, j] dout[t] (of y's type; zeros in rows r with slots[r] < 0) and
 * dweights[t, j] = sum_h dout[t, h] y[rows[t, j], h] (zero for choices without a row). */
int fp8bq_combine_rows_backward(const void* dout, fp8bq_in dt, int64_t lddo, const void* y, fp8bq_in yt, int64_t ldy,
                                int64_t T, int64_t k, int64_t H, const int32_t* rows, const float* weights,
                                const int32_t* slots, void* dy, int64_t lddy, float* dweights, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BQ_ROUTE_H_ */
