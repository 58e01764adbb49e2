/*
 * fp8bq_grouped.h -- the FP8 blockwise linear layer grouped by expert (mixture of experts), with ragged
 * token counts, for AMD Instinct MI355X (gfx950).
 *
 * The tokens are sorted by expert.  offsets [E + 1] (int64, DEVICE memory) holds where each expert's begin:
 * expert e has the rows offsets[e] .. offsets[e+1]-1 of the token matrices, possibly none.  The experts'
 * weights are stacked, W [E N, K]: expert e has the rows e N .. e N + N-1, so one call of
 * fp8bq_quantize_weight_128x128 or fp8bq_quantize_weight_dual quantizes all of them.  Per expert e:
 *   fprop  Y_e [n_e, N] = X_e [n_e, K] . W_e [N, K]^T
 *   dgrad  dX_e [n_e, K] = dY_e [n_e, N] . W_e [N, K]
 *   wgrad  dW_e [N, K] = dY_e^T . X_e    (zero for an expert without tokens)
 * with the quantization rule, scale layouts, accumulation and output types of fp8bq.h.
 *
 * The counts stay on the device: no call reads offsets on the host or waits for it.  The kernels make the
 * offsets safe themselves (each is taken as at least the one before it and at most the rows that the call
 * knows: T, for wgrad the padded ones), so no content of that buffer leads to an access outside the
 * matrices; offsets that do not ascend, or lie past T, give unspecified values.  offsets[0] > 0 or offsets[E] < T is allowed: rows outside every expert are not read, and their
 * output rows are left as they are (a token buffer may be larger than the step's tokens).
 *
 * Conventions, alignment, errors and stream order as in fp8bq.h; offsets is 8-byte aligned.
 * 1 <= E <= FP8BQ_MAX_EXPERTS; T, E N and E K are below 2^30.  T == 0 (or a zero width) is a successful no-op,
 * except that wgrad then writes zeros.
 */
#ifndef FP8BQ_GROUPED_H_
#define FP8BQ_GROUPED_H_

#include "fp8bq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FP8BQ_MAX_EXPERTS 512

/* Rows that hold T tokens with every expert's padded to a multiple of 128, whatever their shares: the token
 * extent of wgrad's operands (a multiple of 128; 0 for arguments out of range). */
int64_t fp8bq_grouped_padded_rows(int64_t T, int64_t E);

/*
 * Token-axis quantizer of wgrad's operands: groups of 128 tokens that begin anew at each expert.  In the
 * outputs expert e's tokens begin at P_e, P_0 = 0, P_{e+1} = P_e + 128 ceil(n_e / 128); the codes between
 * the expert's last token and P_{e+1} are zeros.
 *   x   [T, C] input (BF16 or FP32), row stride ldx; C % 128 == 0.
 *   qt  [C, padded] codes, transposed: token i of expert e, column c is qt[c * ldqt + P_e + i].
 *   st  [padded / 128][C] scales (ldst >= C): one for each 128-token block and column.
 *   padded  at least fp8bq_grouped_padded_rows(T, E), a multiple of 128.  Columns of qt from P_E on are not
 *       written (and never read by wgrad).
 *   q, s  NULL, or the outputs of fp8bq_quantize_act_1x128(x, fmt_rows) from the same read, bit for bit, for
 *       the rows that belong to an expert (fmt_rows is ignored when they are NULL).
 */
int fp8bq_quantize_act_grouped(const void* x, fp8bq_in xt, int64_t T, int64_t C, int64_t ldx, const int64_t* offsets,
                               int64_t E, fp8bq_fp8 fmt_rows, uint8_t* q, int64_t ldq, float* s, int64_t lds,
                               fp8bq_fp8 fmt_cols, uint8_t* qt, int64_t ldqt, float* st, int64_t ldst,
                               int64_t padded, void* stream);

/*
 * Y [T, N] = X_e . W_e^T for the rows of every expert e.
 *   qx/sx  from fp8bq_quantize_act_1x128(X [T, K]).
 *   qw/sw  from fp8bq_quantize_weight_128x128(W [E N, K]): qw [E N, K], sw [E N / 128][K / 128].
 *   y      [T, N] of type yt (BF16 or FP32), row stride ldy.   N % 128 == 0; K % 128 == 0, K >= 128.
 */
int fp8bq_grouped_gemm_fprop(int64_t E, int64_t T, int64_t N, int64_t K, const int64_t* offsets, const uint8_t* qx,
                             int64_t ldqx, const float* sx, int64_t ldsx, fp8bq_fp8 fx, const uint8_t* qw,
                             int64_t ldqw, const float* sw, int64_t ldsw, fp8bq_fp8 fw, void* y, fp8bq_out yt,
                             int64_t ldy, void* stream);

/*
 * dX [T, K] = dY_e . W_e for the rows of every expert e.
 *   qdy/sdy  from fp8bq_quantize_act_1x128(dY [T, N]) or the row outputs of fp8bq_quantize_act_grouped.
 *   qwt      [K, E N]: the transposed codes of fp8bq_quantize_weight_dual(W [E N, K]); sw as for fprop.
 *   dx       [T, K] of type dxt (BF16 or FP32), row stride lddx.   N % 128 == 0, N >= 128; K % 128 == 0.
 */
int fp8bq_grouped_gemm_dgrad(int64_t E, int64_t T, int64_t N, int64_t K, const int64_t* offsets, const uint8_t* qdy,
                             int64_t ldqdy, const float* sdy, int64_t ldsdy, fp8bq_fp8 fdy, const uint8_t* qwt,
                             int64_t ldqwt, const float* sw, int64_t ldsw, fp8bq_fp8 fw, void* dx, fp8bq_out dxt,
                             int64_t lddx, void* stream);

/*
 * dW [E N, K] = dY_e^T . X_e for every expert e.
 *   qdyt/sdyt  from fp8bq_quantize_act_grouped(dY): qdyt [N, padded], sdyt [padded / 128][N].
 *   qxt/sxt    from fp8bq_quantize_act_grouped(X):  qxt [K, padded],  sxt [padded / 128][K].
 *   dw         [E N, K] of type dwt (BF16, FP32, or FP32 accumulated into), row stride lddw.  An expert
 *              without tokens gets zeros, or keeps its values when accumulating.
 *   ws         NULL, or at least fp8bq_grouped_gemm_wgrad_workspace_size(E, padded, N, K) bytes, 16-byte aligned.
 *              With it the contraction of experts with many more tokens than the others is split over several
 *              workgroups (FP32 partial sums, added in a fixed order); without it no expert's is.
 */
size_t fp8bq_grouped_gemm_wgrad_workspace_size(int64_t E, int64_t padded, int64_t N, int64_t K);
int fp8bq_grouped_gemm_wgrad(int64_t E, int64_t padded, int64_t N, int64_t K, const int64_t* offsets,
                             const uint8_t* qdyt, int64_t ldqdyt, const float* sdyt, int64_t ldsdyt, fp8bq_fp8 fdy,
                             const uint8_t* qxt, int64_t ldqxt, const float* sxt, int64_t ldsxt, fp8bq_fp8 fx,
                             void* dw, fp8bq_out dwt, int64_t lddw, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BQ_GROUPED_H_ */
