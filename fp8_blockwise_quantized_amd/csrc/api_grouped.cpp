// C-ABI entry points declared in include/fp8bq_grouped.h: validate, plan, launch on the caller's stream.
#include <hip/hip_runtime.h>

#include "../../include/fp8bq_grouped.h"
#include "device.hpp"
#include "launch.hpp"
#include "plan.hpp"
#include "validate.hpp"

namespace fp8bq {

static int run_grouped(const GroupedArgs& g, void* ws, size_t ws_bytes, void* stream) {
  bool empty = false, zero = false;
  int st = validate_grouped(g, &empty, &zero);
  if (st != kOk || empty) return st;
  int cus = 0;
  if ((st = current_device(&cus)) != kOk) return st;
  hipStream_t s = (hipStream_t)stream;
  if (zero) {  // wgrad without tokens
    if (g.out_t == 2) return kOk;
    const int oes = g.out_t == 0 ? 2 : 4;
    return launched(launch_zero_fill(const_cast<void*>(g.out), g.E * g.N, g.K * oes, g.ldout * oes, s));
  }
  const GemmPlan plan = plan_grouped(g.op, g.E, g.T, g.N, g.K, cus, ws != nullptr);
  if (!plan.fits) return kErrShape;
  if ((st = check_grouped_workspace(g, ws, ws_bytes, plan.ws_gemm)) != kOk) return st;
  GemmDesc d;
  d.a = (const uint8_t*)g.qa;
  d.lda = g.ldqa;
  d.sa = (const float*)g.sa;
  d.ldsa = g.ldsa;
  d.sa_mstride = 1;
  d.b = (const uint8_t*)g.qb;
  d.ldb = g.ldqb;
  d.sb = (const float*)g.sb;
  d.c = const_cast<void*>(g.out);
  d.ldc = g.ldout;
  d.out_f32 = g.out_t;
  d.fa = g.fa;
  d.fb = g.fb;
  d.M = g.op == kOpWgrad ? g.N : g.T;
  d.N = g.op == kOpFprop ? g.N : g.K;
  d.K = g.op == kOpFprop ? g.K : g.op == kOpDgrad ? g.N : g.T;
  d.sb_mode = g.op == kOpWgrad ? kSbColumn : kSbBlock128;
  d.sb_kstride = g.op == kOpFprop ? 1 : g.ldsb;  // fprop: sw[nb * ldsw + kb]; dgrad: sw[nb * ldsw + k / 128]
  d.sb_nstride = g.op == kOpFprop ? g.ldsb : g.op == kOpDgrad ? 1 : 0;
  const double rows_b = g.op == kOpWgrad ? (double)g.K : (double)g.E * (double)d.N;
  const double out = (g.op == kOpWgrad ? (double)g.E : 1.0) * (double)d.M * (double)d.N * (g.out_t == 0 ? 2 : 4);
  d.past = stores_past_caches(g.out_t, out, ((double)d.M + rows_b) * (double)d.K,
                              g.op != kOpWgrad && d.ldc * (g.out_t == 0 ? 2 : 4) % 8192 == 0);
  return launched(launch_grouped_gemm(g.op, d, GroupDesc{(const int64_t*)g.offsets, (int)g.E, g.T, plan.ws_gemm ? ws : nullptr}, plan,
                                      s));
}

}  // namespace fp8bq

using namespace fp8bq;

extern "C" {

int64_t fp8bq_grouped_padded_rows(int64_t T, int64_t E) {
  if (T < 0 || T >= ((int64_t)1 << 30) || E < 1 || E > kMaxGroupExperts) return 0;
  return grouped_padded_rows(T, E);
}

int fp8bq_quantize_act_grouped(const void* x, fp8bq_in xt, int64_t T, int64_t C, int64_t ldx, const int64_t* offsets,
                               int64_t E, fp8bq_fp8 fmt_rows, uint8_t* q, int64_t ldq, float* s, int64_t lds,
                               fp8bq_fp8 fmt_cols, uint8_t* qt, int64_t ldqt, float* st_, int64_t ldst,
                               int64_t padded, void* stream) {
  static_assert(FP8BQ_MAX_EXPERTS == kMaxGroupExperts, "expert limit of the header and the kernels");
  const int64_t needed = fp8bq_grouped_padded_rows(T, E);
  bool empty = false;
  int st = validate_quant_grouped(x, (int)xt, T, C, ldx, offsets, E, (int)fmt_rows, q, ldq, s, lds, (int)fmt_cols, qt,
                                  ldqt, st_, ldst, padded, needed, &empty);
  if (st != kOk || empty) return st;
  int cus = 0;
  if ((st = current_device(&cus)) != kOk) return st;
  return launched(launch_quant_grouped(x, (int)xt, T, C, ldx, offsets, (int)E, (int)fmt_rows, q, ldq, s, lds,
                                       (int)fmt_cols, qt, ldqt, st_, ldst, padded, cus, (hipStream_t)stream));
}

int fp8bq_grouped_gemm_fprop(int64_t E, int64_t T, int64_t N, int64_t K, const int64_t* offsets, const uint8_t* qx,
                             int64_t ldqx, const float* sx, int64_t ldsx, fp8bq_fp8 fx, const uint8_t* qw,
                             int64_t ldqw, const float* sw, int64_t ldsw, fp8bq_fp8 fw, void* y, fp8bq_out yt,
                             int64_t ldy, void* stream) {
  return run_grouped(GroupedArgs{kOpFprop, E, T, N, K, offsets, qx, ldqx, sx, ldsx, (int)fx, qw, ldqw, sw, ldsw,
                                 (int)fw, y, (int)yt, ldy},
                     nullptr, 0, stream);
}

int fp8bq_grouped_gemm_dgrad(int64_t E, int64_t T, int64_t N, int64_t K, const int64_t* offsets, const uint8_t* qdy,
                             int64_t ldqdy, const float* sdy, int64_t ldsdy, fp8bq_fp8 fdy, const uint8_t* qwt,
                             int64_t ldqwt, const float* sw, int64_t ldsw, fp8bq_fp8 fw, void* dx, fp8bq_out dxt,
                             int64_t lddx, void* stream) {
  return run_grouped(GroupedArgs{kOpDgrad, E, T, N, K, offsets, qdy, ldqdy, sdy, ldsdy, (int)fdy, qwt, ldqwt, sw, ldsw,
                                 (int)fw, dx, (int)dxt, lddx},
                     nullptr, 0, stream);
}

int fp8bq_grouped_gemm_wgrad(int64_t E, int64_t padded, int64_t N, int64_t K, const int64_t* offsets,
                             const uint8_t* qdyt, int64_t ldqdyt, const float* sdyt, int64_t ldsdyt, fp8bq_fp8 fdy,
                             const uint8_t* qxt, int64_t ldqxt, const float* sxt, int64_t ldsxt, fp8bq_fp8 fx,
                             void* dw, fp8bq_out dwt, int64_t lddw, void* ws, size_t ws_bytes, void* stream) {
  return run_grouped(GroupedArgs{kOpWgrad, E, padded, N, K, offsets, qdyt, ldqdyt, sdyt, ldsdyt, (int)fdy, qxt, ldqxt,
                                 sxt, ldsxt, (int)fx, dw, (int)dwt, lddw},
                     ws, ws_bytes, stream);
}

size_t fp8bq_grouped_gemm_wgrad_workspace_size(int64_t E, int64_t padded, int64_t N, int64_t K) {
  const GroupedArgs g{kOpWgrad, E, padded, N, K};
  bool empty = false, zero = false;
  if (validate_grouped(g, &empty, &zero) != kErrNull || padded == 0) return 0;  // (sizes alone: no output pointer)
  int cus = 0;
  if (current_device(&cus) != kOk) cus = 0;
  const GemmPlan p = plan_grouped(kOpWgrad, E, padded, N, K, cus);
  return p.fits ? p.ws_gemm : 0;
}

}  // extern "C"
