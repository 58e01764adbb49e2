// C-ABI entry points declared in include/fp8bq_int8.h: validate, plan, launch on the caller's stream.
#include <hip/hip_runtime.h>

#include "../../include/fp8bq_int8.h"
#include "device.hpp"
#include "launch.hpp"
#include "plan.hpp"
#include "validate.hpp"

namespace fp8bq {

static int cus_or_default() {
  int cus = 0;
  return current_device(&cus) == kOk && cus > 0 ? cus : 256;
}

// Workspace of a product on x itself: x's codes and scales, then the product's own.
struct Int8Space {
  size_t codes, scales, product;
  size_t total() const { return codes + scales + product; }
};
static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
static Int8Space int8_space(const MxPlan& p, bool linear, int64_t M, int64_t K) {
  Int8Space s{0, 0, p.ws};
  if (linear && !p.fused) {
    s.codes = up256((size_t)M * (size_t)K);
    s.scales = up256((size_t)M * 4);
  }
  return s;
}
static size_t int8_ws_size(bool linear, int64_t E, int64_t M, int64_t N, int64_t K) {
  MxArgs g{};
  g.E = E;
  g.M = M;
  g.N = N;
  g.K = K;
  bool empty = false, zero = false;
  // (a size that is refused ends in the shape check; sizes that pass end at the missing output)
  if (K == 0 || validate_int8(g, &empty, &zero) != kErrNull) return 0;
  return int8_space(plan_int8(linear, E, M, N, K, cus_or_default()), linear, M, K).total();
}

static int run_int8(const MxArgs& g, void* ws, size_t ws_bytes, void* stream) {
  bool empty = false, zero = false;
  int st = validate_int8(g, &empty, &zero);
  if (st != kOk || empty) return st;
  const bool linear = g.a_type != kMxCodes;
  const MxPlan plan = zero ? MxPlan{} : plan_int8(linear, g.E, g.M, g.N, g.K, cus_or_default());
  const Int8Space space = zero ? Int8Space{0, 0, 0} : int8_space(plan, linear, g.M, g.K);
  if ((st = check_int8_workspace(g, ws, ws_bytes, space.total())) != kOk) return st;
  if ((st = current_device(nullptr)) != kOk) return st;
  hipStream_t s = (hipStream_t)stream;
  const int oes = g.out_t == 0 ? 2 : 4;
  if (zero) {
    if (g.out_t == 2) return kOk;
    return launched(launch_zero_fill(const_cast<void*>(g.out), g.M, g.N * oes, g.ldout * oes, s));
  }
  Int8Desc d;
  d.a = g.a;
  d.lda = g.lda;
  d.sa = (const float*)g.sa;
  d.a_type = g.a_type;
  d.b = (const uint8_t*)g.b;
  d.ldb = g.ldb;
  d.sb = (const float*)g.sb;
  d.c = const_cast<void*>(g.out);
  d.ldc = g.ldout;
  d.out_t = g.out_t;
  d.M = g.M;
  d.N = g.N;
  d.K = g.K;
  d.past = stores_past_caches(g.out_t, (double)g.M * (double)g.N * oes,
                              ((double)g.M + (g.E ? (double)g.E : 1.0) * (double)g.N) * (double)g.K,
                              g.ldout * oes % 8192 == 0);
  if (linear && !plan.fused) {
    uint8_t* q = (uint8_t*)ws;
    float* sc = (float*)((uint8_t*)ws + space.codes);
    if (launch_int8_rows(g.a, g.a_type, g.M, g.K, g.lda, q, g.K, sc, s) != hipSuccess) return kErrLaunch;
    d.a = q;
    d.lda = g.K;
    d.sa = sc;
    d.a_type = kMxCodes;
  }
  const MxGroups grp{(const int64_t*)g.offsets, (int)g.E};
  if (plan.skinny) return launched(launch_int8_skinny(d, grp, plan, s));
  return launched(launch_int8_gemm(d, grp, plan, (uint8_t*)ws + space.codes + space.scales, s));
}

}  // namespace fp8bq

using namespace fp8bq;

extern "C" {

int fp8bq_quantize_int8(const void* x, fp8bq_in xt, int64_t R, int64_t C, int64_t ldx, int8_t* q, int64_t ldq, float* s,
                        void* stream) {
  bool empty = false;
  int st = validate_int8_quant(x, (int)xt, R, C, ldx, false, q, ldq, s, nullptr, 0, 0, &empty);
  if (st != kOk || empty) return st;
  if ((st = current_device(nullptr)) != kOk) return st;
  return launched(launch_int8_rows(x, (int)xt, R, C, ldx, (uint8_t*)q, ldq, s, (hipStream_t)stream));
}

size_t fp8bq_quantize_int8_t_workspace_size(int64_t R, int64_t C) {
  return R < 1 || C < 1 || R >= ((int64_t)1 << 30) || C >= ((int64_t)1 << 30)
             ? 0
             : (size_t)int8_col_chunks(R, C) * (size_t)C * sizeof(float);
}

int fp8bq_quantize_int8_t(const void* x, fp8bq_in xt, int64_t R, int64_t C, int64_t ldx, int8_t* qt, int64_t ldqt,
                          float* st_, void* ws, size_t ws_bytes, void* stream) {
  bool empty = false;
  int st = validate_int8_quant(x, (int)xt, R, C, ldx, true, qt, ldqt, st_, ws, ws_bytes,
                               fp8bq_quantize_int8_t_workspace_size(R, C), &empty);
  if (st != kOk || empty) return st;
  if ((st = current_device(nullptr)) != kOk) return st;
  return launched(launch_int8_cols(x, (int)xt, R, C, ldx, (uint8_t*)qt, ldqt, st_, ws, (hipStream_t)stream));
}

size_t fp8bq_gemm_int8_workspace_size(int64_t M, int64_t N, int64_t K) { return int8_ws_size(false, 0, M, N, K); }
size_t fp8bq_linear_int8_workspace_size(int64_t M, int64_t N, int64_t K) { return int8_ws_size(true, 0, M, N, K); }
size_t fp8bq_grouped_gemm_int8_workspace_size(int64_t E, int64_t T, int64_t N, int64_t K) {
  return E < 1 ? 0 : int8_ws_size(false, E, T, N, K);
}
size_t fp8bq_grouped_linear_int8_workspace_size(int64_t E, int64_t T, int64_t N, int64_t K) {
  return E < 1 ? 0 : int8_ws_size(true, E, T, N, K);
}

int fp8bq_gemm_int8(int64_t M, int64_t N, int64_t K, const int8_t* qa, int64_t ldqa, const float* sa, const int8_t* qb,
                    int64_t ldqb, const float* sb, void* c, fp8bq_out ct, int64_t ldc, void* ws, size_t ws_bytes,
                    void* stream) {
  return run_int8(MxArgs{0, M, N, K, nullptr, kMxCodes, qa, ldqa, sa, 0, qb, ldqb, sb, 0, c, (int)ct, ldc}, ws, ws_bytes,
                  stream);
}

int fp8bq_linear_int8(int64_t M, int64_t N, int64_t K, const void* x, fp8bq_in xt, int64_t ldx, const int8_t* qw,
                      int64_t ldqw, const float* sw, void* y, fp8bq_out yt, int64_t ldy, void* ws, size_t ws_bytes,
                      void* stream) {
  if (xt != FP8BQ_IN_BF16 && xt != FP8BQ_IN_F32) return kErrDtype;
  return run_int8(MxArgs{0, M, N, K, nullptr, (int)xt, x, ldx, nullptr, 0, qw, ldqw, sw, 0, y, (int)yt, ldy}, ws,
                  ws_bytes, stream);
}

int fp8bq_grouped_gemm_int8(int64_t E, int64_t T, int64_t N, int64_t K, const int64_t* offsets, const int8_t* qa,
                            int64_t ldqa, const float* sa, const int8_t* qw, int64_t ldqw, const float* sw, void* y,
                            fp8bq_out yt, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
  if (E < 1) return kErrShape;
  return run_int8(MxArgs{E, T, N, K, offsets, kMxCodes, qa, ldqa, sa, 0, qw, ldqw, sw, 0, y, (int)yt, ldy}, ws, ws_bytes,
                  stream);
}

int fp8bq_grouped_linear_int8(int64_t E, int64_t T, int64_t N, int64_t K, const int64_t* offsets, const void* x,
                              fp8bq_in xt, int64_t ldx, const int8_t* qw, int64_t ldqw, const float* sw, void* y,
                              fp8bq_out yt, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
  if (E < 1) return kErrShape;
  if (xt != FP8BQ_IN_BF16 && xt != FP8BQ_IN_F32) return kErrDtype;
  return run_int8(MxArgs{E, T, N, K, offsets, (int)xt, x, ldx, nullptr, 0, qw, ldqw, sw, 0, y, (int)yt, ldy}, ws,
                  ws_bytes, stream);
}

}  // extern "C"
