// C-ABI entry points declared in include/fp8bq_mx.h: validate, plan, launch on the caller's stream.
#include <hip/hip_runtime.h>

#include "../../include/fp8bq_mx.h"
#include "device.hpp"
#include "launch.hpp"
#include "plan.hpp"
#include "validate.hpp"

namespace fp8bq {

static int cus_or_default() {
  int cus = 0;
  return current_device(&cus) == kOk && cus > 0 ? cus : 256;
}

static bool mx_sizes_ok(int64_t E, int64_t M, int64_t N, int64_t K) {
  MxArgs g{};
  g.E = E;
  g.M = M;
  g.N = N;
  g.K = K;
  bool empty = false, zero = false;
  // (a size that is refused ends in the shape check; sizes that pass end at the missing output)
  return validate_mx(g, &empty, &zero) == kErrNull;
}

// Workspace of a product on x itself: x's codes and scale words, then the product's own.
struct MxSpace {
  size_t codes, scales, product;
  size_t total() const { return codes + scales + product; }
};
static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
static MxSpace mx_space(const MxPlan& p, bool linear, int64_t M, int64_t K) {
  MxSpace s{0, 0, p.ws};
  if (linear && !p.fused) {
    s.codes = up256((size_t)M * (size_t)(K / 2));
    s.scales = up256((size_t)((K + 127) / 128) * (size_t)M * 4);
  }
  return s;
}
static size_t mx_ws_size(bool linear, int64_t E, int64_t M, int64_t N, int64_t K) {
  if (K == 0 || !mx_sizes_ok(E, M, N, K)) return 0;
  return mx_space(plan_mx(linear, E, M, N, K, cus_or_default()), linear, M, K).total();
}

static int run_mx(const MxArgs& g, void* ws, size_t ws_bytes, void* stream) {
  bool empty = false, zero = false;
  int st = validate_mx(g, &empty, &zero);
  if (st != kOk || empty) return st;
  const bool linear = g.a_type != kMxCodes;
  const MxPlan plan = zero ? MxPlan{} : plan_mx(linear, g.E, g.M, g.N, g.K, cus_or_default());
  const MxSpace space = zero ? MxSpace{0, 0, 0} : mx_space(plan, linear, g.M, g.K);
  if ((st = check_workspace(g, ws, ws_bytes, space.total())) != kOk) return st;
  if ((st = current_device(nullptr)) != kOk) return st;
  hipStream_t s = (hipStream_t)stream;
  if (zero) {
    if (g.out_t == 2) return kOk;
    const int oes = g.out_t == 0 ? 2 : 4;
    return launched(launch_zero_fill(const_cast<void*>(g.out), g.M, g.N * oes, g.ldout * oes, s));
  }
  MxDesc d;
  d.a = g.a;
  d.lda = g.lda;
  d.sa = (const uint32_t*)g.sa;
  d.ldsa = g.ldsa;
  d.a_type = g.a_type;
  d.b = (const uint8_t*)g.b;
  d.ldb = g.ldb;
  d.sb = (const uint32_t*)g.sb;
  d.ldsb = g.ldsb;
  d.c = const_cast<void*>(g.out);
  d.ldc = g.ldout;
  d.out_t = g.out_t;
  d.M = g.M;
  d.N = g.N;
  d.K = g.K;
  d.past = stores_past_caches(g.out_t, (double)g.M * (double)g.N * (g.out_t == 0 ? 2 : 4),
                              ((double)g.M + (g.E ? (double)g.E : 1.0) * (double)g.N) * (double)g.K * 0.53,
                              g.ldout * (g.out_t == 0 ? 2 : 4) % 16384 == 0);
  if (linear && !plan.fused) {
    uint8_t* q = (uint8_t*)ws;
    uint32_t* sc = (uint32_t*)((uint8_t*)ws + space.codes);
    if (launch_mx_quant(g.a, g.a_type, g.M, g.K, g.lda, q, g.K / 2, sc, g.M, nullptr, 0, nullptr, 0, s) != hipSuccess)
      return kErrLaunch;
    d.a = q;
    d.lda = g.K / 2;
    d.sa = sc;
    d.ldsa = g.M;
    d.a_type = kMxCodes;
  }
  const MxGroups grp{(const int64_t*)g.offsets, (int)g.E};
  if (plan.skinny) return launched(launch_mx_skinny(d, grp, plan, s));
  return launched(launch_mx_gemm(d, grp, plan, (uint8_t*)ws + space.codes + space.scales, s));
}

}  // namespace fp8bq

using namespace fp8bq;

extern "C" {

int fp8bq_quantize_mxfp4(const void* x, fp8bq_in xt, int64_t R, int64_t C, int64_t ldx, uint8_t* q, int64_t ldq,
                         uint32_t* s, int64_t lds, uint8_t* qt, int64_t ldqt, uint32_t* st_, int64_t ldst,
                         void* stream) {
  bool empty = false;
  int st = validate_mx_quant(x, (int)xt, R, C, ldx, q, ldq, s, lds, qt, ldqt, st_, ldst, &empty);
  if (st != kOk || empty) return st;
  if ((st = current_device(nullptr)) != kOk) return st;
  return launched(launch_mx_quant(x, (int)xt, R, C, ldx, q, ldq, s, lds, qt, ldqt, st_, ldst, (hipStream_t)stream));
}

size_t fp8bq_gemm_mxfp4_workspace_size(int64_t M, int64_t N, int64_t K) { return mx_ws_size(false, 0, M, N, K); }
size_t fp8bq_linear_mxfp4_workspace_size(int64_t M, int64_t N, int64_t K) { return mx_ws_size(true, 0, M, N, K); }
size_t fp8bq_grouped_gemm_mxfp4_workspace_size(int64_t E, int64_t T, int64_t N, int64_t K) {
  return E < 1 ? 0 : mx_ws_size(false, E, T, N, K);
}
size_t fp8bq_grouped_linear_mxfp4_workspace_size(int64_t E, int64_t T, int64_t N, int64_t K) {
  return E < 1 ? 0 : mx_ws_size(true, E, T, N, K);
}

int fp8bq_gemm_mxfp4(int64_t M, int64_t N, int64_t K, const uint8_t* qa, int64_t ldqa, const uint32_t* sa,
                     int64_t ldsa, const uint8_t* qb, int64_t ldqb, const uint32_t* sb, int64_t ldsb, void* c,
                     fp8bq_out ct, int64_t ldc, void* ws, size_t ws_bytes, void* stream) {
  return run_mx(MxArgs{0, M, N, K, nullptr, kMxCodes, qa, ldqa, sa, ldsa, qb, ldqb, sb, ldsb, c, (int)ct, ldc}, ws,
                ws_bytes, stream);
}

int fp8bq_linear_mxfp4(int64_t M, int64_t N, int64_t K, const void* x, fp8bq_in xt, int64_t ldx, const uint8_t* qw,
                       int64_t ldqw, const uint32_t* sw, int64_t ldsw, void* y, fp8bq_out yt, int64_t ldy, void* ws,
                       size_t ws_bytes, void* stream) {
  if (xt != FP8BQ_IN_BF16 && xt != FP8BQ_IN_F32) return kErrDtype;
  return run_mx(MxArgs{0, M, N, K, nullptr, (int)xt, x, ldx, nullptr, 0, qw, ldqw, sw, ldsw, y, (int)yt, ldy}, ws,
                ws_bytes, stream);
}

int fp8bq_grouped_gemm_mxfp4(int64_t E, int64_t T, int64_t N, int64_t K, const int64_t* offsets, const uint8_t* qa,
                             int64_t ldqa, const uint32_t* sa, int64_t ldsa, const uint8_t* qw, int64_t ldqw,
                             const uint32_t* sw, int64_t ldsw, void* y, fp8bq_out yt, int64_t ldy, void* ws,
                             size_t ws_bytes, void* stream) {
  if (E < 1) return kErrShape;
  return run_mx(MxArgs{E, T, N, K, offsets, kMxCodes, qa, ldqa, sa, ldsa, qw, ldqw, sw, ldsw, y, (int)yt, ldy}, ws,
                ws_bytes, stream);
}

int fp8bq_grouped_linear_mxfp4(int64_t E, int64_t T, int64_t N, int64_t K, const int64_t* offsets, const void* x,
                               fp8bq_in xt, int64_t ldx, const uint8_t* qw, int64_t ldqw, const uint32_t* sw,
                               int64_t ldsw, void* y, fp8bq_out yt, int64_t ldy, void* ws, size_t ws_bytes,
                               void* stream) {
  if (E < 1) return kErrShape;
  if (xt != FP8BQ_IN_BF16 && xt != FP8BQ_IN_F32) return kErrDtype;
  return run_mx(MxArgs{E, T, N, K, offsets, (int)xt, x, ldx, nullptr, 0, qw, ldqw, sw, ldsw, y, (int)yt, ldy}, ws,
                ws_bytes, stream);
}

}  // extern "C"
