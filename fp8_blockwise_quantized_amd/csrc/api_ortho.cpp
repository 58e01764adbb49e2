// C-ABI entry points declared in include/fp8bq_ortho.h: validate, plan, launch on the caller's stream.
#include <hip/hip_runtime.h>

#include "../../include/fp8bq_ortho.h"
#include "device.hpp"
#include "launch.hpp"
#include "ortho_plan.hpp"
#include "validate.hpp"

using namespace fp8bq;

static_assert(FP8BQ_MAX_ORTHO_STEPS == kMaxOrthoSteps, "steps of a call");

static int cus_or_default() {
  int cus = 0;
  return current_device(&cus) == kOk && cus > 0 ? cus : 256;
}

extern "C" {

size_t fp8bq_orthogonalize_workspace_size(int64_t B, int64_t R, int64_t C) {
  if (B < 1 || R < 1 || C < 1 || B > kMaxOrthoBatch || R > kMaxOrthoSide || C > kMaxOrthoSide) return 0;
  bool fits = false;
  const OrthoPlan p = plan_ortho(B, R, C, cus_or_default(), &fits);
  return fits ? p.ws : 0;
}

int fp8bq_orthogonalize(const void* g, fp8bq_in gt, int64_t B, int64_t R, int64_t C, int64_t ldg, int64_t gstride, int32_t steps,
                        const double* coefficients, double eps, void* out, int64_t ldo, int64_t ostride, void* ws,
                        size_t ws_bytes, void* stream) {
  bool empty = false;
  const OrthoCheck c{g, (int)gt, B, R, C, ldg, gstride, steps, coefficients, eps, out, ldo, ostride};
  int st = validate_ortho(c, &empty);
  if (st != kOk || empty) return st;
  bool fits = false;
  const OrthoPlan p = plan_ortho(B, R, C, cus_or_default(), &fits);
  if (!fits) return kErrShape;
  if ((st = check_ortho_workspace(c, ws, ws_bytes, p.ws)) != kOk) return st;
  if ((st = current_device(nullptr)) != kOk) return st;
  return launched(launch_ortho(g, (int)gt, ldg, gstride, p, steps, coefficients, eps, out, ldo, ostride, ws, (hipStream_t)stream));
}

}  // extern "C"
