// C-ABI entry points declared in include/fp8bq_route.h: validate and launch on the caller's stream.
#include <hip/hip_runtime.h>

#include "../../include/fp8bq_route.h"
#include "device.hpp"
#include "launch.hpp"
#include "validate.hpp"

using namespace fp8bq;

static_assert(FP8BQ_MAX_EXPERTS == kMaxRouteExperts, "experts of a row");

extern "C" {

int fp8bq_route_experts(const void* logits, fp8bq_in xt, int64_t T, int64_t E, int64_t ldx, int64_t k, fp8bq_score score,
                        const float* bias, int64_t groups, int64_t top_groups, int64_t group_best, int renormalize,
                        double scale, int32_t* experts, float* weights, void* stream) {
  bool empty = false;
  int st = validate_route(RouteCheck{logits, (int)xt, T, E, ldx, k, (int)score, groups, top_groups, group_best, scale}, bias,
                          experts, weights, &empty);
  if (st != kOk || empty) return st;
  if ((st = current_device(nullptr)) != kOk) return st;
  const RouteHow how{(int)E, (int)k, (int)score, (int)groups, (int)top_groups, (int)group_best, renormalize != 0, scale};
  return launched(launch_route(logits, (int)xt, T, ldx, how, bias, experts, weights, (hipStream_t)stream));
}

int fp8bq_route_experts_backward(const float* dweights, const void* logits, fp8bq_in xt, int64_t T, int64_t E, int64_t ldx,
                                 int64_t k, fp8bq_score score, int renormalize, double scale, const int32_t* experts,
                                 void* dlogits, int64_t lddx, void* stream) {
  bool empty = false;
  int st = validate_route_backward(RouteCheck{logits, (int)xt, T, E, ldx, k, (int)score, 1, 1, 1, scale}, dweights, experts,
                                   dlogits, lddx, &empty);
  if (st != kOk || empty) return st;
  if ((st = current_device(nullptr)) != kOk) return st;
  const RouteHow how{(int)E, (int)k, (int)score, 1, 1, 1, renormalize != 0, scale};
  return launched(launch_route_backward(dweights, logits, (int)xt, T, ldx, how, experts, dlogits, lddx, (hipStream_t)stream));
}

size_t fp8bq_expert_rows_workspace_size(int64_t n, int64_t E) {
  if (n < 0 || n >= ((int64_t)1 << 31) || E < 1 || E > kMaxGroupExperts) return 0;
  const int chunks = expert_rows_chunks(n);
  return chunks > 1 ? (size_t)chunks * (size_t)E * sizeof(uint32_t) : 0;
}

int fp8bq_expert_rows(const int32_t* experts, int64_t n, int64_t E, int64_t* offsets, int32_t* rows, int32_t* slots, void* ws,
                      size_t ws_bytes, void* stream) {
  int st = validate_expert_rows(experts, n, E, offsets, rows, slots, ws, ws_bytes, fp8bq_expert_rows_workspace_size(n, E));
  if (st != kOk) return st;
  if ((st = current_device(nullptr)) != kOk) return st;
  return launched(launch_expert_rows(experts, n, (int)E, offsets, rows, slots, ws, (hipStream_t)stream));
}

int fp8bq_gather_rows(const void* x, fp8bq_in xt, int64_t T, int64_t H, int64_t ldx, const int32_t* slots, int64_t k,
                      void* out, int64_t ldo, void* stream) {
  bool empty = false;
  int st = validate_rows(RowsCheck{T, k, H, {x, nullptr}, {(int)xt, 0}, {ldx, 0}, {false, false}, out, (int)xt, ldo, true,
                                   {slots, nullptr, nullptr}, nullptr}, 1, 1, &empty);
  if (st != kOk || empty) return st;
  if ((st = current_device(nullptr)) != kOk) return st;
  return launched(launch_gather_rows(x, (int)xt, T, H, ldx, slots, k, out, ldo, (hipStream_t)stream));
}

int fp8bq_combine_rows(const void* y, fp8bq_in yt, int64_t T, int64_t k, int64_t H, int64_t ldy, const int32_t* rows,
                       const float* weights, void* out, fp8bq_out ot, int64_t ldo, void* stream) {
  bool empty = false;
  // (weights may be missing: the second of the vectors, checked where it is there)
  int st = validate_rows(RowsCheck{T, k, H, {y, nullptr}, {(int)yt, 0}, {ldy, 0}, {true, false}, out, (int)ot, ldo, false,
                                   {rows, weights, nullptr}, nullptr}, 1, weights ? 2 : 1, &empty);
  if (st != kOk || empty) return st;
  if ((st = current_device(nullptr)) != kOk) return st;
  return launched(launch_combine_rows(y, (int)yt, T, k, H, ldy, rows, weights, out, (int)ot, ldo, (hipStream_t)stream));
}

int fp8bq_combine_rows_backward(const void* dout, fp8bq_in dt, int64_t lddo, const void* y, fp8bq_in yt, int64_t ldy,
                                int64_t T, int64_t k, int64_t H, const int32_t* rows, const float* weights,
                                const int32_t* slots, void* dy, int64_t lddy, float* dweights, void* stream) {
  bool empty = false;
  if (dweights == nullptr && T > 0 && H > 0) return kErrNull;
  int st = validate_rows(RowsCheck{T, k, H, {dout, y}, {(int)dt, (int)yt}, {lddo, ldy}, {false, true}, dy, (int)yt, lddy, true,
                                   {rows, weights, slots}, dweights}, 2, 3, &empty);
  if (st != kOk || empty) return st;
  if ((st = current_device(nullptr)) != kOk) return st;
  return launched(launch_combine_rows_backward(dout, (int)dt, lddo, y, (int)yt, ldy, T, k, H, rows, weights, slots, dy, lddy,
                                               dweights, (hipStream_t)stream));
}

}  // extern "C"
