// Host-side checks of the validation and planning of the 8-bit, routing and orthogonalization entry points (pure C++, no
// HIP), built with g++ and the address and undefined-behaviour sanitizers: random and extreme arguments never
// trigger undefined behaviour, every status is a documented one, and every plan of accepted sizes is consistent.  Prints
// "ok" and exits 0 on success.
#include <cstdint>
#include <cstdio>
#include <random>

#include "ortho_plan.hpp"
#include "plan.hpp"
#include "validate.hpp"

using namespace fp8bq;

static int failures = 0;
#define EXPECT(cond)                                                                             \
  do {                                                                                           \
    if (!(cond)) {                                                                               \
      if (failures < 20) std::fprintf(stderr, "%s:%d: failed: %s\n", __FILE__, __LINE__, #cond); \
      ++failures;                                                                                \
    }                                                                                            \
  } while (0)

static std::mt19937_64 rng(99);

static int64_t pick_size() {
  switch (rng() % 10) {
    case 0: return -(int64_t)(rng() % 1000);
    case 1: return (int64_t)(rng() % 3);
    case 2: return (int64_t)1 << (16 + rng() % 47);
    case 3: return INT64_MAX - (int64_t)(rng() % 1000);
    case 4: return 16 * (int64_t)(1 + rng() % 100000);
    default: return 16 * (int64_t)(1 + rng() % 300);
  }
}
static int64_t pick_few(int64_t most) { return rng() % 5 == 0 ? pick_size() : (int64_t)(rng() % (most + 2)); }
static int64_t pick_ld(int64_t cols) {
  switch (rng() % 5) {
    case 0: return (int64_t)(rng() % 1000) - 10;
    case 1: return (int64_t)1 << (rng() % 63);
    default: return cols > 0 && cols < INT64_MAX - 200 ? cols + 16 * (int64_t)(rng() % 8) : 16;
  }
}
static const void* pick_ptr() {
  switch (rng() % 9) {
    case 0: return nullptr;
    case 1: return reinterpret_cast<const void*>((uintptr_t)(rng() % (1ull << 47)) | 1);
    case 2: return reinterpret_cast<const void*>((uintptr_t)0x100000);
    default: return reinterpret_cast<const void*>((uintptr_t)((rng() % (1ull << 46)) & ~(uint64_t)15));
  }
}
static bool documented(int st) { return st >= kOk && st <= kErrValue; }

static void check_int8() {
  const int64_t E = rng() % 2 ? 0 : pick_few(kMaxGroupExperts), M = pick_size(), N = pick_size(), K = pick_size();
  bool empty = false, zero = false;
  MxArgs m{};
  m.E = E;
  m.M = M;
  m.N = N;
  m.K = K;
  m.offsets = pick_ptr();
  m.a_type = (int)(rng() % 4);
  m.a = pick_ptr();
  m.lda = pick_ld(K);
  m.sa = pick_ptr();
  m.b = pick_ptr();
  m.ldb = pick_ld(K);
  m.sb = pick_ptr();
  m.out = pick_ptr();
  m.out_t = (int)(rng() % 4);
  m.ldout = pick_ld(N);
  const int st = validate_int8(m, &empty, &zero);
  EXPECT(documented(st));
  if (st == kOk && !empty) EXPECT(documented(check_int8_workspace(m, pick_ptr(), (size_t)pick_size(), (size_t)(rng() % 100000))));
  m.out = nullptr;
  m.a_type = 2;
  m.out_t = 0;
  if (validate_int8(m, &empty, &zero) == kErrNull && K > 0) {  // sizes that pass: their plan
    const int cus = (int)(rng() % 4 == 0 ? rng() % 400 : 256);
    const bool linear = rng() % 2;
    const MxPlan p = plan_int8(linear, E, M, N, K, cus);
    EXPECT(p.grid >= 1 && p.grid < ((int64_t)1 << 31) && p.split_k >= 1 && p.split_k <= 8);
    EXPECT(!p.fused || (linear && p.skinny && E == 0 && M * K <= 12288));
    EXPECT(!p.skinny || (M <= 16 && 8 % p.split_k == 0 && p.ws == 0));
    if (!p.skinny) {
      EXPECT(p.tiles_m >= 1 && p.tiles_n >= 1 && (double)p.tiles_m * (double)p.tiles_n * p.split_k < 2147483648.0);
      EXPECT((p.split_k > 1) == (p.ws > 0) && p.ws < ((size_t)1 << 46) && (E == 0 || p.split_k == 1));
    }
  }
  for (int columns = 0; columns < 2; ++columns)
    EXPECT(documented(validate_int8_quant(pick_ptr(), (int)(rng() % 3), M, N, pick_ld(N), columns != 0, pick_ptr(),
                                          pick_ld(columns ? M : N), pick_ptr(), pick_ptr(), (size_t)pick_size(),
                                          (size_t)(rng() % 100000), &empty)));
}

static void check_routing() {
  bool empty = false;
  const int64_t T = pick_size(), E = pick_few(kMaxGroupExperts), k = pick_few(64), H = pick_size();
  const double scales[4] = {1.0, 2.5, 1e308 * 10.0, -0.0};
  const RouteCheck r{pick_ptr(), (int)(rng() % 3), T, E, pick_ld(E), k, (int)(rng() % 3), rng() % 2 ? 1 : pick_few(64),
                     rng() % 2 ? 1 : pick_few(8), rng() % 2 ? 1 : pick_few(2), scales[rng() % 4]};
  EXPECT(documented(validate_route(r, pick_ptr(), pick_ptr(), pick_ptr(), &empty)));
  EXPECT(documented(validate_route_backward(r, pick_ptr(), pick_ptr(), pick_ptr(), pick_ld(E), &empty)));
  EXPECT(documented(validate_expert_rows(pick_ptr(), T, E, pick_ptr(), pick_ptr(), pick_ptr(), pick_ptr(), (size_t)pick_size(),
                                         (size_t)(rng() % 100000))));
  const RowsCheck c{T, k, H, {pick_ptr(), pick_ptr()}, {(int)(rng() % 3), (int)(rng() % 3)}, {pick_ld(H), pick_ld(H)},
                    {rng() % 2 == 0, rng() % 2 == 0}, pick_ptr(), (int)(rng() % 3), pick_ld(H), rng() % 2 == 0,
                    {pick_ptr(), pick_ptr(), pick_ptr()}, pick_ptr()};
  EXPECT(documented(validate_rows(c, 1 + (int)(rng() % 2), 1 + (int)(rng() % 3), &empty)));
}

static void check_ortho() {
  bool empty = false;
  const double coef[6] = {3.4445, -4.7750, 2.0315, 3.4445, rng() % 8 ? -4.7750 : 1e308 * 10.0, 2.0315};
  const int64_t B = rng() % 2 ? 1 : pick_few(kMaxOrthoBatch), R = pick_size(), C = rng() % 2 ? pick_size() : 1 + (int64_t)(rng() % 5000);
  const OrthoCheck c{pick_ptr(), (int)(rng() % 3), B, R, C, pick_ld(C), pick_ld(R), (int)(rng() % 4) - 1 > 2 ? 2 : (int)(rng() % 3),
                     rng() % 8 ? coef : nullptr, rng() % 8 ? 1e-7 : 0.0, pick_ptr(), pick_ld(C), pick_size()};
  const int st = validate_ortho(c, &empty);
  EXPECT(documented(st));
  if (B >= 1 && R >= 1 && C >= 1 && B <= kMaxOrthoBatch && R <= kMaxOrthoSide && C <= kMaxOrthoSide) {
    bool fits = false;
    const OrthoPlan p = plan_ortho(B, R, C, (int)(rng() % 4 == 0 ? rng() % 400 : 256), &fits);
    if (fits) {
      EXPECT(p.norm_blocks >= 1 && p.ws < ((size_t)1 << 50));
      const OrthoProduct* q[3] = {&p.gram, &p.poly, &p.update};
      for (int i = 0; i < 3; ++i) {
        EXPECT(q[i]->grid >= 1 && q[i]->split >= 1 && (i < 2 || q[i]->split == 1));
        EXPECT((double)q[i]->tiles * q[i]->split * (double)B < 2147483648.0);
        EXPECT(i == 2 || q[i]->shape != k256x192);
      }
      const size_t at[9] = {p.at_norms, p.at_factor, p.at_x, p.at_xt[0], p.at_xt[1], p.at_low, p.at_gram, p.at_poly, p.at_parts};
      for (int i = 0; i < 9; ++i) EXPECT(at[i] % 256 == 0 && at[i] <= p.ws && (i == 0 || at[i] > at[i - 1]));
      if (st == kOk && !empty) EXPECT(documented(check_ortho_workspace(c, pick_ptr(), (size_t)pick_size(), p.ws)));
    }
  }
}

int main() {
  for (int it = 0; it < 200000; ++it) {
    check_int8();
    check_routing();
    check_ortho();
  }
  if (failures) {
    std::fprintf(stderr, "%d failures\n", failures);
    return 1;
  }
  std::printf("ok\n");
  return 0;
}
