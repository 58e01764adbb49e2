// Host-side checks of the validation and planning of the grouped and MXFP4 entry points (pure C++, no HIP), built
// with g++ and the address and undefined-behaviour sanitizers: random and extreme arguments never trigger
// undefined behaviour, every status is a documented one, and every plan of accepted sizes is consistent.  Prints
// "ok" and exits 0 on success.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <random>

#include "plan.hpp"
#include "validate.hpp"

using namespace fp8bq;

static int failures = 0;
#define EXPECT(cond)                                                                                   \
  do {                                                                                                 \
    if (!(cond)) {                                                                                     \
      if (failures < 20) std::fprintf(stderr, "%s:%d: failed: %s\n", __FILE__, __LINE__, #cond);       \
      ++failures;                                                                                      \
    }                                                                                                  \
  } while (0)

static std::mt19937_64 rng(4321);

static int64_t pick_size() {
  switch (rng() % 9) {
    case 0: return -(int64_t)(rng() % 1000);
    case 1: return 0;
    case 2: return (int64_t)(rng() % 300);
    case 3: return 32 * (int64_t)(1 + rng() % 128);
    case 4: return 128 * (int64_t)(1 + rng() % 4096);
    case 5: return (int64_t)1 << (16 + rng() % 47);
    case 6: return INT64_MAX - (int64_t)(rng() % 1000);
    default: return 128 * (int64_t)(1 + rng() % 16);
  }
}
static int64_t pick_experts() { return rng() % 4 == 0 ? pick_size() : (int64_t)(1 + rng() % 512); }
static int64_t pick_ld(int64_t cols) {
  switch (rng() % 5) {
    case 0: return cols;
    case 1: return cols > INT64_MAX - 200 ? cols : cols + 16 * (int64_t)(rng() % 8);
    case 2: return (int64_t)(rng() % 1000) - 10;
    case 3: return (int64_t)1 << (rng() % 63);
    default: return cols > 0 ? cols : 16;
  }
}
static const void* pick_ptr() {
  switch (rng() % 7) {
    case 0: return nullptr;
    case 1: return reinterpret_cast<const void*>((uintptr_t)(rng() % (1ull << 47)) | 1);
    case 2: return reinterpret_cast<const void*>((uintptr_t)0x100000);
    default: return reinterpret_cast<const void*>((uintptr_t)((rng() % (1ull << 44)) & ~(uint64_t)15));
  }
}
static bool documented(int st) { return st >= kOk && st <= kErrValue; }

static void check_plan(bool linear, int64_t E, int64_t M, int64_t N, int64_t K, int cus) {
  const MxPlan p = plan_mx(linear, E, M, N, K, cus);
  EXPECT(p.grid >= 1 && p.grid < ((int64_t)1 << 31));
  EXPECT(p.split_k >= 1 && p.split_k <= 8);
  EXPECT(!p.fused || (linear && p.skinny));
  if (p.skinny) {
    EXPECT(8 % p.split_k == 0 && p.ws == 0);
  } else {
    EXPECT(p.tiles_m >= 1 && p.tiles_n >= 1 && (double)p.tiles_m * (double)p.tiles_n * p.split_k < 2147483648.0);
    EXPECT((p.split_k > 1) == (p.ws > 0) && p.ws < ((size_t)1 << 46));
    EXPECT(E == 0 || p.split_k == 1);
  }
}

// Splitting of long experts: a chunk is never empty, no more sets are taken than there are, and the choice that
// splits nothing is always open.
static void check_chunks() {
  for (int i = 0; i < 64; ++i) {
    const float s = chunk_candidate(i);
    EXPECT(s >= 4.0f && (i == 0 || s > chunk_candidate(i - 1)));
    for (int n = 1; n < 1 << 24; n += 1 + n / 7) {
      const int c = chunks_of(n, s, 1.0f / s);
      EXPECT(c >= 1 && c <= n && (i != 63 || c == 1) && (double)n / c <= 1.001 * s);
    }
  }
  for (int it = 0; it < 20000; ++it) {
    const GroupSplit g{(int)(rng() % (kMaxSets + 1)), (float)(1 + rng() % 600), 512.0f, (float)(1 << rng() % 3),
                       (float)(rng() % 1000) / 100.0f, 2.5f};
    int n[40];
    const int E = 1 + (int)(rng() % 40);
    for (int e = 0; e < E; ++e) n[e] = rng() % 3 ? (int)(rng() % 10) : (int)(rng() % 3000);
    for (int i = 0; i < 64; ++i) {
      ChunkSums c(*std::max_element(n, n + E), chunk_candidate(i));
      for (int e = 0; e < E; ++e) c.add(n[e], chunk_candidate(i), 1.0f / chunk_candidate(i));
      const float t = chunk_time(c, g);
      EXPECT(t >= 0.0f && (c.sets <= g.sets ? t < 1e30f : t > 1e30f) && (i != 63 || c.sets == 0));
    }
  }
}

int main() {
  check_chunks();
  bool empty = false, zero = false;
  for (int it = 0; it < 300000; ++it) {
    const int64_t E = pick_experts(), T = pick_size(), N = pick_size(), K = pick_size();
    const int fmt = (int)(rng() % 3), cus = (int)(rng() % 4 == 0 ? rng() % 400 : 256);
    GroupedArgs g{(int)(rng() % 4), E, T, N, K, pick_ptr(), pick_ptr(), pick_ld(K), pick_ptr(), pick_ld(T), fmt,
                  pick_ptr(), pick_ld(K), pick_ptr(), pick_ld(K / 128), fmt, pick_ptr(), (int)(rng() % 4), pick_ld(N)};
    const int st = validate_grouped(g, &empty, &zero);
    EXPECT(documented(st));
    if (st == kOk && !empty && !zero) {
      const GemmPlan p = plan_grouped(g.op, E, T, N, K, cus);
      if (p.fits) EXPECT(p.grid >= 1 && p.grid <= p.units && p.units < ((int64_t)1 << 31));
      const int64_t sets = p.group_split.sets;
      EXPECT(sets >= 0 && sets <= kMaxSets && (g.op == kOpWgrad || sets == 0));
      if (p.fits) EXPECT(p.ws_gemm == (sets ? kSplitListBytes + (size_t)sets * (size_t)N * (size_t)K * 4 : 0));
      EXPECT(plan_grouped(g.op, E, T, N, K, cus, false).ws_gemm == 0);
      EXPECT(documented(check_grouped_workspace(g, pick_ptr(), (size_t)pick_size(), p.ws_gemm)));
    }
    if (T >= 0 && T < ((int64_t)1 << 30) && E >= 1 && E <= kMaxGroupExperts) {
      const int64_t padded = grouped_padded_rows(T, E);
      EXPECT(padded % 128 == 0 && padded >= T / 128 * 128 && padded <= T + 127 * E);
      EXPECT(documented(validate_quant_grouped(pick_ptr(), (int)(rng() % 3), T, N, pick_ld(N), pick_ptr(), E, fmt,
                                               pick_ptr(), pick_ld(N), pick_ptr(), pick_ld(T), fmt, pick_ptr(),
                                               pick_ld(padded), pick_ptr(), pick_ld(N), rng() % 2 ? padded : pick_size(),
                                               padded, &empty)));
    }
    EXPECT(documented(validate_mx_quant(pick_ptr(), (int)(rng() % 3), T, N, pick_ld(N), pick_ptr(), pick_ld(N / 2),
                                        pick_ptr(), pick_ld(T), pick_ptr(), pick_ld(T / 2), pick_ptr(), pick_ld(N),
                                        &empty)));
    MxArgs m{};
    m.E = rng() % 2 ? 0 : E;
    m.M = T;
    m.N = N;
    m.K = K;
    m.offsets = pick_ptr();
    m.a_type = (int)(rng() % 4);
    m.a = pick_ptr();
    m.lda = pick_ld(m.a_type == 2 ? K / 2 : K);
    m.sa = pick_ptr();
    m.ldsa = pick_ld(T);
    m.b = pick_ptr();
    m.ldb = pick_ld(K / 2);
    m.sb = pick_ptr();
    m.ldsb = pick_ld(N);
    m.out = pick_ptr();
    m.out_t = (int)(rng() % 4);
    m.ldout = pick_ld(N);
    const int sm = validate_mx(m, &empty, &zero);
    EXPECT(documented(sm));
    if (sm == kOk && !empty) EXPECT(documented(check_workspace(m, pick_ptr(), (size_t)pick_size(), (size_t)(rng() % 100000))));
    // sizes alone: what the validation accepts up to the missing pointers is planned
    m.a_type = 2;
    m.out_t = 0;
    m.out = nullptr;
    if (validate_mx(m, &empty, &zero) == kErrNull && K > 0) {
      check_plan(false, m.E, m.M, m.N, m.K, cus);
      check_plan(true, m.E, m.M, m.N, m.K, cus);
    }
  }
  // a few tokens take the kernel that needs no workspace, a training micro-batch the largest tile
  EXPECT(plan_mx(true, 0, 1, 11264, 2048, 256).fused);
  EXPECT(!plan_mx(true, 0, 16384, 11264, 2048, 256).skinny && plan_mx(true, 0, 16384, 11264, 2048, 256).shape == k256x256);
  EXPECT(plan_grouped(kOpFprop, 64, 32768, 2816, 2048, 256).shape == k256x256);
  // one expert with everything and few tiles is split, the tiles of one expert that fill the card are not
  EXPECT(plan_grouped(kOpWgrad, 1, 30080, 256, 256, 256).group_split.sets > 8);
  EXPECT(plan_grouped(kOpWgrad, 8, 32768, 5632, 4096, 256).group_split.sets == 0);
  EXPECT(plan_grouped(kOpWgrad, 8, 1920, 2048, 1408, 256).group_split.sets == 0);
  if (failures) {
    std::fprintf(stderr, "%d failures\n", failures);
    return 1;
  }
  std::puts("ok");
  return 0;
}
