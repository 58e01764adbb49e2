// Argument validation (pure host C++).
#include "validate.hpp"

namespace fp8bq {

static bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
static bool fmt_ok(int f) { return f == 0 || f == 1; }
static int in_esize(int t) { return t == 0 ? 2 : (t == 1 ? 4 : 0); }

// No device allocation reaches 2^48 bytes; bounding every matrix's byte extent by that keeps the
// extent and overlap arithmetic below free of overflow.
constexpr int64_t kMaxExtentBytes = int64_t(1) << 48;

int check_mat(const Mat& m, bool align_ld) {
  if (m.p == nullptr) return kErrNull;
  if (!aligned16(m.p)) return kErrAlign;
  if (m.ld < m.cols || m.ld < 1) return kErrLd;
  const int64_t max_elems = kMaxExtentBytes / m.esize;
  if (m.ld > max_elems || (m.rows > 1 && m.rows - 1 > (max_elems - m.cols) / m.ld)) return kErrShape;
  if (align_ld && ((m.ld * m.esize) % 16) != 0) return kErrLd;
  return kOk;
}

static void extent(const Mat& m, uintptr_t& lo, uintptr_t& hi) {
  lo = (uintptr_t)m.p;
  hi = lo + (uintptr_t)(((m.rows - 1) * m.ld + m.cols) * m.esize);
}

bool overlaps(const Mat& a, const Mat& b) {
  if (a.rows <= 0 || a.cols <= 0 || b.rows <= 0 || b.cols <= 0) return false;
  uintptr_t alo, ahi, blo, bhi;
  extent(a, alo, ahi);
  extent(b, blo, bhi);
  return alo < bhi && blo < ahi;
}

// Common tail of the three quantizers: input X, codes Q, scales S (each a Mat), checked in order.
static int check_quant(const Mat& x, const Mat& q, const Mat& s, bool s_align) {
  int st;
  if (x.p == nullptr || q.p == nullptr || s.p == nullptr) return kErrNull;
  if ((st = check_mat(x, true)) != kOk) return st;
  if ((st = check_mat(q, true)) != kOk) return st;
  if ((st = check_mat(s, s_align)) != kOk) return st;
  if (overlaps(q, x) || overlaps(s, x) || overlaps(q, s)) return kErrOverlap;
  return kOk;
}

int validate_quant_1x128(const void* x, int xt, int64_t R, int64_t C, int64_t ldx, int fmt, const void* q,
                         int64_t ldq, const void* s, int64_t lds, bool* empty) {
  *empty = false;
  if (in_esize(xt) == 0) return kErrDtype;
  if (!fmt_ok(fmt)) return kErrFormat;
  if (R < 0 || C < 0 || C % 128 != 0) return kErrShape;
  if (R == 0 || C == 0) {
    *empty = true;
    return kOk;
  }
  return check_quant(Mat{x, R, C, ldx, in_esize(xt)}, Mat{q, R, C, ldq, 1}, Mat{s, C / 128, R, lds, 4}, true);
}

int validate_quant_128x1(const void* x, int xt, int64_t R, int64_t C, int64_t ldx, int fmt, const void* qt,
                         int64_t ldqt, const void* st, int64_t ldst, bool* empty) {
  *empty = false;
  if (in_esize(xt) == 0) return kErrDtype;
  if (!fmt_ok(fmt)) return kErrFormat;
  if (R < 0 || C < 0 || R % 128 != 0 || C % 8 != 0) return kErrShape;
  if (R == 0 || C == 0) {
    *empty = true;
    return kOk;
  }
  return check_quant(Mat{x, R, C, ldx, in_esize(xt)}, Mat{qt, C, R, ldqt, 1}, Mat{st, R / 128, C, ldst, 4}, true);
}

int validate_quant_dual(const void* x, int xt, int64_t R, int64_t C, int64_t ldx, int fr, const void* q, int64_t ldq,
                        const void* s, int64_t lds, int fc, const void* qt, int64_t ldqt, const void* st,
                        int64_t ldst, bool* empty) {
  *empty = false;
  if (in_esize(xt) == 0) return kErrDtype;
  if (!fmt_ok(fr) || !fmt_ok(fc)) return kErrFormat;
  if (R < 0 || C < 0 || R % 128 != 0 || C % 128 != 0) return kErrShape;
  if (R == 0 || C == 0) {
    *empty = true;
    return kOk;
  }
  const Mat mx{x, R, C, ldx, in_esize(xt)};
  const Mat mq{q, R, C, ldq, 1}, ms{s, C / 128, R, lds, 4};
  const Mat mqt{qt, C, R, ldqt, 1}, mst{st, R / 128, C, ldst, 4};
  int r;
  if ((r = check_quant(mx, mq, ms, true)) != kOk) return r;
  if ((r = check_quant(mx, mqt, mst, true)) != kOk) return r;
  if (overlaps(mq, mqt) || overlaps(mq, mst) || overlaps(ms, mqt) || overlaps(ms, mst)) return kErrOverlap;
  return kOk;
}

int validate_quant_128x128_dual(const void* w, int wt, int64_t N, int64_t K, int64_t ldw, int fmt, const void* q,
                                int64_t ldq, const void* s, int64_t lds, const void* qt, int64_t ldqt, bool* empty) {
  *empty = false;
  if (in_esize(wt) == 0) return kErrDtype;
  if (!fmt_ok(fmt)) return kErrFormat;
  if (N < 0 || K < 0 || N % 128 != 0 || K % 128 != 0) return kErrShape;
  if (N == 0 || K == 0) {
    *empty = true;
    return kOk;
  }
  const Mat mw{w, N, K, ldw, in_esize(wt)}, mq{q, N, K, ldq, 1}, ms{s, N / 128, K / 128, lds, 4};
  const Mat mqt{qt, K, N, ldqt, 1};
  int r;
  if ((r = check_quant(mw, mq, ms, false)) != kOk) return r;
  if (qt == nullptr) return kErrNull;
  if ((r = check_mat(mqt, true)) != kOk) return r;
  if (overlaps(mqt, mw) || overlaps(mqt, mq) || overlaps(mqt, ms)) return kErrOverlap;
  return kOk;
}

int validate_quant_128x128(const void* w, int wt, int64_t N, int64_t K, int64_t ldw, int fmt, const void* q,
                           int64_t ldq, const void* s, int64_t lds, bool* empty) {
  *empty = false;
  if (in_esize(wt) == 0) return kErrDtype;
  if (!fmt_ok(fmt)) return kErrFormat;
  if (N < 0 || K < 0 || N % 128 != 0 || K % 128 != 0) return kErrShape;
  if (N == 0 || K == 0) {
    *empty = true;
    return kOk;
  }
  return check_quant(Mat{w, N, K, ldw, in_esize(wt)}, Mat{q, N, K, ldq, 1}, Mat{s, N / 128, K / 128, lds, 4},
                     false);
}

int validate_quant_weights_dual(const WeightJobArgs* jobs, int count, int max_jobs, int wt, int fmt, bool* empty) {
  if (count < 0 || count > max_jobs) return kErrValue;
  if (count > 0 && jobs == nullptr) return kErrNull;
  int r;
  for (int j = 0; j < count; ++j) {
    const WeightJobArgs& a = jobs[j];
    if ((r = validate_quant_128x128_dual(a.w, wt, a.N, a.K, a.ldw, fmt, a.q, a.ldq, a.s, a.lds, a.qt, a.ldqt,
                                         &empty[j])) != kOk)
      return r;
  }
  const int es = in_esize(wt);
  for (int i = 0; i < count; ++i) {
    if (empty[i]) continue;
    const WeightJobArgs& a = jobs[i];
    const Mat outs[3] = {{a.q, a.N, a.K, a.ldq, 1}, {a.s, a.N / 128, a.K / 128, a.lds, 4}, {a.qt, a.K, a.N, a.ldqt, 1}};
    for (int j = 0; j < count; ++j) {
      if (j == i || empty[j]) continue;
      const WeightJobArgs& b = jobs[j];
      const Mat theirs[4] = {{b.w, b.N, b.K, b.ldw, es},
                             {b.q, b.N, b.K, b.ldq, 1},
                             {b.s, b.N / 128, b.K / 128, b.lds, 4},
                             {b.qt, b.K, b.N, b.ldqt, 1}};
      for (const Mat& o : outs)
        for (const Mat& t : theirs)
          if (overlaps(o, t)) return kErrOverlap;
    }
  }
  return kOk;
}

static bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

int validate_quant_tensor(const void* x, int xt, int64_t R, int64_t C, int64_t ldx, int fmt, const void* amax,
                          double beta, const void* q, int64_t ldq, const void* qt, int64_t ldqt, const void* s,
                          const void* ws, size_t ws_bytes, size_t ws_needed, bool* empty) {
  *empty = false;
  if (in_esize(xt) == 0) return kErrDtype;
  if (!fmt_ok(fmt)) return kErrFormat;
  if (!(beta >= 0.0 && beta <= 1.0)) return kErrValue;  // also rejects NaN
  if (R < 0 || C < 0 || C % 128 != 0 || (qt != nullptr && R % 128 != 0)) return kErrShape;
  if (R == 0 || C == 0) {
    *empty = true;
    return kOk;
  }
  // ws_needed == 0: the caller passes no workspace (the kernels use the library's own scratch)
  const bool has_ws = ws_needed > 0;
  if (x == nullptr || q == nullptr || amax == nullptr || s == nullptr || (has_ws && ws == nullptr)) return kErrNull;
  int st;
  const Mat mx{x, R, C, ldx, in_esize(xt)}, mq{q, R, C, ldq, 1}, mqt{qt, C, R, ldqt, 1};
  const Mat ma{amax, 1, 1, 1, 4}, ms{s, 1, 1, 1, 4};
  if ((st = check_mat(mx, true)) != kOk) return st;
  if ((st = check_mat(mq, true)) != kOk) return st;
  if (qt != nullptr && (st = check_mat(mqt, true)) != kOk) return st;
  if (!aligned4(amax) || !aligned4(s) || (has_ws && !aligned16(ws))) return kErrAlign;
  if (ws_bytes < ws_needed) return kErrWorkspace;
  const Mat mw{has_ws ? ws : nullptr, 1, (int64_t)ws_needed, (int64_t)ws_needed, 1};
  const Mat outs[4] = {mq, mqt, ma, ms};
  const int nout = 4;
  for (int i = 0; i < nout; ++i) {
    if (outs[i].p == nullptr) continue;
    if (overlaps(outs[i], mx) || (has_ws && overlaps(outs[i], mw))) return kErrOverlap;
    for (int j = i + 1; j < nout; ++j)
      if (outs[j].p != nullptr && overlaps(outs[i], outs[j])) return kErrOverlap;
  }
  if (has_ws && overlaps(mw, mx)) return kErrOverlap;
  return kOk;
}

static bool finite_nonneg(double v) { return v >= 0.0 && v <= 1.7976931348623157e308; }

int validate_hyperball(const void* w, int64_t ldw, const void* g, int gt, int64_t ldg, int64_t R, int64_t C,
                       double lr, double wd, double eps, double radius, const void* norms, const void* ws,
                       size_t ws_bytes, size_t ws_needed, bool* empty) {
  *empty = false;
  if (in_esize(gt) == 0) return kErrDtype;
  if (!finite_nonneg(lr) || !finite_nonneg(wd) || !finite_nonneg(radius) || !(finite_nonneg(eps) && eps > 0.0))
    return kErrValue;
  if (R < 0 || C < 0 || C % 8 != 0) return kErrShape;
  if (R == 0 || C == 0) {
    *empty = true;
    return kOk;
  }
  if (w == nullptr || g == nullptr || ws == nullptr) return kErrNull;
  const Mat mw{w, R, C, ldw, 4}, mg{g, R, C, ldg, in_esize(gt)};
  int st;
  if ((st = check_mat(mw, true)) != kOk) return st;
  if ((st = check_mat(mg, true)) != kOk) return st;
  if (!aligned16(ws) || (norms != nullptr && !aligned4(norms))) return kErrAlign;
  if (ws_bytes < ws_needed) return kErrWorkspace;
  const Mat mws{ws, 1, (int64_t)ws_needed, (int64_t)ws_needed, 1}, mn{norms, 1, 2, 2, 4};
  if (overlaps(mw, mg) || overlaps(mws, mw) || overlaps(mws, mg)) return kErrOverlap;
  if (norms != nullptr && (overlaps(mn, mw) || overlaps(mn, mg) || overlaps(mn, mws))) return kErrOverlap;
  return kOk;
}

int validate_hyperball_batch(const HyperballJobArgs* jobs, int count, int max_jobs, int gt, double lr, double wd,
                             double eps, const void* ws, size_t ws_bytes, size_t ws_needed, bool* empty) {
  if (count < 0 || count > max_jobs) return kErrValue;
  if (count > 0 && jobs == nullptr) return kErrNull;
  if (in_esize(gt) == 0) return kErrDtype;
  if (!finite_nonneg(lr) || !finite_nonneg(wd) || !(finite_nonneg(eps) && eps > 0.0)) return kErrValue;
  bool any = false;
  for (int j = 0; j < count; ++j) {
    const HyperballJobArgs& a = jobs[j];
    // each job alone, with a stand-in workspace (the batch's is checked once below)
    alignas(16) static const double kStandIn[2] = {0.0, 0.0};
    int st = validate_hyperball(a.w, a.ldw, a.g, gt, a.ldg, a.R, a.C, lr, wd, eps, a.radius, a.norms, kStandIn,
                                ws_needed, 0, &empty[j]);
    if (st != kOk) return st;
    any = any || !empty[j];
  }
  if (!any) return kOk;
  if (ws == nullptr) return kErrNull;
  if (!aligned16(ws)) return kErrAlign;
  if (ws_bytes < ws_needed) return kErrWorkspace;
  const Mat mws{ws, 1, (int64_t)ws_needed, (int64_t)ws_needed, 1};
  const int es = in_esize(gt);
  for (int j = 0; j < count; ++j) {
    if (empty[j]) continue;
    const HyperballJobArgs& a = jobs[j];
    const Mat wj{a.w, a.R, a.C, a.ldw, 4}, gj{a.g, a.R, a.C, a.ldg, es}, nj{a.norms, 1, 2, 2, 4};
    if (overlaps(wj, mws) || overlaps(gj, mws) || (a.norms && overlaps(nj, mws))) return kErrOverlap;
    for (int k = 0; k < count; ++k) {
      if (k == j || empty[k]) continue;
      const HyperballJobArgs& b = jobs[k];
      const Mat wk{b.w, b.R, b.C, b.ldw, 4}, gk{b.g, b.R, b.C, b.ldg, es}, nk{b.norms, 1, 2, 2, 4};
      // job j writes w and norms: neither may touch anything job k reads or writes
      if (overlaps(wj, wk) || overlaps(wj, gk) || (b.norms && overlaps(wj, nk))) return kErrOverlap;
      if (a.norms && (overlaps(nj, wk) || overlaps(nj, gk) || (b.norms && overlaps(nj, nk)))) return kErrOverlap;
    }
  }
  return kOk;
}

int validate_stream_copy(const void* src, const void* dst, size_t bytes, bool* empty) {
  *empty = false;
  if (bytes % 16 != 0 || bytes >= ((size_t)1 << 48)) return kErrShape;
  if (bytes == 0) {
    *empty = true;
    return kOk;
  }
  if (!src || !dst) return kErrNull;
  if (!aligned16(src) || !aligned16(dst)) return kErrAlign;
  const uintptr_t a = (uintptr_t)src, b = (uintptr_t)dst;
  if (a < b + bytes && b < a + bytes) return kErrOverlap;
  return kOk;
}

int validate_gemm(const GemmArgs& g, size_t ws_needed, bool* empty, bool* zero_fill) {
  *empty = false;
  *zero_fill = false;
  if (g.op < 0 || g.op > 4) return kErrShape;
  if (!fmt_ok(g.fa) || !fmt_ok(g.fb)) return kErrFormat;
  if (g.out_t != 0 && g.out_t != 1 && !(g.out_t == 2 && g.op == 2)) return kErrDtype;
  const int64_t M = g.M, N = g.N, K = g.K;
  if (M < 0 || N < 0 || K < 0 || N % 128 != 0 || K % 128 != 0) return kErrShape;
  if (g.op == 2 && M % 128 != 0) return kErrShape;

  // Operand geometry per op: (A codes, A scales, B codes, B scales, output) as matrices.
  Mat qa, sa, qb, sb, out;
  int64_t out_rows, out_cols, contraction;
  const int oes = g.out_t == 0 ? 2 : 4;
  if (g.op == 4) {  // per-tensor scales: A[M,K], B[N,K] (one scale each) -> Y[M,N]
    qa = Mat{g.qa, M, K, g.ldqa, 1};
    sa = Mat{g.sa, 1, 1, 1, 4};
    qb = Mat{g.qb, N, K, g.ldqb, 1};
    sb = Mat{g.sb, 1, 1, 1, 4};
    out_rows = M; out_cols = N; contraction = K;
  } else if (g.op == 0) {  // fprop: X[M,K] (1x128), W[N,K] (128x128) -> Y[M,N]
    qa = Mat{g.qa, M, K, g.ldqa, 1};
    sa = Mat{g.sa, K / 128, M, g.ldsa, 4};
    qb = Mat{g.qb, N, K, g.ldqb, 1};
    sb = Mat{g.sb, N / 128, K / 128, g.ldsb, 4};
    out_rows = M; out_cols = N; contraction = K;
  } else if (g.op == 3) {  // dgrad on W^T codes: dY[M,N] (1x128), W^T[K,N] (128x128) -> dX[M,K]
    qa = Mat{g.qa, M, N, g.ldqa, 1};
    sa = Mat{g.sa, N / 128, M, g.ldsa, 4};
    qb = Mat{g.qb, K, N, g.ldqb, 1};
    sb = Mat{g.sb, N / 128, K / 128, g.ldsb, 4};
    out_rows = M; out_cols = K; contraction = N;
  } else if (g.op == 1) {  // dgrad: dY[M,N] (1x128), W[N,K] (128x128) -> dX[M,K]
    qa = Mat{g.qa, M, N, g.ldqa, 1};
    sa = Mat{g.sa, N / 128, M, g.ldsa, 4};
    qb = Mat{g.qb, N, K, g.ldqb, 1};
    sb = Mat{g.sb, N / 128, K / 128, g.ldsb, 4};
    out_rows = M; out_cols = K; contraction = N;
  } else {  // wgrad: dY^T[N,M] (128x1), X^T[K,M] (128x1) -> dW[N,K]
    qa = Mat{g.qa, N, M, g.ldqa, 1};
    sa = Mat{g.sa, M / 128, N, g.ldsa, 4};
    qb = Mat{g.qb, K, M, g.ldqb, 1};
    sb = Mat{g.sb, M / 128, K, g.ldsb, 4};
    out_rows = N; out_cols = K; contraction = M;
  }
  out = Mat{g.out, out_rows, out_cols, g.ldout, oes};
  if (out_rows == 0 || out_cols == 0) {
    *empty = true;
    return kOk;
  }
  int st;
  if (g.out == nullptr) return kErrNull;
  if ((st = check_mat(out, true)) != kOk) return st;
  if (contraction == 0) {
    *zero_fill = true;
    return kOk;
  }
  if (g.qa == nullptr || g.sa == nullptr || g.qb == nullptr || g.sb == nullptr) return kErrNull;
  if ((st = check_mat(qa, true)) != kOk) return st;
  if ((st = check_mat(qb, true)) != kOk) return st;
  // The kernels reach one tile of a code operand (at most 256 rows of the contraction) through a
  // buffer range of 32 bits: 255 row strides plus one row must stay below 4 GiB.  (dgrad's W codes
  // are first transposed into the workspace with rows of N bytes.)
  const int64_t kSpan = (int64_t)1 << 32;
  if (255 * qa.ld + contraction >= kSpan) return kErrLd;
  if (g.op != 1 && 255 * qb.ld + contraction >= kSpan) return kErrLd;
  if (g.op == 4) {  // the two scales are single floats
    if (!aligned4(g.sa) || !aligned4(g.sb)) return kErrAlign;
  } else {
    if ((st = check_mat(sa, true)) != kOk) return st;
    // weight scales are read one value at a time; the wgrad column scales as 16-byte vectors
    if ((st = check_mat(sb, g.op == 2)) != kOk) return st;
  }
  if (overlaps(out, qa) || overlaps(out, sa) || overlaps(out, qb) || overlaps(out, sb)) return kErrOverlap;
  if (ws_needed > 0) {
    if (g.ws == nullptr || g.ws_bytes < ws_needed) return kErrWorkspace;
    if (!aligned16(g.ws)) return kErrAlign;
    Mat wsm{g.ws, 1, (int64_t)ws_needed, (int64_t)ws_needed, 1};
    if (overlaps(wsm, out) || overlaps(wsm, qa) || overlaps(wsm, sa) || overlaps(wsm, qb) || overlaps(wsm, sb))
      return kErrOverlap;
  }
  return kOk;
}

int check_grouped_workspace(const GroupedArgs& g, const void* ws, size_t ws_bytes, size_t ws_needed) {
  if (ws_needed == 0) return kOk;
  if (ws == nullptr || ws_bytes < ws_needed) return kErrWorkspace;
  if (((uintptr_t)ws & 15u) != 0) return kErrAlign;
  if (ws_needed >= (size_t)1 << 62) return kErrShape;
  const int64_t n = (int64_t)ws_needed;
  const Mat w{ws, 1, n, n, 1};  // (wgrad: dY^T [N, T], X^T [K, T] -> dW [E N, K])
  const Mat m[] = {Mat{g.qa, g.N, g.T, g.ldqa, 1},          Mat{g.sa, g.T / 128, g.N, g.ldsa, 4},
                   Mat{g.qb, g.K, g.T, g.ldqb, 1},          Mat{g.sb, g.T / 128, g.K, g.ldsb, 4},
                   Mat{g.out, g.E * g.N, g.K, g.ldout, g.out_t == 0 ? 2 : 4}, Mat{g.offsets, 1, g.E + 1, g.E + 1, 8}};
  for (const Mat& v : m)
    if (overlaps(w, v)) return kErrOverlap;
  return kOk;
}

static bool aligned8(const void* p) { return ((uintptr_t)p & 7u) == 0; }

int validate_grouped(const GroupedArgs& g, bool* empty, bool* zero_fill) {
  *empty = false;
  *zero_fill = false;
  if (g.op < 0 || g.op > 2) return kErrShape;
  if (!fmt_ok(g.fa) || !fmt_ok(g.fb)) return kErrFormat;
  if (g.out_t != 0 && g.out_t != 1 && !(g.out_t == 2 && g.op == 2)) return kErrDtype;
  const int64_t E = g.E, T = g.T, N = g.N, K = g.K;
  if (E < 1 || E > kMaxGroupExperts || T < 0 || N < 0 || K < 0 || N % 128 != 0 || K % 128 != 0) return kErrShape;
  if (g.op == 2 && T % 128 != 0) return kErrShape;
  if (N == 0 || K == 0) {
    // a zero width leaves nothing to write, but a zero contraction has no defined output rows
    const bool none = g.op == 2 || T == 0 || (g.op == 0 ? N : K) == 0;
    *empty = none;
    return none ? kOk : kErrShape;
  }
  if (T == 0 && g.op != 2) {
    *empty = true;
    return kOk;
  }
  // token counts and stacked rows are 32-bit in the kernels, and scale offsets 32-bit byte offsets
  const int64_t kRows = (int64_t)1 << 30;
  if (T >= kRows || N >= kRows || K >= kRows || N > kRows / E || K > kRows / E) return kErrShape;
  const int oes = g.out_t == 0 ? 2 : 4;
  Mat qa, sa, qb, sb, out;
  int64_t contraction;
  if (g.op == 0) {  // X [T, K], W [E N, K] -> Y [T, N]
    qa = Mat{g.qa, T, K, g.ldqa, 1};
    sa = Mat{g.sa, K / 128, T, g.ldsa, 4};
    qb = Mat{g.qb, E * N, K, g.ldqb, 1};
    sb = Mat{g.sb, E * N / 128, K / 128, g.ldsb, 4};
    out = Mat{g.out, T, N, g.ldout, oes};
    contraction = K;
  } else if (g.op == 1) {  // dY [T, N], W^T [K, E N] -> dX [T, K]
    qa = Mat{g.qa, T, N, g.ldqa, 1};
    sa = Mat{g.sa, N / 128, T, g.ldsa, 4};
    qb = Mat{g.qb, K, E * N, g.ldqb, 1};
    sb = Mat{g.sb, E * N / 128, K / 128, g.ldsb, 4};
    out = Mat{g.out, T, K, g.ldout, oes};
    contraction = N;
  } else {  // dY^T [N, Tp], X^T [K, Tp] -> dW [E N, K]
    qa = Mat{g.qa, N, T, g.ldqa, 1};
    sa = Mat{g.sa, T / 128, N, g.ldsa, 4};
    qb = Mat{g.qb, K, T, g.ldqb, 1};
    sb = Mat{g.sb, T / 128, K, g.ldsb, 4};
    out = Mat{g.out, E * N, K, g.ldout, oes};
    contraction = T;
  }
  int st;
  if (g.out == nullptr) return kErrNull;
  if ((st = check_mat(out, true)) != kOk) return st;
  if (contraction == 0) {
    *zero_fill = true;
    return kOk;
  }
  if (g.offsets == nullptr || g.qa == nullptr || g.sa == nullptr || g.qb == nullptr || g.sb == nullptr) return kErrNull;
  if (!aligned8(g.offsets)) return kErrAlign;
  if ((st = check_mat(qa, true)) != kOk) return st;
  if ((st = check_mat(qb, true)) != kOk) return st;
  // one tile of a code operand is reached through a 32-bit buffer range
  const int64_t kSpan = (int64_t)1 << 32;
  if (255 * qa.ld + contraction >= kSpan || 255 * qb.ld + contraction >= kSpan) return kErrLd;
  if ((st = check_mat(sa, true)) != kOk) return st;
  if ((st = check_mat(sb, g.op == 2)) != kOk) return st;
  // fprop reaches the scale of weight block nb at byte 4 nb ldsb of a 32-bit range
  if (g.op == 0 && sb.ld > (kSpan / 4 - 1) / sb.rows) return kErrLd;
  const Mat off{g.offsets, 1, E + 1, E + 1, 8};
  if (overlaps(out, qa) || overlaps(out, sa) || overlaps(out, qb) || overlaps(out, sb) || overlaps(out, off))
    return kErrOverlap;
  return kOk;
}

int validate_quant_grouped(const void* x, int xt, int64_t T, int64_t C, int64_t ldx, const void* offsets, int64_t E,
                           int fr, const void* q, int64_t ldq, const void* s, int64_t lds, int fc, const void* qt,
                           int64_t ldqt, const void* st, int64_t ldst, int64_t padded, int64_t padded_needed,
                           bool* empty) {
  *empty = false;
  const bool rows = q != nullptr || s != nullptr;
  if (in_esize(xt) == 0) return kErrDtype;
  if ((rows && !fmt_ok(fr)) || !fmt_ok(fc)) return kErrFormat;
  if (E < 1 || E > kMaxGroupExperts || T < 0 || C < 0 || C % 128 != 0) return kErrShape;
  if (T >= ((int64_t)1 << 30) || padded % 128 != 0 || padded < padded_needed || padded >= ((int64_t)1 << 31) ||
      C / 128 >= ((int64_t)1 << 31))
    return kErrShape;
  if (T == 0 || C == 0) {
    *empty = true;
    return kOk;
  }
  if (offsets == nullptr) return kErrNull;
  if (!aligned8(offsets)) return kErrAlign;
  const Mat mx{x, T, C, ldx, in_esize(xt)}, off{offsets, 1, E + 1, E + 1, 8};
  const Mat mqt{qt, C, padded, ldqt, 1}, mst{st, padded / 128, C, ldst, 4};
  const Mat mq{q, T, C, ldq, 1}, ms{s, C / 128, T, lds, 4};
  int r;
  if ((r = check_quant(mx, mqt, mst, true)) != kOk) return r;
  if (overlaps(mqt, off) || overlaps(mst, off)) return kErrOverlap;
  if (rows) {
    if ((r = check_quant(mx, mq, ms, true)) != kOk) return r;
    if (overlaps(mq, off) || overlaps(ms, off) || overlaps(mq, mqt) || overlaps(mq, mst) || overlaps(ms, mqt) ||
        overlaps(ms, mst))
      return kErrOverlap;
  }
  return kOk;
}

int validate_mx_quant(const void* x, int xt, int64_t R, int64_t C, int64_t ldx, const void* q, int64_t ldq,
                      const void* s, int64_t lds, const void* qt, int64_t ldqt, const void* st, int64_t ldst,
                      bool* empty) {
  *empty = false;
  const bool rows = q != nullptr || s != nullptr, cols = qt != nullptr || st != nullptr;
  if (in_esize(xt) == 0) return kErrDtype;
  // row blocks need whole blocks of columns; column blocks are padded, but are stored per 8 columns
  if (R < 0 || C < 0 || C % 8 != 0 || (rows && C % 32 != 0)) return kErrShape;
  if (R == 0 || C == 0) {
    *empty = true;
    return kOk;
  }
  if (x == nullptr || (!rows && !cols)) return kErrNull;
  const int64_t kMost = (int64_t)1 << 31;
  if (R >= kMost || C >= kMost || (R / 128 + 1) * (C / 128 + 1) >= kMost) return kErrShape;  // tiles of one launch
  const Mat mx{x, R, C, ldx, in_esize(xt)};
  const Mat mq{q, R, C / 2, ldq, 1}, ms{s, (C + 127) / 128, R, lds, 4};
  const Mat mqt{qt, C, (R + 31) / 32 * 16, ldqt, 1}, mst{st, (R + 127) / 128, C, ldst, 4};
  int r;
  if (rows) {
    if ((r = check_quant(mx, mq, ms, false)) != kOk) return r;
  }
  if (cols) {
    if ((r = check_quant(mx, mqt, mst, false)) != kOk) return r;
  }
  if (rows && cols && (overlaps(mq, mqt) || overlaps(mq, mst) || overlaps(ms, mqt) || overlaps(ms, mst)))
    return kErrOverlap;
  return kOk;
}

// The operands of an MXFP4 product as matrices: A (codes or values), its scales (codes only), B, its scales,
// the output and the offsets (grouped only); absent ones have no rows.
static void mx_mats(const MxArgs& g, Mat (&m)[6]) {
  const int64_t rows_b = g.E ? g.E * g.N : g.N, kw = (g.K + 127) / 128;
  const bool codes = g.a_type == 2;
  m[0] = codes ? Mat{g.a, g.M, g.K / 2, g.lda, 1} : Mat{g.a, g.M, g.K, g.lda, g.a_type == 0 ? 2 : 4};
  m[1] = Mat{g.sa, codes ? kw : 0, g.M, g.ldsa, 4};
  m[2] = Mat{g.b, rows_b, g.K / 2, g.ldb, 1};
  m[3] = Mat{g.sb, kw, rows_b, g.ldsb, 4};
  m[4] = Mat{g.out, g.M, g.N, g.ldout, g.out_t == 0 ? 2 : 4};
  m[5] = Mat{g.offsets, g.E ? 1 : 0, g.E + 1, g.E + 1, 8};
}

int validate_mx(const MxArgs& g, bool* empty, bool* zero_fill) {
  *empty = false;
  *zero_fill = false;
  if (g.a_type < 0 || g.a_type > 2 || g.out_t < 0 || g.out_t > 2) return kErrDtype;
  if (g.out_t == 2 && (g.E != 0 || g.a_type != 2)) return kErrDtype;  // only the dense product of codes is added to C
  if (g.E < 0 || g.E > kMaxGroupExperts || g.M < 0 || g.N < 0 || g.K < 0 || g.K % 32 != 0) return kErrShape;
  if (g.M == 0 || g.N == 0) {
    *empty = true;
    return kOk;
  }
  const int64_t kRows = (int64_t)1 << 30;
  const int64_t copies = g.E ? g.E : 1;
  if (g.M >= kRows || g.K >= kRows || g.N >= kRows / copies) return kErrShape;
  // work units of one launch: tiles of at least 16 x 16, every expert with a started one of its own
  if ((g.M / 16 + copies) * (g.N / 16 + 1) >= ((int64_t)1 << 31)) return kErrShape;
  Mat m[6];
  mx_mats(g, m);
  int st;
  if (g.out == nullptr) return kErrNull;
  if ((st = check_mat(m[4], false)) != kOk) return st;
  if (g.K == 0) {
    if (g.E) return kErrShape;  // (which rows belong to an expert is not known on the host)
    *zero_fill = true;
    return kOk;
  }
  for (int i = 0; i < 6; ++i)
    if (m[i].rows && m[i].p == nullptr) return kErrNull;
  if (g.E && !aligned8(g.offsets)) return kErrAlign;
  if ((st = check_mat(m[0], true)) != kOk) return st;
  if ((st = check_mat(m[2], true)) != kOk) return st;
  if (m[1].rows && (st = check_mat(m[1], false)) != kOk) return st;
  if ((st = check_mat(m[3], false)) != kOk) return st;
  // one tile of a code operand is reached through a 32-bit buffer range
  const int64_t kSpan = (int64_t)1 << 32;
  if ((m[1].rows && 255 * g.lda + g.K >= kSpan) || 255 * g.ldb + g.K >= kSpan) return kErrLd;
  for (int i = 0; i < 6; ++i)
    if (i != 4 && overlaps(m[4], m[i])) return kErrOverlap;
  return kOk;
}

int check_workspace(const MxArgs& g, const void* ws, size_t ws_bytes, size_t ws_needed) {
  if (ws_needed == 0) return kOk;
  if (ws == nullptr || ws_bytes < ws_needed) return kErrWorkspace;
  if (!aligned16(ws)) return kErrAlign;
  if (ws_needed >= (size_t)kMaxExtentBytes) return kErrShape;
  const Mat w{ws, 1, (int64_t)ws_needed, (int64_t)ws_needed, 1};
  Mat m[6];
  mx_mats(g, m);
  for (int i = 0; i < 6; ++i)
    if (overlaps(w, m[i])) return kErrOverlap;
  return kOk;
}

}  // namespace fp8bq
