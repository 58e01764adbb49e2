// Routing: from the router's logits [T, E] each token's k experts and their weights, and the logits' gradient.
//
// Mathematics.  s = softmax(x) or sigmoid(x), c = s + bias; groups of E / G experts score the sum of their best one or
// two c, the best `top` groups stay; of their experts the k largest c are chosen, descending; w = scale s, or scale s /
// (sum of the chosen s).  Without a bias and with groups scored by their best expert the order of c is that of x, and
// no score is computed for the choice; a normalized softmax then needs the chosen logits only.
//
// Near scores: c is computed in 64 bits (about 1e-14, exp_all below) and compared by its first 43 bits and, where those
// are equal, by the index, the lower first.  In 32 bits one token in some ten thousand would swap two experts.  FP64
// runs at FP32's rate on this card, so what it costs is registers.
//
// Bound by instructions: 16384 tokens of 256 experts are 17 MB, 4 us at the copy's rate, and some 100 wave instructions
// a token for scores and as many for the choice (8 of 256 sigmoid scores with a bias, in 8 groups of which 4 stay, 17.2 us; 8 of
// 256 softmax scores 9.0; 2 of 96 in BF16 at 8192 tokens 5.0; a call of few tokens 3 to 6, a launch's 2 and one pass of
// dependent steps).  A token is shared by 16 lanes (many tokens) or 64 (few, where latency counts).  The lanes are dealt to the groups first, so that a group's score is a reduction over neighbouring lanes; a
// lane holds V consecutive experts of its group.  A key is c with the index in place of its last nine bits (key_of), so
// keys are distinct, one maximum over the lanes names the winner, and the winner alone clears its slot.
#include "device_common.hpp"
#include "launch.hpp"

namespace fp8bq {

// Maximum and minimum of numbers that are no NaN (written out: the compiler quiets NaNs before each of its own).
__device__ __forceinline__ double max64(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double min64(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

// e^x in 64 bits of V numbers up to 709, all through one step before the next, so that a step's constant is loaded once;
// below -708: 0.  2^n e^r, |r| <= ln 2 / 2, by the Taylor series to r^12 / 12! (the rest is below 2 10^-16).
template <int V>
__device__ __forceinline__ void exp_all(double (&x)[V]) {
  double p[V];
  int n[V];
  bool low[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    low[j] = x[j] < -708.0;  // (a NaN goes on)
    const double t = low[j] ? -708.0 : x[j];
    const double m = __builtin_rint(t * 1.4426950408889634);
    // (ln 2 in two parts, as Cody and Waite do it: the first is its 32 bits behind the point, so m times it is exact)
    x[j] = __builtin_fma(m, -0x1.a39ef35793c76p-33, __builtin_fma(m, -0x1.62e42fee00000p-1, t));
    n[j] = (int)m;
    p[j] = 1.0 / 479001600.0;
  }
  auto step = [&](double c) {
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = __builtin_fma(p[j], x[j], c);
  };
  step(1.0 / 39916800.0);
  step(1.0 / 3628800.0);
  step(1.0 / 362880.0);
  step(1.0 / 40320.0);
  step(1.0 / 5040.0);
  step(1.0 / 720.0);
  step(1.0 / 120.0);
  step(1.0 / 24.0);
  step(1.0 / 6.0);
  step(0.5);
  step(1.0);
  step(1.0);
#pragma unroll
  for (int j = 0; j < V; ++j) x[j] = low[j] ? 0.0 : __builtin_ldexp(p[j], n[j]);
}
__device__ __forceinline__ double exp64(double x) {
  double v[1] = {x};
  exp_all(v);
  return v[0];
}
// 1 / (1 + e^-x): the hardware's estimate of the reciprocal and two Newton steps.  (e^708 is finite, so the steps stay
// finite; below -708 the weight is zero in FP32 many times over.)
template <int V>
__device__ __forceinline__ void sigmoid_all(double (&x)[V]) {
  double e[V];
#pragma unroll
  for (int j = 0; j < V; ++j) e[j] = x[j] < -708.0 ? 708.0 : -x[j];
  exp_all(e);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const double v = 1.0 + e[j];
    double r = __builtin_amdgcn_rcp(v);
    r = __builtin_fma(__builtin_fma(-v, r, 1.0), r, r);
    r = __builtin_fma(__builtin_fma(-v, r, 1.0), r, r);
    x[j] = x[j] < -708.0 ? 0.0 : r;
  }
}
__device__ __forceinline__ double sigmoid64(double x) {
  double v[1] = {x};
  sigmoid_all(v);
  return v[0];
}

// c with the index in its last nine bits, so that of equal ones the lower index is the larger number: 511 - e where c is
// positive, e where it is negative and more bits are a smaller number.  c is kept within 10^308 (infinities; a NaN counts
// as -infinity); kShut, of a slot that cannot be chosen or was, is below all.
constexpr double kMostKey = 1e308;
constexpr uint32_t kShutHigh = 0xFFEFFFFFu;  // the high word of numbers below -1.797 10^308
__device__ __forceinline__ double shut_key() { return __builtin_bit_cast(double, (uint64_t)kShutHigh << 32); }
__device__ __forceinline__ double key_of(double c, int e) {
  c = c > -kMostKey ? c : -kMostKey;
  c = c < kMostKey ? c + 0.0 : kMostKey;  // (-0 and 0 are equal)
  const uint64_t b = __builtin_bit_cast(uint64_t, c);
  const uint32_t low = ((uint32_t)b & ~511u) | (uint32_t)((int64_t)b < 0 ? e : 511 - e);
  return __builtin_bit_cast(double, (b & 0xFFFFFFFF00000000ull) | low);
}
__device__ __forceinline__ int index_of(double key) {
  const uint64_t b = __builtin_bit_cast(uint64_t, key);
  return (int64_t)b < 0 ? (int)(b & 511) : 511 - (int)(b & 511);
}

// The value that lane l ^ d holds (16 <= d), or of the partner in a reduction over 2 d lanes that leaves equal values
// in the lanes below: xor 1 and 2, then mirrored halves, then a rotation by 8.
template <int D>
__device__ __forceinline__ uint32_t partner32(uint32_t v) {
  if constexpr (D == 1) return dpp_read<kDppXor1>(v);
  else if constexpr (D == 2) return dpp_read<kDppXor2>(v);
  else if constexpr (D == 4) return dpp_read<kDppMirror8>(v);
  else if constexpr (D == 8) return dpp_read<kDppXor8>(v);
  else return (uint32_t)__shfl_xor((int)v, D);
}
template <int D>
__device__ __forceinline__ uint64_t partner(uint64_t v) {
  return (uint64_t)partner32<D>((uint32_t)v) | (uint64_t)partner32<D>((uint32_t)(v >> 32)) << 32;
}
template <int D>
__device__ __forceinline__ double partner(double v) {
  return __builtin_bit_cast(double, partner<D>(__builtin_bit_cast(uint64_t, v)));
}
template <int L, int D = 1, typename T, typename F>
__device__ __forceinline__ T over_lanes(T v, const F& f) {
  if constexpr (D < L) return over_lanes<L, D * 2>(f(v, partner<D>(v)), f);
  else return v;
}

// The lane's experts: e0 .. e0 + n - 1 (n <= V) of the group its lane belongs to.
template <typename TIn>
__device__ __forceinline__ double logit_at(const TIn* p) {
  if constexpr (sizeof(TIn) == 2) return (double)bf16lo(*p);
  else return (double)*p;
}

struct RouteArgs {
  RouteHow how;
  int lanes_log2;  // of a group
  int per;         // experts of a group
  int wide;        // a lane's V logits can be loaded as 16-byte pieces
};

// Runs f with the number of lanes of a group as a constant.
template <int L, typename F>
__device__ __forceinline__ void with_lanes(int log2, const F& f) {
  switch (log2) {
    case 0: f(std::integral_constant<int, 1>{}); break;
    case 1: f(std::integral_constant<int, 2>{}); break;
    case 2: f(std::integral_constant<int, 4>{}); break;
    case 3: f(std::integral_constant<int, 8>{}); break;
    case 4: f(std::integral_constant<int, 16>{}); break;
    default:
      if constexpr (L == 64) {
        if (log2 == 5) f(std::integral_constant<int, 32>{});
        else f(std::integral_constant<int, 64>{});
      }
  }
}

template <typename TIn, int L, int V>
__global__ __launch_bounds__(256) void route_kernel(const TIn* __restrict__ x, int64_t T, int64_t ldx, RouteArgs a,
                                                    const float* __restrict__ bias, int32_t* __restrict__ experts,
                                                    float* __restrict__ weights) {
  const int64_t token = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
  if (token >= T) return;  // (all L lanes of a token together; the DPP patterns stay within them)
  const int lane = threadIdx.x % L;
  const TIn* xr = x + token * ldx;
  const RouteHow& how = a.how;
  const int group = lane >> a.lanes_log2, l = lane & ((1 << a.lanes_log2) - 1);
  const int first = l * V;  // within the group
  const int e0 = group * a.per + first;
  const int n = group < how.groups ? (a.per - first < V ? a.per - first : V) : 0;
  const double inf = __builtin_inf();

  double c[V];
  bool loaded = false;
  if constexpr (V * sizeof(TIn) >= 16) {
    if (a.wide) {  // (then n is V or not positive)
      loaded = true;
      constexpr int P = 16 / sizeof(TIn);
      const TIn* at = xr + (n > 0 ? e0 : 0);
#pragma unroll
      for (int j = 0; j < V; j += P) {
        const v4i w = *reinterpret_cast<const v4i*>(at + j);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          if constexpr (P == 8) c[j + i] = (double)((i & 1) ? bf16hi((uint32_t)w[i / 2]) : bf16lo((uint32_t)w[i / 2]));
          else c[j + i] = (double)__int_as_float(w[i]);
        }
      }
    }
  }
  if (!loaded) {  // (slots without an expert read another's logit)
#pragma unroll
    for (int j = 0; j < V; ++j) c[j] = logit_at(xr + (j < n ? e0 + j : 0));
  }

  // softmax of all: the largest logit and the sum of the exponentials, where they are needed
  const bool ordered = bias == nullptr && (how.groups == 1 || how.group_best == 1);  // c has the order of x
  const bool softmax = how.score == 0;
  double top = -inf, norm = 0.0;
  if (softmax && (!ordered || !how.renormalize)) {
#pragma unroll
    for (int j = 0; j < V; ++j) top = j < n && c[j] > top ? c[j] : top;
    top = over_lanes<L>(top, [](double p, double q) { return max64(p, q); });
    const double shift = top == -inf ? 0.0 : top;
    double e[V];
#pragma unroll
    for (int j = 0; j < V; ++j) e[j] = c[j] - shift;
    exp_all(e);
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) sum += j < n ? e[j] : 0.0;
    norm = over_lanes<L>(sum, [](double p, double q) { return p + q; });
    norm = norm == 0.0 ? 0.0 : 1.0 / norm;  // (every expert switched off: all scores are zero)
    if (!ordered) {
#pragma unroll
      for (int j = 0; j < V; ++j) c[j] = e[j] * norm;
    }
  } else if (!ordered) {
    sigmoid_all(c);
  }
  if (bias != nullptr) {
#pragma unroll
    for (int j = 0; j < V; ++j) c[j] += (double)bias[j < n ? e0 + j : 0];
  }
  double key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) key[j] = j < n ? key_of(c[j], e0 + j) : shut_key();

  if (how.top_groups < how.groups) {
    // (by c itself and not by its key: the sum of two keys has the indexes in it)
    double t1 = -kMostKey, t2 = -kMostKey;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const double v = j < n && c[j] > -kMostKey ? c[j] : -kMostKey;  // (NaN is below every score)
      t2 = max64(t2, min64(v, t1));
      t1 = max64(t1, v);
    }
    with_lanes<L>(a.lanes_log2, [&](auto lanes) {
      auto step = [&](auto d) {
        constexpr int D = decltype(d)::value;
        if constexpr (D < decltype(lanes)::value) {
          const double o1 = partner<D>(t1), o2 = partner<D>(t2);
          t2 = max64(max64(t2, o2), min64(t1, o1));  // one of the two seconds, or the smaller of the firsts
          t1 = max64(t1, o1);
        }
      };
      step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{});
      step(std::integral_constant<int, 4>{});
      step(std::integral_constant<int, 8>{});
      if constexpr (L == 64) {
        step(std::integral_constant<int, 16>{});
        step(std::integral_constant<int, 32>{});
      }
    });
    const double mine = key_of(how.group_best == 2 ? t1 + t2 : t1, group);
    int ahead = 0;
    for (int g = 0; g < how.groups; ++g) {
      const uint64_t b = __builtin_bit_cast(uint64_t, mine);
      const int from = g << a.lanes_log2;
      const uint64_t o = (uint64_t)(uint32_t)__shfl((int)(uint32_t)b, from, L) |
                         (uint64_t)(uint32_t)__shfl((int)(uint32_t)(b >> 32), from, L) << 32;
      ahead += __builtin_bit_cast(double, o) > mine ? 1 : 0;
    }
    if (ahead >= how.top_groups) {
#pragma unroll
      for (int j = 0; j < V; ++j) key[j] = shut_key();
    }
  }

  int chosen = 0;  // of lane r: expert r
  for (int r = 0; r < how.k; ++r) {
    double best = key[0];
#pragma unroll
    for (int j = 1; j < V; ++j) best = max64(best, key[j]);
    best = over_lanes<L>(best, [](double p, double q) { return max64(p, q); });
#pragma unroll
    for (int j = 0; j < V; ++j) {  // (the high word alone makes it one of the shut)
      const uint64_t b = __builtin_bit_cast(uint64_t, key[j]);
      const uint32_t high = key[j] == best ? kShutHigh : (uint32_t)(b >> 32);
      key[j] = __builtin_bit_cast(double, (uint64_t)high << 32 | (uint32_t)b);
    }
    if (lane == r) chosen = index_of(best);
  }

  const bool live = lane < how.k;
  const double xc = live ? logit_at(xr + chosen) : -inf;
  double w;
  if (!softmax) {
    w = live ? sigmoid64(xc) : 0.0;
  } else if (how.renormalize) {  // (the chosen ones against their own largest: the quotients are the same)
    const double m = over_lanes<L>(xc, [](double p, double q) { return p > q ? p : q; });
    w = live ? exp64(xc - (m == -inf ? 0.0 : m)) : 0.0;
  } else {
    w = live ? exp64(xc - (top == -inf ? 0.0 : top)) * norm : 0.0;
  }
  if (how.renormalize) {
    const double sum = over_lanes<L>(w, [](double p, double q) { return p + q; });
    w = sum == 0.0 ? 0.0 : w / sum;
  }
  if (live) {
    experts[token * how.k + lane] = chosen;
    weights[token * how.k + lane] = (float)(how.scale * w);
  }
}

// Gradient of the logits.  With d = scale dw of the chosen experts (zero for the others) and, where the weights are
// normalized, d' = (d - sum d w) / sum s with w = s / sum s:
//   softmax, normalized: dx = w (d - sum d w) of the chosen;   softmax: dx = s (d - sum d s), all experts;
//   sigmoid: dx = d s (1 - s) of the chosen (d' for normalized weights).
// 64 lanes a token; the row is gathered in LDS, so that it leaves whole, zeros and all.
template <typename TIn>
__global__ __launch_bounds__(256) void route_backward_kernel(const float* __restrict__ dw, const TIn* __restrict__ x, int64_t T,
                                                             int64_t ldx, RouteHow how, const int32_t* __restrict__ experts,
                                                             TIn* __restrict__ dx, int64_t lddx) {
  __shared__ float rows[4][kMaxRouteExperts];
  const int wid = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t token = (int64_t)blockIdx.x * 4 + wid;
  if (token >= T) return;  // (no barrier follows: a wave reads its own row only)
  float* row = rows[wid];
  const TIn* xr = x + token * ldx;
  const int E = how.experts, k = how.k;
  const double inf = __builtin_inf();
  const int e = lane < k ? experts[token * k + lane] : -1;
  const bool live = e >= 0 && e < E;
  const double xc = live ? logit_at(xr + e) : -inf;
  double d = live ? how.scale * (double)dw[token * k + lane] : 0.0;
  auto add = [](double p, double q) { return p + q; };
  auto most = [](double p, double q) { return p > q ? p : q; };
  double g;
  if (how.score == 0 && !how.renormalize) {
    constexpr int V = kMaxRouteExperts / 64;
    double v[V], top = -inf, sum = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = lane + 64 * j;
      v[j] = -inf;
      if (64 * j < E) v[j] = i < E ? logit_at(xr + i) : -inf;
      top = most(v[j], top);
    }
    top = over_lanes<64>(top, most);
    top = top == -inf ? 0.0 : top;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (64 * j >= E) break;
      v[j] = exp64(v[j] - top);
      sum += v[j];
    }
    sum = over_lanes<64>(sum, add);
    const double norm = sum == 0.0 ? 0.0 : 1.0 / sum;
    const double s = live ? exp64(xc - top) * norm : 0.0;
    const double mean = over_lanes<64>(d * s, add);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (64 * j >= E) break;
      row[lane + 64 * j] = (float)(-mean * v[j] * norm);
    }
    g = s * (d - mean);
  } else {
    for (int i = lane; i < E; i += 64) row[i] = 0.0f;
    if (how.score == 0) {
      double m = over_lanes<64>(xc, most);
      m = m == -inf ? 0.0 : m;
      double w = live ? exp64(xc - m) : 0.0;
      const double sum = over_lanes<64>(w, add);
      w = sum == 0.0 ? 0.0 : w / sum;
      g = w * (d - over_lanes<64>(d * w, add));
    } else {
      const double s = live ? sigmoid64(xc) : 0.0;
      if (how.renormalize) {
        const double sum = over_lanes<64>(s, add);
        const double inv = sum == 0.0 ? 0.0 : 1.0 / sum;
        d = (d - over_lanes<64>(d * s, add) * inv) * inv;
      }
      g = d * s * (1.0 - s);
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (live) row[e] = (float)g;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  TIn* out = dx + token * lddx;
  for (int i = lane; i < E; i += 64) {
    if constexpr (sizeof(TIn) == 2) out[i] = (TIn)pack_bf16x2(row[i], 0.0f);
    else out[i] = row[i];
  }
}

static int log2_up(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

template <typename TIn, int L, int V>
static hipError_t launch_route_as(const void* x, int64_t T, int64_t ldx, const RouteArgs& a, const float* bias,
                                  int32_t* experts, float* weights, hipStream_t st) {
  const int64_t blocks = (T + 256 / L - 1) / (256 / L);
  hipLaunchKernelGGL((route_kernel<TIn, L, V>), dim3((unsigned)blocks), dim3(256), 0, st, (const TIn*)x, T, ldx, a, bias,
                     experts, weights);
  return hipGetLastError();
}

template <typename TIn>
static hipError_t launch_route_t(const void* x, int64_t T, int64_t ldx, const RouteHow& how, const float* bias,
                                 int32_t* experts, float* weights, hipStream_t st) {
  // 16 lanes a token where a lane has four experts at most, or once the tokens fill the card, and where the experts fit its
  // 16 slots (us with 16 lanes and 64: 64 experts, 64 tokens 3.3 / 3.9, 16384 tokens 4.7 / 10.6; 96 experts, 2048 tokens
  // 4.2 / 3.8, 8192 tokens 5.0 / 6.4; 256 sigmoid scores in 8 groups, 64 tokens 9.3 / 5.6, 4096 9.7 / 8.5, 8192 12.0 / 13.4,
  // 16384 17.2 / 22.3).
  const int glog = log2_up(how.groups), per = how.experts / how.groups;
  const bool fits = how.k <= 16 && glog <= 4 && per <= 16 << (4 - glog);
  const bool narrow = fits && (T > 4096 || per <= 4 << (4 - glog));
  RouteArgs a{how, (narrow ? 4 : 6) - glog, per, 0};
  const int need = (per + (1 << a.lanes_log2) - 1) >> a.lanes_log2;
  const int v = 1 << log2_up(need);
  a.wide = per % v == 0 && ((uintptr_t)x & 15) == 0 && ldx * (int64_t)sizeof(TIn) % 16 == 0 && v * sizeof(TIn) >= 16;
#define FP8BQ_ROUTE(L, V) \
  case V: return launch_route_as<TIn, L, V>(x, T, ldx, a, bias, experts, weights, st);
  if (narrow) {
    switch (v) { FP8BQ_ROUTE(16, 1) FP8BQ_ROUTE(16, 2) FP8BQ_ROUTE(16, 4) FP8BQ_ROUTE(16, 8) FP8BQ_ROUTE(16, 16) }
  } else {
    switch (v) { FP8BQ_ROUTE(64, 1) FP8BQ_ROUTE(64, 2) FP8BQ_ROUTE(64, 4) FP8BQ_ROUTE(64, 8) FP8BQ_ROUTE(64, 16) }
  }
#undef FP8BQ_ROUTE
  return hipErrorInvalidValue;
}

// Tokens of one launch: at 64 threads each, its threads stay below 2^32.
constexpr int64_t kLaunchTokens = (int64_t)1 << 24;

hipError_t launch_route(const void* x, int xt, int64_t T, int64_t ldx, const RouteHow& how, const float* bias,
                        int32_t* experts, float* weights, hipStream_t st) {
  for (int64_t t = 0; t < T; t += kLaunchTokens) {
    const int64_t n = T - t < kLaunchTokens ? T - t : kLaunchTokens;
    const hipError_t e =
        xt == 0 ? launch_route_t<uint16_t>((const uint16_t*)x + t * ldx, n, ldx, how, bias, experts + t * how.k, weights + t * how.k, st)
                : launch_route_t<float>((const float*)x + t * ldx, n, ldx, how, bias, experts + t * how.k, weights + t * how.k, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_route_backward(const float* dw, const void* x, int xt, int64_t T, int64_t ldx, const RouteHow& how,
                                 const int32_t* experts, void* dx, int64_t lddx, hipStream_t st) {
  for (int64_t t = 0; t < T; t += kLaunchTokens) {
    const int64_t n = T - t < kLaunchTokens ? T - t : kLaunchTokens;
    const dim3 grid((unsigned)((n + 3) / 4)), block(256);
    if (xt == 0)
      hipLaunchKernelGGL(route_backward_kernel<uint16_t>, grid, block, 0, st, dw + t * how.k, (const uint16_t*)x + t * ldx, n, ldx,
                         how, experts + t * how.k, (uint16_t*)dx + t * lddx, lddx);
    else
      hipLaunchKernelGGL(route_backward_kernel<float>, grid, block, 0, st, dw + t * how.k, (const float*)x + t * ldx, n, ldx, how,
                         experts + t * how.k, (float*)dx + t * lddx, lddx);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fp8bq
