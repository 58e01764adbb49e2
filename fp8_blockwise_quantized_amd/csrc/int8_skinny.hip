// 8-bit integer product for up to 16 rows of A (tokens) a product: C[m, n] = sa[m] sb[n] sum_k A[m, k] B[n, k].
//
// Bound by the weights' bytes, and where those are few by one pass's latency.  v_mfma_i32_16x16x64_i8 takes B as its
// first operand: lane l holds 16 contraction bytes of row l % 16 of both operands, straight from memory, and ends with
// C row l % 16 and columns 4 (l / 16) .. +3.  A wave owns 16 columns and reads 128 bytes of each of its B rows at a
// time; the waves that share them split the contraction and join their integer sums in LDS.
//
// A in BF16 or FP32, few values of it and one product: the workgroup quantizes the rows itself, into LDS (the scale needs
// the whole row, so all its threads look for the maxima first), while its first weights are on their way.  That is spared
// a launch, and costs every workgroup about 0.3 us for 4096 values.
//
// Measured (us, weights in the caches; an empty launch takes 2): one row, 2048 x 2048 from codes 3.9, from BF16 5.1;
// 11264 x 2048 6.4 and 7.8 (3.6 and 3.0 TB/s); 16 rows, 2048 x 2048 4.5.  Codes and scales are asked for with the weights,
// ahead of the products (behind them one row of 11264 x 2048 took 7.6), and registers are kept for three workgroups a
// compute unit (from BF16 9.2 with two).
#include "group_table.hpp"
#include "int8_common.hpp"
#include "launch.hpp"

namespace fp8bq {

constexpr int kSkinnyWaves = 8;
constexpr int kSkinnyThreads = kSkinnyWaves * 64;

template <int OUT>
__device__ __forceinline__ void int8_store4(void* c, int64_t ldc, int64_t m, int64_t n, int64_t nend, v4f v) {
  if constexpr (OUT == 0) {
    uint16_t* p = reinterpret_cast<uint16_t*>(c) + m * ldc + n;
    const uint32_t lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
    if (n + 4 <= nend && (((uintptr_t)p) & 7) == 0) {
      *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
    } else {
      const uint16_t e[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < nend) p[i] = e[i];
    }
  } else {
    float* p = reinterpret_cast<float*>(c) + m * ldc + n;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < nend) p[i] = OUT == 2 ? p[i] + v[i] : v[i];
  }
}

// LDS of quantized rows: `rows` (a power of two) of K codes, 16 bytes apart beyond that so that the 16 rows of an
// operand read fall on different banks.
__host__ __device__ inline int64_t skinny_row_bytes(int64_t K) { return (K + 127) / 128 * 128 + 16; }

// Codes and scales of the first `rows` rows (zeros from M on), all threads of the workgroup.
template <typename TA>
__device__ __forceinline__ void quantize_rows(const Int8Desc& d, int rows, uint8_t* qx, float* rs, uint32_t* amax) {
  const int t = threadIdx.x, tpr = kSkinnyThreads / rows, row = t / tpr, c0 = 8 * (t % tpr);
  const int64_t rb = skinny_row_bytes(d.K);
  const bool live = row < d.M;
  const TA* x = reinterpret_cast<const TA*>(d.a) + (live ? row : 0) * d.lda;
  if (t < 16) amax[t] = 0;
  __syncthreads();
  uint32_t a = 0;
  if (live)
    for (int64_t k = c0; k < d.K; k += 8 * tpr) {
      float v[8];
      Load8<TA>::run(x + k, v);
      a = amax8(v, a);
    }
  a = row16_umax(a);  // (16 lanes or more share a row)
  if ((t & 15) == 0) atomicMax(&amax[row], a);
  __syncthreads();
  const float s = int8_scale(amax[row]), r = 1.0f / s;
  for (int64_t k = c0; k < rb - 16; k += 8 * tpr) {
    uint2 w = make_uint2(0, 0);
    if (live && k < d.K) {
      float v[8];
      Load8<TA>::run(x + k, v);
      w = int8_quant8(v, s, r);
    }
    *reinterpret_cast<uint2*>(qx + row * rb + k) = w;
  }
  if (t % tpr == 0) rs[row] = s;
  __syncthreads();
}

// ks: waves that split the contraction (a power of two up to 8); rows: of A in LDS (unused with codes).
template <typename TA, int OUT, bool GROUPED>
__global__ __launch_bounds__(kSkinnyThreads, 6) void int8_skinny_kernel(Int8Desc d, MxGroups grp, int ks, int rows) {
  extern __shared__ __attribute__((aligned(16))) uint8_t qx[];
  __shared__ int part[kSkinnyWaves][4][64];
  __shared__ float rs[16];
  __shared__ uint32_t amax[16];
  __shared__ int starts[GROUPED ? kMaxExperts + 1 : 1];
  __shared__ uint32_t units[GROUPED ? kMaxExperts + 1 : 1];
  constexpr bool FUSED = !std::is_same_v<TA, uint8_t>;
  const int t = threadIdx.x, lane = t & 63;
  const int wid = __builtin_amdgcn_readfirstlane(t >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int phase = wid & (ks - 1);
  const int cols = kSkinnyWaves / ks * 16;  // of the workgroup
  const uint32_t tiles_n = (uint32_t)((d.N + cols - 1) / cols);
  const int64_t rb = skinny_row_bytes(d.K);

  uint32_t total;
  if constexpr (GROUPED) {
    if (wid == 0) group_table_rows(grp.offsets, grp.experts, d.M, 16, tiles_n, starts, units, lane);
    __syncthreads();
    total = units[grp.experts];
  } else {
    total = tiles_n * (uint32_t)((d.M + 15) / 16);
  }

  bool held = false;  // the rows' codes are in LDS
  for (uint32_t u = blockIdx.x; u < total; u += gridDim.x) {
    int64_t m0 = 0, mend = d.M, nbase = 0;
    uint32_t w = u;
    if constexpr (GROUPED) {
      const int e = group_find(units, grp.experts, u, lane);
      w = u - units[e];
      m0 = starts[e];
      mend = starts[e + 1];
      nbase = (int64_t)e * d.N;
    }
    m0 += (int64_t)(w / tiles_n) * 16;
    const int64_t m = m0 + r16;
    const int64_t nt = (int64_t)(w % tiles_n) * cols + wid / ks * 16;  // the wave's first column
    const uint8_t* brow = d.b + (nbase + (nt + r16 < d.N ? nt + r16 : d.N - 1)) * d.ldb;
    auto bload = [&](int64_t k) { return *reinterpret_cast<const v4i*>(brow + (k < d.K ? k : d.K - 16)); };
    const int64_t k0 = (int64_t)phase * 128 + 16 * g, step = (int64_t)ks * 128;
    v4i b[2] = {bload(k0), bload(k0 + 64)};
    const bool mine = m < mend;
    const uint8_t* arow = reinterpret_cast<const uint8_t*>(d.a) + (mine ? m : mend - 1) * d.lda;  // (codes)
    auto aload = [&](int64_t k) { return *reinterpret_cast<const v4i*>(arow + (k < d.K ? k : d.K - 16)); };
    v4i ca[2];
    float sa = 0.0f, sb[4];
    if constexpr (!FUSED) {
      ca[0] = aload(k0);
      ca[1] = aload(k0 + 64);
      sa = d.sa[mine ? m : mend - 1];
    }
    if constexpr (FUSED) {
      if (!held) quantize_rows<TA>(d, rows, qx, rs, amax);
      held = true;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {  // (here, so that the end does not wait for them)
      const int64_t n = nt + 4 * g + r;
      sb[r] = d.sb[nbase + (n < d.N ? n : d.N - 1)];
    }
    v4i acc = {0, 0, 0, 0};
    for (int64_t k = k0; k - 16 * g < d.K; k += step) {
      const v4i b0 = b[0], b1 = b[1];
      b[0] = bload(k + step);
      b[1] = bload(k + step + 64);
      v4i a[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t at = k + 64 * h;
        a[h] = (v4i){0, 0, 0, 0};
        if constexpr (FUSED) {
          if (r16 < rows) a[h] = *reinterpret_cast<const v4i*>(qx + r16 * rb + at);  // (zeros from K on)
        } else {
          if (at < d.K) a[h] = ca[h];
          ca[h] = aload(at + step);
        }
      }
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(b0, a[0], acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(b1, a[1], acc, 0, 0, 0);
    }
    if (ks > 1) {
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wid][r][lane] = acc[r];
      __syncthreads();
      if (phase == 0) {
        for (int k = 1; k < ks; ++k)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[r] += part[wid + k][r][lane];
      }
      __syncthreads();
    }
    if (phase == 0 && mine && nt < d.N) {
      if constexpr (FUSED) sa = rs[r16];
      v4f y;
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = (float)acc[r] * sa * sb[r];
      int8_store4<OUT>(d.c, d.ldc, m, nt + 4 * g, d.N, y);
    }
  }
}

template <typename TA, int OUT, bool GROUPED>
static hipError_t launch_one(const Int8Desc& d, const MxGroups& grp, const MxPlan& p, hipStream_t st) {
  int rows = 1;
  size_t lds = 0;
  if constexpr (!std::is_same_v<TA, uint8_t>) {
    while (rows < d.M) rows *= 2;
    lds = (size_t)rows * (size_t)skinny_row_bytes(d.K);
  }
  hipLaunchKernelGGL((int8_skinny_kernel<TA, OUT, GROUPED>), dim3((unsigned)p.grid), dim3(kSkinnyThreads), lds, st, d, grp,
                     p.split_k, rows);
  return hipGetLastError();
}

template <typename TA>
static hipError_t launch_out(const Int8Desc& d, const MxGroups& grp, const MxPlan& p, hipStream_t st) {
  if constexpr (std::is_same_v<TA, uint8_t>) {  // (what is quantized here is dense and not added to the output)
    if (grp.offsets) return d.out_t == 0 ? launch_one<TA, 0, true>(d, grp, p, st) : launch_one<TA, 1, true>(d, grp, p, st);
    if (d.out_t == 2) return launch_one<TA, 2, false>(d, grp, p, st);
  }
  return d.out_t == 0 ? launch_one<TA, 0, false>(d, grp, p, st) : launch_one<TA, 1, false>(d, grp, p, st);
}

hipError_t launch_int8_skinny(const Int8Desc& d, const MxGroups& grp, const MxPlan& p, hipStream_t st) {
  if (d.a_type == kMxCodes) return launch_out<uint8_t>(d, grp, p, st);
  return d.a_type == kMxBf16 ? launch_out<uint16_t>(d, grp, p, st) : launch_out<float>(d, grp, p, st);
}

}  // namespace fp8bq
