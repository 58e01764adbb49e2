// MXFP4 product for few rows of A (tokens): C[m, n] = sum_k A[m, k] B[n, k], B (the weights) streamed once.
//
// Bound by the weights' bytes (0.53 per weight) and, at the smallest sizes, by the latency of one pass.  A
// workgroup owns 16 columns n (rows of B) and up to 16 MC rows of A; its eight waves split the contraction in
// pieces of 256 (a 128-byte line of every B row), so all of a workgroup's loads are in flight at once, and
// join their FP32 sums in LDS in wave order.  v_mfma_scale_f32_16x16x128_f8f6f4 takes B as its first operand:
// lane l holds block l / 16 of row l % 16 of both operands (16 bytes of codes, one scale byte), straight from
// memory, and ends with C row l % 16 and columns 4 (l / 16) .. +3.
//
// FUSED: A comes as BF16 or FP32 and each lane quantizes the block it needs itself: the 32 values of its MFMA
// operand are exactly one block, so the maximum needs no other lane and no separate launch is paid.
#include "group_table.hpp"
#include "launch.hpp"
#include "mx_common.hpp"
#include "quant_common.hpp"

namespace fp8bq {

constexpr int kSkinnyWaves = 8;

// The lane's block of A: codes and scale byte (zeros where the row or the block does not exist).
template <typename TA>
struct MxBlockOf {  // TA = uint16_t (BF16) or float: quantized here
  static __device__ __forceinline__ void run(const MxDesc& d, int64_t m, int64_t blk, bool valid, v4i& codes,
                                             int& scale) {
    codes = (v4i){0, 0, 0, 0};
    scale = 0;
    if (!valid) return;
    const TA* p = reinterpret_cast<const TA*>(d.a) + m * d.lda + blk * kMxBlock;
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) Load8<TA>::run(p + 8 * i, v[i]);
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) mx = umax(mx, mx_abs_bits(v[i][j]));
    const uint32_t b = mx_scale_byte(mx);
    const float inv = mx_inverse(b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= inv;
      codes[i] = (int)mx_pack8(v[i]);
    }
    scale = (int)b;
  }
};
template <>
struct MxBlockOf<uint8_t> {  // quantized before
  static __device__ __forceinline__ void run(const MxDesc& d, int64_t m, int64_t blk, bool valid, v4i& codes,
                                             int& scale) {
    codes = (v4i){0, 0, 0, 0};
    scale = 0;
    if (!valid) return;
    codes = *reinterpret_cast<const v4i*>(reinterpret_cast<const uint8_t*>(d.a) + m * d.lda + blk * 16);
    scale = (int)(d.sa[(blk >> 2) * d.ldsa + m] >> (8 * (blk & 3)));
  }
};

// Stores up to four consecutive columns of one row (v), n .. n+3, those below nend.
template <int OUT>
__device__ __forceinline__ void mx_store4(void* c, int64_t ldc, int64_t m, int64_t n, int64_t nend, v4f v) {
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

template <typename TA, int MC, int OUT, bool GROUPED>
__global__ __launch_bounds__(kSkinnyWaves * 64) void mx_skinny_kernel(MxDesc d, MxGroups grp) {
  __shared__ float part[kSkinnyWaves][MC][4][64];
  __shared__ int starts[GROUPED ? kMaxExperts + 1 : 1];
  __shared__ uint32_t units[GROUPED ? kMaxExperts + 1 : 1];
  const int t = threadIdx.x, lane = t & 63;
  const int wid = __builtin_amdgcn_readfirstlane(t >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const uint32_t tiles_n = (uint32_t)((d.N + 15) / 16);
  const int64_t nblk = d.K / kMxBlock;

  uint32_t total;
  if constexpr (GROUPED) {
    if (wid == 0) group_table_rows(grp.offsets, grp.experts, d.M, 16 * MC, tiles_n, starts, units, lane);
    __syncthreads();
    total = units[grp.experts];
  } else {
    total = tiles_n * (uint32_t)((d.M + 16 * MC - 1) / (16 * MC));
  }

  for (uint32_t u = blockIdx.x; u < total; u += gridDim.x) {
    int64_t m0, mend, nbase = 0;
    uint32_t w = u;
    if constexpr (GROUPED) {
      const int e = group_find(units, grp.experts, u, lane);
      w = u - units[e];
      m0 = starts[e];
      mend = starts[e + 1];
      nbase = (int64_t)e * d.N;
    } else {
      m0 = 0;
      mend = d.M;
    }
    m0 += (int64_t)(w / tiles_n) * (16 * MC);
    const int64_t nt = (int64_t)(w % tiles_n) * 16;  // first column within the expert's N
    const int64_t nrow = nt + r16 < d.N ? nt + r16 : d.N - 1;
    const uint8_t* brow = d.b + (nbase + nrow) * d.ldb;
    const uint32_t* bscale = d.sb + nbase + nrow;

    v4f acc[MC];
#pragma unroll
    for (int i = 0; i < MC; ++i) acc[i] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t k8 = (int64_t)wid * 8; k8 < nblk; k8 += kSkinnyWaves * 8) {  // 8 blocks: two MFMA steps
      v4i bc[2];
      int bs[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t blk = k8 + 4 * h + g;
        const bool valid = blk < nblk;
        const int64_t at = valid ? blk : nblk - 1;
        bc[h] = *reinterpret_cast<const v4i*>(brow + at * 16);
        bs[h] = valid ? (int)(bscale[(at >> 2) * d.ldsb] >> (8 * (at & 3))) : 0;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t blk = k8 + 4 * h + g;
#pragma unroll
        for (int i = 0; i < MC; ++i) {
          const int64_t m = m0 + 16 * i + r16;
          v4i ac;
          int as;
          MxBlockOf<TA>::run(d, m, blk, m < mend && blk < nblk, ac, as);
          acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(bc[h]), mx_operand(ac), acc[i], 4, 4, 0,
                                                                    bs[h], 0, as);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MC; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wid][i][r][lane] = acc[i][r];
    __syncthreads();
    if (wid < MC) {
      v4f sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < kSkinnyWaves; ++k)
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[r] += part[k][wid][r][lane];
      const int64_t m = m0 + 16 * wid + r16;
      if (m < mend) mx_store4<OUT>(d.c, d.ldc, m, nt + 4 * g, d.N, sum);
    }
    __syncthreads();
  }
}

template <typename TA, int MC, int OUT>
static hipError_t launch_mc(const MxDesc& d, const MxGroups& grp, int cus, hipStream_t st) {
  const int64_t tiles_n = (d.N + 15) / 16;
  if (grp.offsets) {
    const int64_t most = (d.M / (16 * MC) + (grp.experts < d.M ? grp.experts : d.M)) * tiles_n;
    const int64_t g = most < 16 * (int64_t)cus ? most : 16 * (int64_t)cus;
    hipLaunchKernelGGL((mx_skinny_kernel<TA, MC, OUT, true>), dim3((unsigned)g), dim3(kSkinnyWaves * 64), 0, st, d,
                       grp);
  } else {
    const int64_t all = (d.M + 16 * MC - 1) / (16 * MC) * tiles_n;
    const int64_t g = all < 65536 ? all : 65536;
    hipLaunchKernelGGL((mx_skinny_kernel<TA, MC, OUT, false>), dim3((unsigned)g), dim3(kSkinnyWaves * 64), 0, st, d,
                       grp);
  }
  return hipGetLastError();
}

template <typename TA, int OUT>
static hipError_t launch_a(const MxDesc& d, const MxGroups& grp, int64_t rows, int cus, hipStream_t st) {
  if (rows <= 16) return launch_mc<TA, 1, OUT>(d, grp, cus, st);
  if (rows <= 32) return launch_mc<TA, 2, OUT>(d, grp, cus, st);
  return launch_mc<TA, 4, OUT>(d, grp, cus, st);
}

template <typename TA>
static hipError_t launch_out(const MxDesc& d, const MxGroups& grp, int64_t rows, int cus, hipStream_t st) {
  if (d.out_t == 0) return launch_a<TA, 0>(d, grp, rows, cus, st);
  if (d.out_t == 1) return launch_a<TA, 1>(d, grp, rows, cus, st);
  return launch_a<TA, 2>(d, grp, rows, cus, st);
}

hipError_t launch_mx_skinny(const MxDesc& d, const MxGroups& grp, int64_t rows, int cus, hipStream_t st) {
  if (d.a_type == kMxCodes) return launch_out<uint8_t>(d, grp, rows, cus, st);
  return d.a_type == kMxBf16 ? launch_out<uint16_t>(d, grp, rows, cus, st) : launch_out<float>(d, grp, rows, cus, st);
}

}  // namespace fp8bq
