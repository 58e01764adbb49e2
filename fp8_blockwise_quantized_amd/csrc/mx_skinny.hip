// MXFP4 product for up to 16 rows of A (tokens) a product: C[m, n] = sum_k A[m, k] B[n, k].
//
// For few column tiles, where one pass's latency counts (one token through 11264 x 2048: 5.6 us with the
// quantization, 4.7 us from codes, most of it launch, first loads and the joining of sums; 12 MB of weights
// at the copy's rate would take 2 us).  From about 1500 column tiles on the LDS-tiled kernel streams the
// weights faster, whatever the rows (45056 x 2048, one row: 10.1 us there, 11.5 us here).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes B as its first operand: lane l holds block l / 16 of row l % 16 of both
// operands (16 bytes of codes, one scale byte), straight from memory, and ends with C row l % 16 and columns
// 4 (l / 16) .. +3.  A wave owns 16 columns and reads 256 values of its B rows (128-byte lines) at a time; the KS
// waves that share them split the contraction, so that every load of a workgroup is in flight at once, and
// join their FP32 sums in LDS in wave order.
//
// FUSED (A in BF16 or FP32): the 32 values of a lane's operand are exactly one block, so each lane quantizes the
// block it needs itself, without another lane and without a launch of its own, while the weights are on
// their way.  Every column tile repeats that work, so it is taken for few tiles and rows only (plan_mx).
#include "group_table.hpp"
#include "launch.hpp"
#include "mx_common.hpp"
#include "quant_common.hpp"

namespace fp8bq {

constexpr int kSkinnyWaves = 8;

// The lane's block of A on its way to an operand: load() issues the reads, get() gives codes and scale byte
// (zeros where the row or the block does not exist).
template <typename TA>
struct MxBlockOf;
template <>
struct MxBlockOf<uint8_t> {  // quantized before
  v4i c;
  uint32_t w;
  __device__ __forceinline__ void load(const MxDesc& d, int64_t m, int64_t blk, bool valid) {
    c = (v4i){0, 0, 0, 0};
    w = 0;
    if (valid) {
      c = *reinterpret_cast<const v4i*>(reinterpret_cast<const uint8_t*>(d.a) + m * d.lda + blk * 16);
      w = d.sa[(blk >> 2) * d.ldsa + m] >> (8 * (blk & 3));
    }
  }
  __device__ __forceinline__ void get(v4i& codes, int& scale) const {
    codes = c;
    scale = (int)w;
  }
};
template <>
struct MxBlockOf<uint16_t> {  // BF16
  u32x4 w[4];
  __device__ __forceinline__ void load(const MxDesc& d, int64_t m, int64_t blk, bool valid) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (u32x4){0, 0, 0, 0};
    if (valid) {
      const u32x4* p = reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(d.a) + m * d.lda + blk * kMxBlock);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = p[i];
    }
  }
  __device__ __forceinline__ void get(v4i& codes, int& scale) {
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) m2 = pk_umax16(m2, w[i][j] & 0x7FFF7FFFu);
    const uint32_t m = umax(m2 & 0xFFFFu, m2 >> 16) << 16;
    const uint32_t b = mx_scale_byte(m);
    if (b == 0u && m != 0u) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) w[i][j] = mx_lift_bf16(w[i][j]);
    }
    const float sc = mx_scale_of(b);
#pragma unroll
    for (int i = 0; i < 4; ++i) codes[i] = (int)mx_pack8_bf16(w[i][0], w[i][1], w[i][2], w[i][3], sc);
    scale = (int)b;
  }
};
template <>
struct MxBlockOf<float> {
  float v[4][8];
  __device__ __forceinline__ void load(const MxDesc& d, int64_t m, int64_t blk, bool valid) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    if (valid) {
      const float* p = reinterpret_cast<const float*>(d.a) + m * d.lda + blk * kMxBlock;
#pragma unroll
      for (int i = 0; i < 4; ++i) Load8<float>::run(p + 8 * i, v[i]);
    }
  }
  __device__ __forceinline__ void get(v4i& codes, int& scale) {
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

// ks: waves that split the contraction (a power of two up to 8).
template <typename TA, int OUT, bool GROUPED>
__global__ __launch_bounds__(kSkinnyWaves * 64, 4) void mx_skinny_kernel(MxDesc d, MxGroups grp, int ks) {
  __shared__ float part[kSkinnyWaves][4][64];
  __shared__ int starts[GROUPED ? kMaxExperts + 1 : 1];
  __shared__ uint32_t units[GROUPED ? kMaxExperts + 1 : 1];
  const int t = threadIdx.x, lane = t & 63;
  const int wid = __builtin_amdgcn_readfirstlane(t >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int phase = wid & (ks - 1);
  const int cols = kSkinnyWaves / ks * 16;  // of the workgroup
  const uint32_t tiles_n = (uint32_t)((d.N + cols - 1) / cols);
  const int64_t nblk = d.K / kMxBlock;

  uint32_t total;
  if constexpr (GROUPED) {
    if (wid == 0) group_table_rows(grp.offsets, grp.experts, d.M, 16, tiles_n, starts, units, lane);
    __syncthreads();
    total = units[grp.experts];
  } else {
    total = tiles_n * (uint32_t)((d.M + 15) / 16);
  }

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
    const int64_t m = m0 + (int64_t)(w / tiles_n) * 16 + r16;
    const int64_t nt = (int64_t)(w % tiles_n) * cols + wid / ks * 16;  // the wave's first column
    const int64_t row = nbase + (nt + r16 < d.N ? nt + r16 : d.N - 1);
    const uint8_t* brow = d.b + row * d.ldb;
    const uint32_t* bscale = d.sb + row;

    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
    if (nt < d.N) {
      for (int64_t k8 = (int64_t)phase * 8; k8 < nblk; k8 += ks * 8) {  // 8 blocks: two MFMA steps
        // A's reads first: memory answers in order, and quantizing can then begin before B is there
        MxBlockOf<TA> a[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t blk = k8 + 4 * h + g;
          a[h].load(d, m, blk, m < mend && blk < nblk);
        }
        v4i bc[2];
        int bs[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t blk = k8 + 4 * h + g;
          const int64_t at = blk < nblk ? blk : nblk - 1;
          bc[h] = *reinterpret_cast<const v4i*>(brow + at * 16);
          bs[h] = (int)bscale[(at >> 2) * d.ldsb];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t blk = k8 + 4 * h + g;
          v4i ac;
          int as;
          a[h].get(ac, as);
          acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(bc[h]), mx_operand(ac), acc, 4, 4, 0,
                                                                 blk < nblk ? bs[h] >> (8 * (blk & 3)) : 0, 0, as);
        }
      }
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
    if (phase == 0 && m < mend && nt < d.N) mx_store4<OUT>(d.c, d.ldc, m, nt + 4 * g, d.N, acc);
  }
}

template <typename TA, int OUT, bool GROUPED>
static hipError_t launch_one(const MxDesc& d, const MxGroups& grp, const MxPlan& p, hipStream_t st) {
  hipLaunchKernelGGL((mx_skinny_kernel<TA, OUT, GROUPED>), dim3((unsigned)p.grid), dim3(kSkinnyWaves * 64), 0, st, d, grp,
                     p.split_k);
  return hipGetLastError();
}

template <typename TA>
static hipError_t launch_out(const MxDesc& d, const MxGroups& grp, const MxPlan& p, hipStream_t st) {
  if (grp.offsets) return d.out_t == 0 ? launch_one<TA, 0, true>(d, grp, p, st) : launch_one<TA, 1, true>(d, grp, p, st);
  if constexpr (std::is_same_v<TA, uint8_t>) {  // (only the dense product of codes is added to the output)
    if (d.out_t == 2) return launch_one<TA, 2, false>(d, grp, p, st);
  }
  return d.out_t == 0 ? launch_one<TA, 0, false>(d, grp, p, st) : launch_one<TA, 1, false>(d, grp, p, st);
}

hipError_t launch_mx_skinny(const MxDesc& d, const MxGroups& grp, const MxPlan& p, hipStream_t st) {
  if (d.a_type == kMxCodes) return launch_out<uint8_t>(d, grp, p, st);
  return d.a_type == kMxBf16 ? launch_out<uint16_t>(d, grp, p, st) : launch_out<float>(d, grp, p, st);
}

}  // namespace fp8bq
