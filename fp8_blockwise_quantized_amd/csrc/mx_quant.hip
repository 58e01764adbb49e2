// MXFP4 quantizer: row blocks (32 consecutive elements of a row), column blocks (32 consecutive rows of a
// column, outputs transposed so that the contraction is contiguous), or both from one read.
//
// Bound by HBM: 2 (BF16) or 4 (FP32) bytes read and 0.53 written per element and layout.  A workgroup of
// four waves owns a tile of 128 rows by 128 columns; a wave holds 32 rows of it, a thread a patch of 8 rows by
// 8 columns (eight independent 16-byte loads of BF16).  A row block is then 4 neighbouring lanes (two DPP
// exchanges) and a column block the 4 lanes of the wave that are 16 apart, so neither maximum needs LDS or a
// barrier; only the transposed codes are staged in LDS, for stores of 64 contiguous bytes per column.
#include "launch.hpp"
#include "mx_common.hpp"
#include "quant_common.hpp"

namespace fp8bq {

// Largest of the value and those of the lanes 16, 32 and 48 away (the wave's other row groups).
__device__ __forceinline__ uint32_t column_max(uint32_t v) {
  v = umax(v, (uint32_t)__shfl_xor((int)v, 16));
  return umax(v, (uint32_t)__shfl_xor((int)v, 32));
}

// Staged codes of column c: 64 bytes (four 32-row blocks of 16), the 16-byte units XORed by the column so
// that the 16 columns one store instruction writes spread over the banks.
__device__ __forceinline__ int mx_stage(int c, int unit) { return 64 * c + 16 * (unit ^ ((c >> 3) & 3)); }

template <typename TIn, bool ROWS, bool COLS>
__global__ __launch_bounds__(256) void mx_quant_kernel(const TIn* __restrict__ x, int64_t R, int64_t C, int64_t ldx,
                                                       uint8_t* __restrict__ q, int64_t ldq,
                                                       uint32_t* __restrict__ s, int64_t lds,
                                                       uint8_t* __restrict__ qt, int64_t ldqt,
                                                       uint32_t* __restrict__ st, int64_t ldst, uint32_t ncg) {
  __shared__ __attribute__((aligned(16))) uint8_t codes[COLS ? 128 * 64 : 16];
  __shared__ uint8_t scales[COLS ? 128 * 4 : 4];

  const int t = threadIdx.x;
  const int wid = t >> 6;
  const int cc = t & 15;        // 8-column chunk of the tile
  const int rg = (t >> 4) & 3;  // 8-row group of the wave's 32 rows
  const TileRC tile = tile_of_block(ncg);
  const int64_t r0 = tile.row * 128 + 32 * wid + 8 * rg;
  const int64_t col = tile.col * 128 + 8 * cc;
  const bool cvalid = col < C;  // C % 8 == 0: a chunk is all in or all out

  float v[8][8];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    if (cvalid && r0 + p < R) {
      Load8<TIn>::run(x + (r0 + p) * ldx + col, v[p]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[p][i] = 0.0f;
    }
  }

  if constexpr (ROWS) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      uint32_t m = mx_abs_bits(v[p][0]);
#pragma unroll
      for (int i = 1; i < 8; ++i) m = umax(m, mx_abs_bits(v[p][i]));
      m = umax_partner<kDppXor1>(m, m);
      m = umax_partner<kDppXor2>(m, m);
      const uint32_t b = mx_scale_byte(m);
      const float inv = mx_inverse(b);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = v[p][i] * inv;
      if (cvalid && r0 + p < R) *reinterpret_cast<uint32_t*>(q + (r0 + p) * ldq + col / 2) = mx_pack8(y);
      // the word of the row's four blocks, from lanes 0, 4, 8 and 12 of the 16
      const uint32_t w = dpp_read<0x150>(b) | dpp_read<0x154>(b) << 8 | dpp_read<0x158>(b) << 16 | dpp_read<0x15C>(b) << 24;
      if (cc == 0 && r0 + p < R) s[tile.col * lds + r0 + p] = w;
    }
  }

  if constexpr (COLS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = mx_abs_bits(v[0][i]);
#pragma unroll
      for (int p = 1; p < 8; ++p) m = umax(m, mx_abs_bits(v[p][i]));
      m = column_max(m);
      const uint32_t b = mx_scale_byte(m);
      const float inv = mx_inverse(b);
      float y[8];
#pragma unroll
      for (int p = 0; p < 8; ++p) y[p] = v[p][i] * inv;
      const int c = 8 * cc + i;
      *reinterpret_cast<uint32_t*>(codes + mx_stage(c, wid) + 4 * rg) = mx_pack8(y);
      if (rg == 0) scales[4 * c + wid] = (uint8_t)b;
    }
    __syncthreads();
    const int64_t rows32 = (R + 31) / 32;  // 32-row blocks of a column that exist
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      const int c = (t >> 2) + 64 * pass, unit = t & 3;
      if (tile.col * 128 + c < C && tile.row * 4 + unit < rows32)
        store_codes16(qt + (tile.col * 128 + c) * ldqt + (tile.row * 4 + unit) * 16,
                      *reinterpret_cast<const uint4*>(codes + mx_stage(c, unit)));
    }
    if (t < 128 && tile.col * 128 + t < C)
      st[tile.row * ldst + tile.col * 128 + t] = *reinterpret_cast<const uint32_t*>(scales + 4 * t);
  }
}

template <typename TIn>
static hipError_t launch_in(const void* x, int64_t R, int64_t C, int64_t ldx, uint8_t* q, int64_t ldq, uint32_t* s,
                            int64_t lds, uint8_t* qt, int64_t ldqt, uint32_t* st_, int64_t ldst, hipStream_t st) {
  const uint32_t ncg = (uint32_t)((C + 127) / 128);
  const dim3 grid((unsigned)((R + 127) / 128) * ncg);
  if (q && qt)
    hipLaunchKernelGGL((mx_quant_kernel<TIn, true, true>), grid, dim3(256), 0, st, (const TIn*)x, R, C, ldx, q, ldq, s,
                       lds, qt, ldqt, st_, ldst, ncg);
  else if (q)
    hipLaunchKernelGGL((mx_quant_kernel<TIn, true, false>), grid, dim3(256), 0, st, (const TIn*)x, R, C, ldx, q, ldq,
                       s, lds, qt, ldqt, st_, ldst, ncg);
  else
    hipLaunchKernelGGL((mx_quant_kernel<TIn, false, true>), grid, dim3(256), 0, st, (const TIn*)x, R, C, ldx, q, ldq,
                       s, lds, qt, ldqt, st_, ldst, ncg);
  return hipGetLastError();
}

hipError_t launch_mx_quant(const void* x, int xt, int64_t R, int64_t C, int64_t ldx, uint8_t* q, int64_t ldq,
                           uint32_t* s, int64_t lds, uint8_t* qt, int64_t ldqt, uint32_t* st_, int64_t ldst,
                           hipStream_t st) {
  return xt == 0 ? launch_in<uint16_t>(x, R, C, ldx, q, ldq, s, lds, qt, ldqt, st_, ldst, st)
                 : launch_in<float>(x, R, C, ldx, q, ldq, s, lds, qt, ldqt, st_, ldst, st);
}

}  // namespace fp8bq
