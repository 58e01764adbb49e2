// Token-axis quantizer of the products grouped by expert, with the row quantizer from the same read.
//
// wgrad contracts over the tokens of one expert, so its 128-token groups must begin at the expert's
// first token.  Expert e's tokens are laid out from block P[e] on, P[e+1] = P[e] + ceil(n_e / 128): the
// last block's missing tokens are zero codes, which add nothing.  Codes and scales are those of the
// 128x1 quantizer on the expert's rows padded with zeros, and of the 1x128 quantizer, bit for bit.
//
// Bound by HBM (2 bytes read and 1 or 2 written per element): 32768 x 2048 tokens on 32 experts take 55 us both
// ways (4.9 TB/s of 6.05 that a copy of 1 GiB reaches; the experts' padding adds 6%), 32768 x 1408 down the columns
// alone 25 us from the Infinity Cache and 32 us from HBM.  A workgroup owns one 128-column group
// and walks the 128-token blocks with a stride, so the table of experts is built once per workgroup and
// not once per block.  Thread mapping and LDS layouts are those of the dense dual quantizer.
#include "group_table.hpp"
#include "launch.hpp"
#include "quant_common.hpp"

namespace fp8bq {

// A thread's 8 rows by 8 columns.  BF16 stays packed in half the registers: its magnitudes compare as 16-bit
// integers, two at a time, and a value is unpacked (one shift or mask) where it is divided.
template <typename TIn>
struct Patch;
template <>
struct Patch<float> {
  float v[8][8];
  __device__ __forceinline__ void load(int p, const float* x) { Load8<float>::run(x, v[p]); }
  __device__ __forceinline__ void clear(int p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[p][i] = 0.0f;
  }
  __device__ __forceinline__ void renew() {}
  __device__ __forceinline__ float at(int p, int i) const { return v[p][i]; }
  __device__ __forceinline__ float row_max(int p) const {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __builtin_fmaxf(m, __builtin_fabsf(v[p][i]));
    return m;
  }
  __device__ __forceinline__ void column_max(int c, float& even, float& odd) const {
    even = odd = 0.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      even = __builtin_fmaxf(even, __builtin_fabsf(v[p][2 * c]));
      odd = __builtin_fmaxf(odd, __builtin_fabsf(v[p][2 * c + 1]));
    }
  }
};
template <>
struct Patch<uint16_t> {
  u32x4 w[8];
  __device__ __forceinline__ void load(int p, const uint16_t* x) { w[p] = *reinterpret_cast<const u32x4*>(x); }
  __device__ __forceinline__ void clear(int p) { w[p] = (u32x4){0, 0, 0, 0}; }
  // Between the row and the column layout: the compiler would otherwise keep all 64 unpacked values from the
  // one for the other (170 registers, two waves per SIMD).
  __device__ __forceinline__ void renew() {
#pragma unroll
    for (int p = 0; p < 8; ++p) asm volatile("" : "+v"(w[p]));
  }
  __device__ __forceinline__ float at(int p, int i) const { return i & 1 ? bf16hi(w[p][i >> 1]) : bf16lo(w[p][i >> 1]); }
  __device__ __forceinline__ float row_max(int p) const {
    uint32_t m = w[p][0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 4; ++i) m = pk_umax16(m, w[p][i] & 0x7FFF7FFFu);
    return bf16lo(umax(m & 0xFFFFu, m >> 16));
  }
  __device__ __forceinline__ void column_max(int c, float& even, float& odd) const {
    uint32_t m = w[0][c] & 0x7FFF7FFFu;
#pragma unroll
    for (int p = 1; p < 8; ++p) m = pk_umax16(m, w[p][c] & 0x7FFF7FFFu);
    even = bf16lo(m);
    odd = bf16hi(m);
  }
};

template <typename TIn, int FR, int FC, bool ROWS>
__global__ __launch_bounds__(256) void quant_grouped_kernel(const TIn* __restrict__ x, int64_t T, int64_t ldx,
                                                            const int64_t* __restrict__ offsets, int E,
                                                            uint8_t* __restrict__ q, int64_t ldq,
                                                            float* __restrict__ s, int64_t lds,
                                                            uint8_t* __restrict__ qt, int64_t ldqt,
                                                            float* __restrict__ st, int64_t ldst, int64_t padded) {
  __shared__ float red[16][kRedStride];
  __shared__ __attribute__((aligned(16))) float ssc[kColPos];
  __shared__ __attribute__((aligned(16))) float src[kColPos];
  __shared__ __attribute__((aligned(16))) uint8_t tileT[kQtBytes];
  __shared__ int rows[kMaxExperts + 1];
  __shared__ uint32_t blocks[kMaxExperts + 1];

  const int t = threadIdx.x;
  const int lane = t & 63;
  const int cc = t & 15;
  const int rg = t >> 4;
  const int64_t g = blockIdx.x;  // 128-column group
  const int64_t c0 = g * kQtCols;
  const int64_t col = c0 + 8 * cc;

  if (t < 64) group_table_rows(offsets, E, T, kGroup, 1, rows, blocks, lane);
  __syncthreads();
  const uint32_t cap = (uint32_t)(padded / kGroup);
  const uint32_t nblk = blocks[E] < cap ? blocks[E] : cap;

  for (uint32_t rb = blockIdx.y; rb < nblk; rb += gridDim.y) {
    const int e = group_find(blocks, E, rb, lane);
    const int64_t r0 = rows[e] + (int64_t)(rb - blocks[e]) * kGroup;  // first token of the block
    const int left = (int)(rows[e + 1] - r0);                        // tokens in it (128 if more)

    Patch<TIn> v;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      if (8 * rg + p < left)
        v.load(p, x + (r0 + 8 * rg + p) * ldx + col);
      else
        v.clear(p);
    }

    if constexpr (ROWS) {
      float m[8];
#pragma unroll
      for (int p = 0; p < 8; ++p) m[p] = v.row_max(p);
      const float sc_own = group_scale<FR>(row16_max_scatter<8>(m, cc));
      const float rc_own = 1.0f / sc_own;
      const int own = 8 * rg + (cc >> scatter_shift<8>());
      if ((cc & 1) == 0 && own < left) s[g * lds + r0 + own] = sc_own;
      static_for<8>([&](auto P) {
        constexpr int p = decltype(P)::value;
        const float sc = row16_bcast<(p << scatter_shift<8>())>(sc_own);
        const float rc = row16_bcast<(p << scatter_shift<8>())>(rc_own);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = v.at(p, i);
        if (8 * rg + p < left) store_codes8(q + (r0 + 8 * rg + p) * ldq + col, quant8<FR>(y, sc, rc));
      });
      v.renew();
    }

#pragma unroll
    for (int i = 0; i < 4; ++i)
      v.column_max(i, red[rg][col_pos(8 * cc + 2 * i)], red[rg][col_pos(8 * cc + 2 * i + 1)]);
    __syncthreads();
    if (t < kQtCols) {
      float m = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) m = __builtin_fmaxf(m, red[k][col_pos(t)]);
      const float sc = group_scale<FC>(m);
      ssc[col_pos(t)] = sc;
      src[col_pos(t)] = 1.0f / sc;
      st[rb * ldst + c0 + t] = sc;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = 8 * cc + i;
      const float sc = ssc[col_pos(c)], rc = src[col_pos(c)];
      float y[8];
#pragma unroll
      for (int p = 0; p < 8; ++p) y[p] = blockwise_quotient(v.at(p, i), sc, rc);
      const uint2 w = make_uint2(pack4<FC>(y[0], y[1], y[2], y[3]), pack4<FC>(y[4], y[5], y[6], y[7]));
      *reinterpret_cast<uint2*>(tileT + qt_off(c, rg)) = w;
    }
    __syncthreads();
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
      const int c = (t >> 3) + 32 * pass;
      const int ch = t & 7;
      const uint4 codes = *reinterpret_cast<const uint4*>(tileT + qt_off(c, 2 * ch));
      store_codes16(qt + (c0 + c) * ldqt + (int64_t)rb * kGroup + 16 * ch, codes);
    }
    __syncthreads();  // tileT and red are written again for the next block
  }
}

template <typename TIn, int FR, int FC, bool ROWS>
static hipError_t launch_t(const void* x, int64_t T, int64_t C, int64_t ldx, const int64_t* offsets, int E, uint8_t* q,
                           int64_t ldq, float* s, int64_t lds, uint8_t* qt, int64_t ldqt, float* st_, int64_t ldst,
                           int64_t padded, int cus, hipStream_t st) {
  // about eight workgroups per CU (four resident), at most one per 128x128 tile
  const int64_t ncg = C / kQtCols, nrb = padded / kGroup;
  int64_t gy = (8 * (int64_t)cus + ncg - 1) / ncg;
  gy = gy < nrb ? gy : nrb;
  gy = gy < 65535 ? gy : 65535;
  hipLaunchKernelGGL((quant_grouped_kernel<TIn, FR, FC, ROWS>), dim3((unsigned)ncg, (unsigned)gy), dim3(256), 0, st,
                     (const TIn*)x, T, ldx, offsets, E, q, ldq, s, lds, qt, ldqt, st_, ldst, padded);
  return hipGetLastError();
}

template <typename TIn>
static hipError_t launch_in(const void* x, int64_t T, int64_t C, int64_t ldx, const int64_t* offsets, int E, int fr,
                            uint8_t* q, int64_t ldq, float* s, int64_t lds, int fc, uint8_t* qt, int64_t ldqt,
                            float* st_, int64_t ldst, int64_t padded, int cus, hipStream_t st) {
  if (q == nullptr)
    return fc == kE4M3 ? launch_t<TIn, kE4M3, kE4M3, false>(x, T, C, ldx, offsets, E, q, ldq, s, lds, qt, ldqt, st_,
                                                             ldst, padded, cus, st)
                       : launch_t<TIn, kE4M3, kE5M2, false>(x, T, C, ldx, offsets, E, q, ldq, s, lds, qt, ldqt, st_,
                                                             ldst, padded, cus, st);
  if (fr == kE4M3)
    return fc == kE4M3 ? launch_t<TIn, kE4M3, kE4M3, true>(x, T, C, ldx, offsets, E, q, ldq, s, lds, qt, ldqt, st_,
                                                            ldst, padded, cus, st)
                       : launch_t<TIn, kE4M3, kE5M2, true>(x, T, C, ldx, offsets, E, q, ldq, s, lds, qt, ldqt, st_,
                                                            ldst, padded, cus, st);
  return fc == kE4M3 ? launch_t<TIn, kE5M2, kE4M3, true>(x, T, C, ldx, offsets, E, q, ldq, s, lds, qt, ldqt, st_, ldst,
                                                          padded, cus, st)
                     : launch_t<TIn, kE5M2, kE5M2, true>(x, T, C, ldx, offsets, E, q, ldq, s, lds, qt, ldqt, st_, ldst,
                                                          padded, cus, st);
}

hipError_t launch_quant_grouped(const void* x, int xt, int64_t T, int64_t C, int64_t ldx, const int64_t* offsets,
                                int experts, int fr, uint8_t* q, int64_t ldq, float* s, int64_t lds, int fc,
                                uint8_t* qt, int64_t ldqt, float* st_, int64_t ldst, int64_t padded, int cus,
                                hipStream_t st) {
  return xt == 0 ? launch_in<uint16_t>(x, T, C, ldx, offsets, experts, fr, q, ldq, s, lds, fc, qt, ldqt, st_, ldst,
                                       padded, cus, st)
                 : launch_in<float>(x, T, C, ldx, offsets, experts, fr, q, ldq, s, lds, fc, qt, ldqt, st_, ldst,
                                    padded, cus, st);
}

}  // namespace fp8bq
