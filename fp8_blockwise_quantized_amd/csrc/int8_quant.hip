// Quantizers of the 8-bit linear layer: rows (a scale for each token) and columns, transposed (a scale for each channel
// over all the tokens: the operands of the products that contract over the tokens).  The rule is in int8_common.hpp.
//
// Bound by memory.  Rows: a row's values stay in registers between the maximum and the codes, so x is read once (16384 x
// 2048 BF16 17 us, 5.9 TB/s; 16384 x 11264 102 us, 5.4).  Columns: the maximum of a column needs all rows, so x is
// read twice, by column blocks of 128; the first pass leaves the maxima of each chunk of rows, the second joins them
// (4099 x 5632 BF16 9 + 14 us, of which 11 are the 69 MB at the copy's rate that one read of x and the codes need; the second
// read comes from the caches).
#include "int8_common.hpp"
#include "launch.hpp"

namespace fp8bq {

// Eight elements as loaded.
template <typename TIn>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  u32x4 w;
  __device__ __forceinline__ void load(const uint16_t* p) { w = *reinterpret_cast<const u32x4*>(p); }
  __device__ __forceinline__ void zero() { w = (u32x4){0, 0, 0, 0}; }
  __device__ __forceinline__ uint32_t amax(uint32_t m) const {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) a = pk_umax16(a, w[i] & 0x7FFF7FFFu);
    return umax(m, umax(a & 0xFFFFu, a >> 16) << 16);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16lo(w[i]);
      v[2 * i + 1] = bf16hi(w[i]);
    }
  }
};
template <>
struct Raw8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const f32x4*>(p);
    b = *(reinterpret_cast<const f32x4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = (f32x4){0.0f, 0.0f, 0.0f, 0.0f}; }
  __device__ __forceinline__ uint32_t amax(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = umax(m, umax(abs_bits(a[i]), abs_bits(b[i])));
    return m;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
};

constexpr int kQRowThreads = 256;

// WPR waves share a row; a lane holds CH chunks of eight elements in registers (CH = 0: rows of any length, read twice).
template <typename TIn, int WPR, int CH>
__global__ __launch_bounds__(kQRowThreads) void int8_rows_kernel(const TIn* __restrict__ x, int64_t R, int64_t C,
                                                                 int64_t ldx, uint8_t* __restrict__ q, int64_t ldq,
                                                                 float* __restrict__ s) {
  constexpr int RPB = kQRowThreads / 64 / WPR;  // rows of a workgroup
  __shared__ uint32_t part[kQRowThreads / 64];
  const int t = threadIdx.x, wid = t >> 6;
  const int64_t row = (int64_t)blockIdx.x * RPB + wid / WPR;
  const int lane = t % (64 * WPR);
  const bool live = row < R;
  const TIn* xr = x + row * ldx;
  Raw8<TIn> v[CH > 0 ? CH : 1];
  uint32_t m = 0;
  if (live) {
    if constexpr (CH > 0) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int64_t c = 8 * ((int64_t)i * 64 * WPR + lane);
        if (c < C) v[i].load(xr + c); else v[i].zero();
      }
#pragma unroll
      for (int i = 0; i < CH; ++i) m = v[i].amax(m);
    } else {
      for (int64_t c = 8 * (int64_t)lane; c < C; c += 512 * WPR) {
        v[0].load(xr + c);
        m = v[0].amax(m);
      }
    }
  }
  m = wave_umax(m);
  if constexpr (WPR > 1) {
    if ((t & 63) == 0) part[wid] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WPR; ++i) m = umax(m, part[wid / WPR * WPR + i]);
  }
  if (!live) return;
  const float sc = int8_scale(m), r = 1.0f / sc;
  if (lane == 0) s[row] = sc;
  auto put = [&](const Raw8<TIn>& raw, int64_t c) {
    float f[8];
    raw.get(f);
    store_codes8(q + row * ldq + c, int8_quant8(f, sc, r));
  };
  if constexpr (CH > 0) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int64_t c = 8 * ((int64_t)i * 64 * WPR + lane);
      if (c < C) put(v[i], c);
    }
  } else {
    for (int64_t c = 8 * (int64_t)lane; c < C; c += 512 * WPR) {
      v[0].load(xr + c);
      put(v[0], c);
    }
  }
}

template <typename TIn, int WPR, int CH>
static hipError_t launch_rows(const void* x, int64_t R, int64_t C, int64_t ldx, uint8_t* q, int64_t ldq, float* s,
                              hipStream_t st) {
  constexpr int RPB = kQRowThreads / 64 / WPR;
  constexpr int64_t kMost = (int64_t)1 << 22;  // rows of a launch: its threads stay below 2^32
  for (int64_t r = 0; r < R; r += kMost) {
    const int64_t n = R - r < kMost ? R - r : kMost;
    hipLaunchKernelGGL((int8_rows_kernel<TIn, WPR, CH>), dim3((unsigned)((n + RPB - 1) / RPB)), dim3(kQRowThreads), 0, st,
                       (const TIn*)x + r * ldx, n, C, ldx, q + r * ldq, ldq, s + r);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// A wave holds rows of up to 2048 elements, four waves longer ones (us with one wave and four: 16384 x 512 6.3 / 14, x 2048
// 17 / 19, x 4096 34 / 30, x 11264 162 / 103; 512 x 2048 2.9 / 2.9, x 5632 4.7 / 3.4).
template <typename TIn>
static hipError_t launch_rows_any(const void* x, int64_t R, int64_t C, int64_t ldx, uint8_t* q, int64_t ldq, float* s,
                                  hipStream_t st) {
  if (C <= 4 * 512) return launch_rows<TIn, 1, 4>(x, R, C, ldx, q, ldq, s, st);
  if (C <= 4 * 2048) return launch_rows<TIn, 4, 4>(x, R, C, ldx, q, ldq, s, st);
  if (C <= 12 * 2048) return launch_rows<TIn, 4, 12>(x, R, C, ldx, q, ldq, s, st);
  return launch_rows<TIn, 4, 0>(x, R, C, ldx, q, ldq, s, st);
}

hipError_t launch_int8_rows(const void* x, int xt, int64_t R, int64_t C, int64_t ldx, uint8_t* q, int64_t ldq, float* s,
                            hipStream_t st) {
  return xt == 0 ? launch_rows_any<uint16_t>(x, R, C, ldx, q, ldq, s, st) : launch_rows_any<float>(x, R, C, ldx, q, ldq, s, st);
}

// Columns, first pass: maxima of 128 columns over a chunk of `rows` rows, part[chunk][C].
template <typename TIn>
__global__ __launch_bounds__(256) void int8_colmax_kernel(const TIn* __restrict__ x, int64_t R, int64_t C, int64_t ldx,
                                                          int64_t rows, uint32_t ctiles, uint32_t* __restrict__ part) {
  __shared__ uint32_t red[16][kQtCols + 1];
  const TileRC b = tile_of_block(ctiles);
  const int t = threadIdx.x, cc = t & 15, rr = t >> 4;
  const int64_t c = b.col * kQtCols + 8 * cc;
  const int64_t r0 = b.row * rows, r1 = r0 + rows < R ? r0 + rows : R;
  uint32_t m[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (c < C) {
#pragma unroll 4
    for (int64_t r = r0 + rr; r < r1; r += 16) {
      float v[8];
      Load8<TIn>::run(x + r * ldx + c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = umax(m[i], abs_bits(v[i]));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) red[rr][8 * cc + i] = m[i];
  __syncthreads();
  if (t < kQtCols && b.col * kQtCols + t < C) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = umax(a, red[i][t]);
    part[b.row * C + b.col * kQtCols + t] = a;
  }
}

// Second pass: a tile of 128 rows by 128 columns; codes go through LDS and leave transposed, 16 rows to a store.  A
// thread's values are on their way while the maxima of the chunks are joined.
template <typename TIn>
__global__ __launch_bounds__(256) void int8_cols_kernel(const TIn* __restrict__ x, int64_t R, int64_t C, int64_t ldx,
                                                        uint32_t ctiles, const uint32_t* __restrict__ part, int chunks,
                                                        uint8_t* __restrict__ qt, int64_t ldqt, float* __restrict__ st) {
  __shared__ float scale[kColPos], inverse[kColPos];
  __shared__ uint32_t other[kQtCols];
  __shared__ __attribute__((aligned(16))) uint8_t codes[kQtBytes];
  const TileRC b = tile_of_block(ctiles);
  const int t = threadIdx.x;
  const int64_t c0 = b.col * kQtCols;
  const int64_t r0 = b.row * 128;
  // thread: columns 8 cc .. +7 of rows 8 rr .. +7
  const int cc = t & 15, rr = t >> 4;
  const int64_t c = c0 + 8 * cc;
  Raw8<TIn> raw[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t r = r0 + 8 * rr + k;
    if (r < R && c < C) raw[k].load(x + r * ldx + c); else raw[k].zero();
  }
  {
    const int col = t & (kQtCols - 1), half = t >> 7;  // each half of the threads takes every other chunk
    const int64_t at = c0 + col < C ? c0 + col : C - 1;
    uint32_t a = 0;
#pragma unroll 8
    for (int k = half; k < chunks; k += 2) a = umax(a, part[(int64_t)k * C + at]);
    if (half) other[col] = a;
    __syncthreads();
    if (!half) {
      const float sc = int8_scale(umax(a, other[col]));
      scale[col_pos(col)] = sc;
      inverse[col_pos(col)] = 1.0f / sc;
      if (b.row == 0 && c0 + col < C) st[c0 + col] = sc;
    }
  }
  __syncthreads();
  uint32_t w[8][2];  // [column][half]: codes of eight rows
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float v[4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k) raw[4 * half + k].get(v[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float sc = scale[col_pos(8 * cc + i)], rc = inverse[col_pos(8 * cc + i)];
      w[i][half] = int8_pack4(div_by_scale(v[0][i], sc, rc), div_by_scale(v[1][i], sc, rc), div_by_scale(v[2][i], sc, rc),
                              div_by_scale(v[3][i], sc, rc));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint2*>(codes + qt_off(8 * cc + i, rr)) = make_uint2(w[i][0], w[i][1]);
  __syncthreads();
  // 16 rows a store, eight stores to a column's 128 codes
  const int64_t rpad = (R + 15) / 16 * 16;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int col = 32 * k + (t >> 3), u = t & 7;
    if (c0 + col < C && r0 + 16 * u < rpad)
      store_codes16(qt + (c0 + col) * ldqt + r0 + 16 * u, *reinterpret_cast<const uint4*>(codes + qt_off(col, 2 * u)));
  }
}

int int8_col_chunks(int64_t R, int64_t C) {
  const int64_t tiles = (C + kQtCols - 1) / kQtCols, most = (R + 127) / 128;
  int64_t chunks = (1024 + tiles - 1) / tiles;  // about 1024 workgroups; every tile of the second pass reads all chunks
  chunks = chunks < most ? chunks : most;
  return (int)(chunks < 1 ? 1 : chunks > 32 ? 32 : chunks);
}

template <typename TIn>
static hipError_t launch_cols(const void* x, int64_t R, int64_t C, int64_t ldx, uint8_t* qt, int64_t ldqt, float* st_,
                              uint32_t* part, hipStream_t st) {
  const uint32_t ctiles = (uint32_t)((C + kQtCols - 1) / kQtCols);
  const int chunks = int8_col_chunks(R, C);
  const int64_t rows = (R + chunks - 1) / chunks;
  const TIn* xp = reinterpret_cast<const TIn*>(x);
  hipLaunchKernelGGL(int8_colmax_kernel<TIn>, dim3((unsigned)(ctiles * (uint32_t)chunks)), dim3(256), 0, st, xp, R, C, ldx,
                     rows, ctiles, part);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t blocks = (int64_t)ctiles * ((R + 127) / 128);
  hipLaunchKernelGGL(int8_cols_kernel<TIn>, dim3((unsigned)blocks), dim3(256), 0, st, xp, R, C, ldx, ctiles, part, chunks,
                     qt, ldqt, st_);
  return hipGetLastError();
}

hipError_t launch_int8_cols(const void* x, int xt, int64_t R, int64_t C, int64_t ldx, uint8_t* qt, int64_t ldqt,
                            float* st_, void* ws, hipStream_t st) {
  return xt == 0 ? launch_cols<uint16_t>(x, R, C, ldx, qt, ldqt, st_, (uint32_t*)ws, st)
                 : launch_cols<float>(x, R, C, ldx, qt, ldqt, st_, (uint32_t*)ws, st);
}

}  // namespace fp8bq
