// Output of the products whose wave tiles are patches of 32 x 32 (32-row MFMAs): the rows of the B patches, and
// how a tile leaves the registers.
//
// The MFMA's first operand is the B patch, its second the A patch: lane l ends with row l % 32 of the A patch, and its
// accumulators 8 r .. 8 r + 7 (r = 0, 1) are columns 16 r + 8 (l / 32) .. +7 of the B patch, whose rows are
// permuted for that.
#pragma once

#include "device_common.hpp"

namespace fp8bq {

typedef float v16f __attribute__((ext_vector_type(16)));

// B patch: tile row n of MFMA row rho = 8 a + 4 h + b (lane half h, accumulators 4 a + b), so that a half holds
// columns 8 h .. +7 and 16 + 8 h .. +7 of the patch; and the inverse.
__device__ __forceinline__ int row_of_rho(int rho) {
  const int a = rho >> 3, h = (rho >> 2) & 1, b = rho & 3;
  return 16 * (a >> 1) + 8 * h + 4 * (a & 1) + b;
}
__device__ __forceinline__ int rho_of_row(int n) {
  return 8 * (2 * ((n >> 4) & 1) + ((n >> 2) & 1)) + 4 * ((n >> 3) & 1) + (n & 3);
}

// Where a lane's part of the tile lies: its first row m and column n0 (8 (lane / 32) included), the ends of the
// rows and columns that exist, whether the whole tile exists and 16-byte stores are possible everywhere (full), and
// whether rows are aligned for wide stores at all (vec).
struct TileEdge {
  int64_t m, n0, mlim, nlim;
  bool full, vec;
};

// FP32: o points at (m, n0), rows ldo apart.  add: to what lies there.  ADD: the kernel's output is one that is added to
// (the adding has just read its lines, so they are never stored past the caches).
template <bool ADD, int MI, int NI>
__device__ __forceinline__ void store_tile_f32(const v16f (&acc)[MI][NI], float* o, int64_t ldo, const TileEdge& at,
                                               bool add, bool past, int lane) {
  if (at.full) {
    // A lane's four 16-byte chunks of a patch row and the four rows 8 apart of the lanes l ^ 8, l ^ 16, l ^ 24 change
    // places, so that a store instruction writes eight rows of a patch, whole 128-byte lines (us with the chunks
    // where they are and so, added to the output: 8192^3 395 / 347, 16384 x 2048 x 5632 138 / 117).
    o += 16 * (lane >> 4 & 1) + 4 * (lane >> 3 & 1) - (lane & 24) * ldo;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const v16f& v = acc[i][j];
        v4i x[4], w[4];  // chunks 0 and 1 of rows l % 16 and 16 + l % 16; then rows l % 8 + 0, 8, 16, 24
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[4 * r + k]),
                                                            __float_as_uint(v[8 + 4 * r + k]), false, false);
            x[r][k] = (int)p[0];
            x[2 + r][k] = (int)p[1];
          }
        join_halves(x[0], x[1], w[0], w[1]);
        join_halves(x[2], x[3], w[2], w[3]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v4f s = __builtin_bit_cast(v4f, w[q]);
          v4f* o4 = reinterpret_cast<v4f*>(o + (32 * i + 8 * q) * ldo + 32 * j);
          if (add) s = *o4 + s;
          store_line(s, o4, past && !ADD);
        }
      }
  } else {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int64_t c = 32 * j + 16 * (r >> 1) + 4 * (r & 1);
          float* p = o + 32 * i * ldo + c;
          if (at.m + 32 * i >= at.mlim || at.n0 + c >= at.nlim) continue;
          if (at.vec && at.n0 + c + 4 <= at.nlim) {
            v4f w = {acc[i][j][4 * r], acc[i][j][4 * r + 1], acc[i][j][4 * r + 2], acc[i][j][4 * r + 3]};
            if (add) w = *reinterpret_cast<v4f*>(p) + w;
            *reinterpret_cast<v4f*>(p) = w;
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (at.n0 + c + k < at.nlim) p[k] = add ? p[k] + acc[i][j][4 * r + k] : acc[i][j][4 * r + k];
          }
        }
  }
}

// BF16, as above.
template <int MI, int NI>
__device__ __forceinline__ void store_tile_bf16(const v16f (&acc)[MI][NI], uint16_t* o, int64_t ldc, const TileEdge& at,
                                                bool past, int lane) {
  if (at.full) {
    // a lane's two 16-byte chunks of a patch row: lanes l and l + 16 swap one, so that a store instruction
    // writes 64 contiguous bytes of 16 rows (four lanes each) and not 32 of 32 rows
    uint16_t* s0 = o - (lane & 16) * ldc + (lane & 16);
    auto rows = [&](const v16f& v, v4i& x, v4i& y) {  // rows 0 .. 15 and 16 .. 31 of the patch
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const auto p = __builtin_amdgcn_permlane16_swap(pack_bf16x2(v[2 * r], v[2 * r + 1]),
                                                        pack_bf16x2(v[8 + 2 * r], v[9 + 2 * r]), false, false);
        x[r] = (int)p[0];
        y[r] = (int)p[1];
      }
    };
    if constexpr (NI == 2) {
      // two patches side by side: whole 128-byte lines.  Where they go past the caches (stores_past_caches) that is
      // what makes it worth it: us with 64-byte stores, whole lines, and whole lines past the caches
      // 16384 x 11264 x 2048 242 / 238 / 209, 4096 x 2560 x 2048 20.4 / 20.6 / 18.4.
      const int half = (lane >> 3) & 1;
      s0 += 32 * half - 8 * half * ldc;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        v4i x[2], y[2], upper, lower;
#pragma unroll
        for (int j = 0; j < 2; ++j) rows(acc[i][j], x[j], y[j]);
        uint16_t* s = s0 + 32 * i * ldc;
        join_halves(x[0], x[1], upper, lower);
        store_line(upper, reinterpret_cast<v4i*>(s), past);
        store_line(lower, reinterpret_cast<v4i*>(s + 8 * ldc), past);
        join_halves(y[0], y[1], upper, lower);
        store_line(upper, reinterpret_cast<v4i*>(s + 16 * ldc), past);
        store_line(lower, reinterpret_cast<v4i*>(s + 24 * ldc), past);
      }
    } else {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          v4i x, y;
          rows(acc[i][j], x, y);
          uint16_t* s = s0 + 32 * i * ldc + 32 * j;
          *reinterpret_cast<v4i*>(s) = x;
          *reinterpret_cast<v4i*>(s + 16 * ldc) = y;
        }
    }
  } else {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int64_t c = 32 * j + 16 * r;
          uint16_t* p = o + 32 * i * ldc + c;
          if (at.m + 32 * i >= at.mlim || at.n0 + c >= at.nlim) continue;
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = pack_bf16x2(acc[i][j][8 * r + 2 * k], acc[i][j][8 * r + 2 * k + 1]);
          if (at.vec && at.n0 + c + 8 <= at.nlim) {
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (at.n0 + c + k < at.nlim) p[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
          }
        }
  }
}

}  // namespace fp8bq
