// Products of rows, C[m, n] = sum_k A[m, k] B[n, k], for operands whose 16 contraction bytes a lane feeds to one MFMA:
// 8-bit integers (v_mfma_i32_32x32x32_i8) and halves (v_mfma_f32_32x32x16_f16).  Both read their operands alike, so
// the 8-bit linear layer and the orthogonalized update share this tile loop and differ in what they do with a tile.
//
// Layout.  As the MXFP4 product: a stage holds 128 contraction bytes of the tile's rows of A and B and arrives by
// direct global->LDS loads into a ring of two stages (three in 64 x 64 tiles that are all on the card at once, where a
// stage is shorter than memory's answer takes: 64 x 2048 x 2048 in 8 bits 9.8 -> 7.9 us, 512 x 2048 x 2048 10.2 -> 8.3),
// whose loads go out between the last MFMAs of the stage that held the slot; 16-byte chunks are XOR-swizzled by row (no
// bank conflicts); workgroups are persistent and the ring runs on across tiles.
// Tried on the 256 x 256 tile and not better: four waves of 128 x 128 with their sums in accumulation registers, rings of
// four and eight shorter stages, LDS reads spread between the MFMAs, staggered workgroups, not waiting for a tile's stores;
// touching the lines of a stage ahead of its loads cost 10%.
// A contraction that ends inside a stage: chunks past its end get an offset past the buffer's end, which reads zeros.
#pragma once

#include "gemm_kernel.hpp"
#include "tile_store.hpp"

namespace fp8bq {

typedef int v16i __attribute__((ext_vector_type(16)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

// What the tile loop needs to know of a product; sizes in bytes along the contraction.
struct RowDesc {
  const uint8_t* a;
  int64_t lda;
  const uint8_t* b;
  int64_t ldb;
  int64_t M, N;
  int64_t K;          // contraction bytes, a multiple of 16
  int64_t abatch, bbatch;  // bytes between the matrices of a batch
  // Halves: an operand of 22 bits is a sum of two matrices, low bytes apart.  Of (a + al)(b + bl) the first `terms` of
  // a b, a bl and al b are taken, one stage after the other (al bl is 2^-22 of the whole).
  int64_t alow, blow;
  int terms;
};

enum RowKind : int { kRowsI8 = 0, kRowsF16 = 1 };
template <int KIND>
struct RowAcc;
template <>
struct RowAcc<kRowsI8> {
  typedef v16i type;
  static __device__ __forceinline__ v16i mfma(v4i b, v4i a, v16i c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(b, a, c, 0, 0, 0);
  }
};
template <>
struct RowAcc<kRowsF16> {
  typedef v16f type;
  static __device__ __forceinline__ v16f mfma(v4i b, v4i a, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, b), __builtin_bit_cast(v8h, a), c, 0, 0, 0);
  }
};

// Work units of a batch of products.  TRIANGLE: of a square symmetric result the tiles on and above the diagonal.
enum RowUnits : int { kUnitsFull = 0, kUnitsTriangle = 1, kUnitsGrouped = 2 };

struct RowUnit : GroupUnit {
  int batch;
  uint32_t tile;  // number of the tile among its matrix's
};

// Tile (i, j), i <= j, number w of the upper triangle of t x t tiles, columns of tiles one after the other:
// w = j (j + 1) / 2 + i.
__device__ __forceinline__ void triangle_tile(uint32_t w, uint32_t& i, uint32_t& j) {
  j = (uint32_t)((__builtin_sqrtf(8.0f * (float)w + 1.0f) - 1.0f) * 0.5f);
  while (j * (j + 1) / 2 > w) --j;  // (the root of a rounded number may be one off)
  while ((j + 1) * (j + 2) / 2 <= w) ++j;
  i = w - j * (j + 1) / 2;
}

// The XCD-contiguous position of workgroup number u of U.
__device__ __forceinline__ uint32_t xcd_contiguous(uint32_t u, uint32_t U) {
  const uint32_t q8 = U / kXcds, r8 = U % kXcds, x = u % kXcds;
  return x * q8 + (x < r8 ? x : r8) + u / kXcds;
}

template <int BM, int BN, int NW, int NST>
struct RowTile {
  static constexpr int kB = BM * 128;
  static constexpr int kStage = (BM + BN) * 128;
  static constexpr int kRing = NST * kStage;
  static constexpr int kLds = kRing + kGroupTableBytes;
  static constexpr int kBlocks = 160 * 1024 / kLds < 4 ? 160 * 1024 / kLds : 4;  // workgroups per CU
  static constexpr int kMinWaves = kBlocks * NW / 4;  // waves per SIMD that the launch bound keeps registers for
  static_assert(kLds <= 160 * 1024, "LDS ring does not fit");
};

// What a tile's end needs: the unit, and the wave's and lane's place in it.
struct RowPlace {
  int64_t m0, n0;        // the tile's first row and column
  int64_t mlim, nlim;    // ends of the rows and columns that exist
  int64_t m, n;          // the lane's first row and column
  int64_t ccol;          // output column = column + ccol
  int split, batch, lane;
  uint32_t tile;
  int wave;
  bool whole;            // the whole tile exists
  bool mirror;           // (triangle) the tile's transpose is another tile of the result
};

// Tile number w of a matrix: its row and column of tiles.
template <int UNITS>
__device__ __forceinline__ void row_tile(uint32_t w, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn) {
  if constexpr (UNITS == kUnitsTriangle) {
    triangle_tile(w, tm, tn);
  } else {
    const uint32_t group = (uint32_t)kGroupRows * tiles_n;
    const uint32_t gid = w / group, first = gid * kGroupRows;
    const uint32_t gsz = (tiles_m - first) < (uint32_t)kGroupRows ? (tiles_m - first) : (uint32_t)kGroupRows;
    const uint32_t rem = w - gid * group;
    tm = first + rem % gsz;
    tn = rem / gsz;
  }
}

// smem: ring (and group table).  END: end(acc, place) takes a finished tile.
template <int KIND, int BM, int BN, int WGM, int WGN, int NST, int UNITS, typename END>
__device__ __forceinline__ void row_gemm_units(const RowDesc& d, uint32_t tiles_m, uint32_t tiles_n, int nsplit,
                                               int batches, const GroupArgs<kGroupRowsMode>* grp, uint8_t* smem,
                                               const END& end) {
  constexpr int NW = WGM * WGN;
  using Tile = RowTile<BM, BN, NW, NST>;
  using Acc = RowAcc<KIND>;
  constexpr int WTM = BM / WGM, WTN = BN / WGN;
  constexpr int MI = WTM / 32, NI = WTN / 32;
  constexpr int AL = BM / 8 / NW, BL = BN / 8 / NW;  // 1 KB loads per wave and stage (8 rows each)
  constexpr int LOADS = AL + BL;
  static_assert(BM / 8 % NW == 0 && BN / 8 % NW == 0, "loads split evenly");
  uint32_t* gunits = reinterpret_cast<uint32_t*>(smem + Tile::kRing);
  int* gstarts = reinterpret_cast<int*>(gunits + kMaxExperts + 1);

  const int t = threadIdx.x;
  const int lane = t & 63;
  const int wid = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wid / WGN, wn = wid % WGN;
  const int terms = KIND == kRowsF16 ? d.terms : 1;
  const int nkb = (int)((d.K + 127) / 128) * terms;  // stages of the contraction
  const int tail = (int)(d.K % 128);         // bytes of a last stage that is not whole
  const uint32_t G = gridDim.x;
  const uint32_t T = UNITS == kUnitsTriangle ? tiles_m * (tiles_m + 1) / 2 : tiles_m * tiles_n;
  uint32_t U = T * (uint32_t)nsplit * (uint32_t)batches;
  if constexpr (UNITS == kUnitsGrouped) {
    if (wid == 0) group_table_rows(grp->offsets, grp->experts, grp->tokens, BM, tiles_n, gstarts, gunits, lane);
    __syncthreads();
    U = __builtin_amdgcn_readfirstlane(gunits[grp->experts]);
  }
  if (blockIdx.x >= U) return;
  auto unit_at = [&](uint32_t u) {
    RowUnit r;
    if constexpr (UNITS == kUnitsGrouped) {
      static_cast<GroupUnit&>(r) =
          group_unit_of<kGroupRowsMode, BM, BN>(u, gunits, gstarts, grp->experts, (int)d.M, (int)d.N, nkb, lane);
      r.batch = 0;
      r.split = 0;
      r.tile = 0;
    } else {
      // (opaque here, so that what the divisions by them need is not worked out once and held over the loop)
      uint32_t tiles = T, cols = tiles_n, parts = (uint32_t)nsplit;
      asm volatile("" : "+s"(tiles), "+s"(cols), "+s"(parts));
      const uint32_t L = xcd_contiguous(u, U);
      const uint32_t z = L / tiles, w = L - z * tiles;
      uint32_t tm, tn;
      row_tile<UNITS>(w, tiles_m, cols, tm, tn);
      r.tile = (uint32_t)__builtin_amdgcn_readfirstlane((int)w);
      const int ns = (int)parts;
      r.batch = __builtin_amdgcn_readfirstlane((int)(z / parts));
      r.split = (int)z - r.batch * ns;
      r.m0 = __builtin_amdgcn_readfirstlane((int)tm) * BM;
      r.n0 = __builtin_amdgcn_readfirstlane((int)tn) * BN;
      r.kb0 = __builtin_amdgcn_readfirstlane(r.split * nkb / ns);
      r.kb1 = __builtin_amdgcn_readfirstlane((r.split + 1) * nkb / ns);
      r.mend = (int)d.M;
      r.nend = (int)d.N;
      r.ccol = 0;
    }
    return r;
  };

  // load side
  uint32_t lu = blockIdx.x;
  RowUnit L = unit_at(lu);
  int lkb = L.kb0;
  int lk = 0, lt = 0;  // halves: the stage's place along the rows, and its term
  bool lmore = true;
  const uint8_t* abase = nullptr;
  const uint8_t* bbase = nullptr;
  uint32_t abytes = 0, bbytes = 0;
  uint32_t aoff[AL], boff[BL];
  auto set_sources = [&](const RowUnit& u) {
    if constexpr (KIND == kRowsF16) {
      lk = lkb / terms;
      lt = lkb - lk * terms;
    }
    abase = d.a + (int64_t)u.batch * d.abatch + (int64_t)u.m0 * d.lda;
    bbase = d.b + (int64_t)u.batch * d.bbatch + (int64_t)u.n0 * d.ldb;
    // (32-bit throughout: a tile's rows lie within 2^31 bytes)
    const int mleft = u.mend - 1 - u.m0, nleft = u.nend - 1 - u.n0;
    const uint32_t lda = (uint32_t)d.lda, ldb = (uint32_t)d.ldb;
    abytes = (uint32_t)(mleft < BM - 1 ? mleft : BM - 1) * lda + (uint32_t)d.K;
    bbytes = (uint32_t)(nleft < BN - 1 ? nleft : BN - 1) * ldb + (uint32_t)d.K;
    int el = lane;  // (worked out anew for each unit, as the place in the output)
    asm volatile("" : "+v"(el));
#pragma unroll
    for (int i = 0; i < AL; ++i) {
      const int row = 8 * (wid + NW * i) + el / 8;
      aoff[i] = (uint32_t)(row < mleft ? row : mleft) * lda + (uint32_t)(((el % 8) ^ swz(row)) * 16);
    }
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const int row = 8 * (wid + NW * i) + el / 8;
      boff[i] = (uint32_t)(row < nleft ? row : nleft) * ldb + (uint32_t)(((el % 8) ^ swz(rho_of_row(row))) * 16);
    }
  };
  // the last stage of a contraction that ends inside it: chunks past the end are sent past the buffers' ends (which
  // are below 2^31)
  auto cut_sources = [&]() {
    if (tail == 0 || lkb != nkb - 1) return;
    int el = lane;
    asm volatile("" : "+v"(el));
#pragma unroll
    for (int i = 0; i < AL; ++i) {
      const int row = 8 * (wid + NW * i) + el / 8;
      if (((el % 8) ^ swz(row)) * 16 >= tail) aoff[i] = 0x80000000u;
    }
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const int row = 8 * (wid + NW * i) + el / 8;
      if (((el % 8) ^ swz(rho_of_row(row))) * 16 >= tail) boff[i] = 0x80000000u;
    }
  };
  auto issue_load = [&](int i, uint8_t* stg) {
    const int at = (KIND == kRowsF16 ? lk : lkb) * 128;
    if (i < AL) {
      const int64_t low = KIND == kRowsF16 && lt == 2 ? d.alow : 0;
      dma16(rsrc_of(abase + low + at, abytes - (uint32_t)at), aoff[i], stg + (wid + NW * i) * 1024);
    } else {
      const int64_t low = KIND == kRowsF16 && lt == 1 ? d.blow : 0;
      dma16(rsrc_of(bbase + low + at, bbytes - (uint32_t)at), boff[i - AL], stg + Tile::kB + (wid + NW * (i - AL)) * 1024);
    }
  };
  auto advance = [&]() {
    if (!lmore) return;
    if (++lkb == L.kb1) {
      if (lu + G < U) {
        lu += G;
        L = unit_at(lu);
        lkb = L.kb0;
        set_sources(L);
      } else {
        lkb = L.kb1 - 1;  // (loaded again into a slot that is never read)
        lmore = false;
        return;
      }
    } else if constexpr (KIND == kRowsF16) {
      if (++lt == terms) {
        lt = 0;
        ++lk;
      }
    }
    cut_sources();
  };

  // compute side
  uint32_t cu = lu;
  RowUnit C = L;
  int ckb = C.kb0;
  const int r32 = lane & 31, h = lane >> 5;
  const int arow = wm * WTM + r32, brow = wn * WTN + row_of_rho(r32);
  const int sw = swz(r32);  // (patches start at multiples of 32 rows)
  auto aread = [&](const uint8_t* stg, int i, int step) {
    return *reinterpret_cast<const v4i*>(stg + (arow + 32 * i) * 128 + (((2 * step + h) ^ sw) << 4));
  };
  auto bread = [&](const uint8_t* stg, int j, int step) {
    return *reinterpret_cast<const v4i*>(stg + Tile::kB + (brow + 32 * j) * 128 + (((2 * step + h) ^ sw) << 4));
  };
  v4i fa[2][MI], fb[2][NI];  // operands of the current and the next step
  auto read_step = [&](const uint8_t* stg, int step, int to) {
#pragma unroll
    for (int i = 0; i < MI; ++i) fa[to][i] = aread(stg, i, step);
#pragma unroll
    for (int j = 0; j < NI; ++j) fb[to][j] = bread(stg, j, step);
  };
  typename Acc::type acc[MI][NI];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  };
  clear();

  set_sources(L);
  cut_sources();
#pragma unroll
  for (int s = 0; s < NST; ++s) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) issue_load(i, smem + s * Tile::kStage);
    advance();
  }
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((NST - 1) * LOADS) : "memory");
  read_step(smem, 0, 0);

  int rd = 0;
  while (true) {
    uint8_t* stage = smem + rd * Tile::kStage;
    const int nx = rd + 1 == NST ? 0 : rd + 1;
    const uint8_t* nstage = smem + nx * Tile::kStage;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s < 3) {
        read_step(stage, s + 1, (s + 1) & 1);
      } else {
        // everything this wave needs of the stage is in registers and the next stage has landed; after the
        // barrier that holds for all waves, and the slot takes the stage NST ahead
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NST - 2) * LOADS) : "memory");
        read_step(nstage, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < MI * NI; ++u) {
        const int i = u / NI, j = u % NI;
        acc[i][j] = Acc::mfma(fb[s & 1][j], fa[s & 1][i], acc[i][j]);
        if (s == 3) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int l = u * LOADS / (MI * NI); l < (u + 1) * LOADS / (MI * NI); ++l) issue_load(l, stage);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // keep the MFMAs in the step sequence (not sunk past the cursor update's branches)
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) asm volatile("" : "+v"(acc[i][j]));
    advance();
    rd = nx;
    if (++ckb < C.kb1) continue;

    RowPlace p;
    int el = lane;  // (the lane's place is worked out here: held over the loop it costs registers)
    asm volatile("" : "+v"(el));
    p.m0 = C.m0;
    p.n0 = C.n0;
    p.mlim = C.mend;
    p.nlim = C.nend;
    p.m = (int64_t)C.m0 + wm * WTM + (el & 31);
    p.n = (int64_t)C.n0 + wn * WTN + 8 * (el >> 5);
    p.ccol = C.ccol;
    p.split = C.split;
    p.batch = C.batch;
    p.lane = el;
    p.tile = C.tile;
    p.wave = wid;
    p.whole = (int64_t)C.m0 + BM <= p.mlim && (int64_t)C.n0 + BN <= p.nlim;
    p.mirror = UNITS == kUnitsTriangle && C.m0 != C.n0;
    end(acc, p);
    clear();
    cu += G;
    if (cu >= U) break;
    C = unit_at(cu);
    ckb = C.kb0;
  }
  // no direct-to-LDS load may still be writing when the workgroup's LDS is handed on
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

}  // namespace fp8bq
