// MXFP4 product for many rows: C[m, n] = sum_k A[m, k] B[n, k], tiles staged in LDS.
//
// Mathematics: the MFMA multiplies the two block scales into each 32-long partial sum itself
// (v_mfma_scale_f32_32x32x64_f8f6f4, two blocks per operand row), so the whole contraction accumulates in one
// set of FP32 registers and nothing is folded afterwards.
//
// Bound at large sizes by the LDS reads that feed the matrix pipes (busy 46% of the cycles at 16384 x 11264 x 2048; four
// instructions of this kind on end reach 7.1 PFLOP/s on the card): LDS has to deliver 1 KB per 32-row patch and
// 64-long step.  A wave tile of 128 x 64 needs 6 patch reads for 8 MFMAs of 32 cycles, three quarters of the LDS
// bandwidth with eight waves.
//
// Layout.  A stage holds 256 values (128 bytes) of the tile's rows of A and B and the two scale words of each
// row, and arrives by direct global->LDS loads into a ring of two stages; a stage's loads go out between the
// last MFMAs of the stage whose slot it takes.  16-byte chunks are XOR-swizzled by row.  The MFMA's first operand
// is the B patch: lane l ends with row l % 32 of the A patch and 16 of the B patch's 32 columns, B patch rows
// being permuted so that those 16 are two runs of eight.
// Measured (us for 16384 x 11264 x 2048 / 2048 x 5632 x 16384 / 8192^3): 196-219 / 99 / 245-252, that is 3.4-3.9 / 3.8 /
// 4.4-4.5 PFLOP/s, by card.
// Alternatives, against 285 / 122 / 284 for this form with other stores on a slower card: loads all issued after the
// barrier 294 / 132 / 287; four stages of 128 values 304 / 128 / 295; 128 x 256 tiles, two workgroups per CU
// 345 / 148 / 344.  Without the loads 8192^3 took 228 us, without loads, barriers and writes 217 (the bare instructions
// would take 155): the matrix pipes with the LDS reads they need are the larger part, at the clock the card's power
// allows them.
//
// A lane's operand is block l / 32 of a 64-long step; it shifts the row's scale word by 8 (l / 32) once per
// 128-long stretch, and the instruction's byte select (0 or 2) picks the step.  The words of a contraction's
// last stretches are masked past the last block (zero bytes, 2^-127 on both sides: the product of whatever codes
// lie there vanishes below FP32's range).
//
// Workgroups are persistent and the ring runs on across tiles, as in the FP8 kernel.
#include "gemm_kernel.hpp"
#include "mx_common.hpp"

namespace fp8bq {

// B patch: tile row n of MFMA row rho = 8 a + 4 h + b (lane half h, accumulators 4 a + b), so that a half holds
// columns 8 h .. +7 and 16 + 8 h .. +7 of the patch; and the inverse.
__device__ __forceinline__ int mx_row_of_rho(int rho) {
  const int a = rho >> 3, h = (rho >> 2) & 1, b = rho & 3;
  return 16 * (a >> 1) + 8 * h + 4 * (a & 1) + b;
}
__device__ __forceinline__ int mx_rho(int n) {
  return 8 * (2 * ((n >> 4) & 1) + ((n >> 2) & 1)) + 4 * ((n >> 3) & 1) + (n & 3);
}

// LDS ring: NST stages of STEPS 64-long steps.
template <int BM, int BN, int NW, int STEPS, int NST>
struct MxTile {
  static constexpr int kRow = 32 * STEPS;  // bytes of a row in a stage
  static constexpr int kB = BM * kRow;
  static constexpr int kSA = (BM + BN) * kRow;  // per 128-long stretch: scale words of A's rows, then of B's
  static constexpr int kStage = kSA + STEPS / 2 * (BM + BN) * 4;
  static constexpr int kLds = NST * kStage + kGroupTableBytes;
  static constexpr int kBlocks = 4 * kLds <= 160 * 1024 ? 4 : 2 * kLds <= 160 * 1024 ? 2 : 1;  // workgroups per CU
  // waves per SIMD that the launch bound keeps registers for
  static constexpr int kMinWaves = kBlocks * NW / 4;
  static_assert(kLds <= 160 * 1024, "LDS ring does not fit");
};
template <int BM, int BN, int WGM, int WGN, int STEPS, int NST, int OUT, bool GROUPED>
__global__ __launch_bounds__(WGM* WGN * 64, (MxTile<BM, BN, WGM * WGN, STEPS, NST>::kMinWaves)) void mx_gemm_kernel(
    MxDesc d, uint32_t tiles_m, uint32_t tiles_n, int nsplit, float* __restrict__ partial, int64_t ldp, int vec,
    GroupArgs<GROUPED ? kGroupRowsMode : kGroupNone> grp) {
  constexpr int NW = WGM * WGN;
  using Tile = MxTile<BM, BN, NW, STEPS, NST>;
  constexpr int WTM = BM / WGM, WTN = BN / WGN;
  constexpr int MI = WTM / 32, NI = WTN / 32;
  constexpr int CH = 2 * STEPS;   // 16-byte chunks of a row
  constexpr int RPL = 64 / CH;    // rows of a 1 KB code load
  constexpr int AL = BM / RPL / NW, BL = BN / RPL / NW;  // code loads per wave and stage
  constexpr int SJ = STEPS / 2 * (BM + BN) / 64;         // scale jobs of 64 words
  constexpr int SL = SJ > NW ? SJ / NW : 1;              // (with fewer jobs than waves some are loaded twice)
  constexpr int LOADS = AL + BL + SL;
  static_assert(CH == 8, "the chunk swizzle is that of 128-byte rows");
  static_assert((SJ % NW == 0 || NW % SJ == 0) && BM / RPL % NW == 0 && BN / RPL % NW == 0, "loads split evenly");
  // (one array: a second __shared__ object makes the compiler wait for every LDS-DMA load in flight before
  // each LDS read)
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NST * Tile::kStage + (GROUPED ? kGroupTableBytes : 0)];
  uint32_t* gunits = reinterpret_cast<uint32_t*>(smem + NST * Tile::kStage);
  int* gstarts = reinterpret_cast<int*>(gunits + kMaxExperts + 1);

  const int t = threadIdx.x;
  const int lane = t & 63;
  const int wid = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wid / WGN, wn = wid % WGN;
  const int nblk = (int)(d.K / kMxBlock);
  const int nwords = (nblk + 3) / 4;
  const int nkb = (nblk + 2 * STEPS - 1) / (2 * STEPS);  // stages of the contraction
  const uint32_t G = gridDim.x;
  using UnitT = std::conditional_t<GROUPED, GroupUnit, Unit>;
  uint32_t U = tiles_m * tiles_n * (uint32_t)nsplit;
  if constexpr (GROUPED) {
    if (wid == 0) group_table_rows(grp.offsets, grp.experts, grp.tokens, BM, tiles_n, gstarts, gunits, lane);
    __syncthreads();
    U = __builtin_amdgcn_readfirstlane(gunits[grp.experts]);
  }
  if (blockIdx.x >= U) return;
  auto unit_at = [&](uint32_t u) {
    if constexpr (GROUPED)
      return group_unit_of<kGroupRowsMode, BM, BN>(u, gunits, gstarts, grp.experts, (int)d.M, (int)d.N, nkb, lane);
    else
      return unit_of<BM, BN>(u, tiles_m, tiles_n, nsplit, nkb);
  };
  auto m_end = [&](const UnitT& u) -> int64_t {
    if constexpr (GROUPED) return u.mend; else return d.M;
  };
  auto n_end = [&](const UnitT& u) -> int64_t {
    if constexpr (GROUPED) return u.nend; else return d.N;
  };

  // load side
  uint32_t lu = blockIdx.x;
  UnitT L = unit_at(lu);
  int lkb = L.kb0;
  bool lmore = true;
  const uint8_t* abase = nullptr;
  const uint8_t* bbase = nullptr;
  uint32_t abytes = 0, bbytes = 0;
  uint32_t aoff[AL], boff[BL], soff[SL];
  const uint32_t* sbase[SL];
  uint32_t sbytes[SL];
  // scale job j: stretch j / JS of the stage, the words of 64 rows, A's rows first
  constexpr int JS = (BM + BN) / 64;
  int64_t sld[SL];  // words between a job's stretches
  int sword[SL];
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    const int j = (wid + NW * i) % SJ;
    sld[i] = j % JS < BM / 64 ? d.ldsa : d.ldsb;
    sword[i] = j / JS;
  }
  auto set_sources = [&](const UnitT& u) {
    abase = (const uint8_t*)d.a + (int64_t)u.m0 * d.lda;
    bbase = d.b + (int64_t)u.n0 * d.ldb;
    const int64_t mleft = m_end(u) - 1 - u.m0, nleft = n_end(u) - 1 - u.n0;
    abytes = sat32((mleft < BM - 1 ? mleft : BM - 1) * d.lda + d.K / 2);
    bbytes = sat32((nleft < BN - 1 ? nleft : BN - 1) * d.ldb + d.K / 2);
#pragma unroll
    for (int i = 0; i < AL; ++i) {
      const int row = RPL * (wid + NW * i) + lane / CH;
      const int64_t r = row < mleft ? row : mleft;
      aoff[i] = (uint32_t)(r * d.lda) + (uint32_t)(((lane % CH) ^ swz(row)) * 16);
    }
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const int row = RPL * (wid + NW * i) + lane / CH;
      const int64_t r = row < nleft ? row : nleft;
      boff[i] = (uint32_t)(r * d.ldb) + (uint32_t)(((lane % CH) ^ swz(mx_rho(row))) * 16);
    }
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      const int j = (wid + NW * i) % SJ % JS;
      const bool a = j < BM / 64;
      const int64_t r = 64 * (a ? j : j - BM / 64) + lane, left = a ? mleft : nleft, most = (a ? BM : BN) - 1;
      soff[i] = (uint32_t)((r < left ? r : left) * 4);
      sbase[i] = a ? d.sa + u.m0 : d.sb + u.n0;
      sbytes[i] = (uint32_t)((left < most ? left : most) * 4 + 4);
    }
  };
  auto issue_load = [&](int i, uint8_t* stg) {
    if (i < AL) {
      dma16(rsrc_of(abase + (int64_t)lkb * Tile::kRow, abytes - (uint32_t)(lkb * Tile::kRow)), aoff[i], stg + (wid + NW * i) * 1024);
    } else if (i < AL + BL) {
      dma16(rsrc_of(bbase + (int64_t)lkb * Tile::kRow, bbytes - (uint32_t)(lkb * Tile::kRow)), boff[i - AL],
            stg + Tile::kB + (wid + NW * (i - AL)) * 1024);
    } else {
      const int q = i - AL - BL;
      const int word = STEPS / 2 * lkb + sword[q];
      const bool in = word < nwords;  // (past the last word: zeros)
      dma4(rsrc_of(sbase[q] + (in ? word : 0) * sld[q], in ? sbytes[q] : 0u), soff[q],
           stg + Tile::kSA + 256 * ((wid + NW * q) % SJ));
    }
  };
  auto advance = [&]() {
    if (lmore && ++lkb == L.kb1) {
      if (lu + G < U) {
        lu += G;
        L = unit_at(lu);
        lkb = L.kb0;
        set_sources(L);
      } else {
        lkb = L.kb1 - 1;
        lmore = false;
      }
    }
  };
  auto load_stage = [&](uint8_t* stg) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) issue_load(i, stg);
    advance();
  };

  // compute side
  uint32_t cu = lu;
  UnitT C = L;
  int ckb = C.kb0;
  const int r32 = lane & 31, h = lane >> 5;
  const int arow = wm * WTM + r32, brow = wn * WTN + mx_row_of_rho(r32);
  const int sw = swz(r32);  // (patches start at multiples of 32 rows)
  auto aread = [&](const uint8_t* stg, int i, int step) {
    return *reinterpret_cast<const v4i*>(stg + (arow + 32 * i) * Tile::kRow + (((2 * step + h) ^ sw) << 4));
  };
  auto bread = [&](const uint8_t* stg, int j, int step) {
    return *reinterpret_cast<const v4i*>(stg + Tile::kB + (brow + 32 * j) * Tile::kRow + (((2 * step + h) ^ sw) << 4));
  };
  v4i fa[2][MI], fb[2][NI];  // operands of the current and the next step
  uint32_t sa[MI], sb[NI];   // scale words as read, and with the lane's bytes in place
  uint32_t ua[MI], ub[NI];
  auto read_step = [&](const uint8_t* stg, int step, int to) {
#pragma unroll
    for (int i = 0; i < MI; ++i) fa[to][i] = aread(stg, i, step);
#pragma unroll
    for (int j = 0; j < NI; ++j) fb[to][j] = bread(stg, j, step);
  };
  auto read_scales = [&](const uint8_t* stg, int p) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(stg + Tile::kSA) + p * (BM + BN);
#pragma unroll
    for (int i = 0; i < MI; ++i) sa[i] = w[arow + 32 * i];
#pragma unroll
    for (int j = 0; j < NI; ++j) sb[j] = w[BM + brow + 32 * j];
  };
  // keep the bytes of existing blocks and bring the lane's two to bytes 0 and 2
  auto place_scales = [&](int kb, int p) {
    const int left = nblk - 2 * STEPS * kb - 4 * p;
    const uint32_t mask = left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
#pragma unroll
    for (int i = 0; i < MI; ++i) ua[i] = (sa[i] & mask) >> (8 * h);
#pragma unroll
    for (int j = 0; j < NI; ++j) ub[j] = (sb[j] & mask) >> (8 * h);
  };

  v16f acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  set_sources(L);
#pragma unroll
  for (int s = 0; s < NST; ++s) load_stage(smem + s * Tile::kStage);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((NST - 1) * LOADS) : "memory");
  read_step(smem, 0, 0);
  read_scales(smem, 0);

  int rd = 0;
  while (true) {
    uint8_t* stage = smem + rd * Tile::kStage;
    const int nx = rd + 1 == NST ? 0 : rd + 1;
    const uint8_t* nstage = smem + nx * Tile::kStage;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if (s % 2 == 0) place_scales(ckb, s / 2);
      if (s < STEPS - 1) {
        read_step(stage, s + 1, (s + 1) & 1);
        if (s % 2 == 1) read_scales(stage, (s + 1) / 2);
      } else {
        // everything this wave needs of the stage is in registers and the next stage has landed; after the
        // barrier that holds for all waves, and the slot takes the stage NST ahead
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NST - 2) * LOADS) : "memory");
        read_step(nstage, 0, 0);
        read_scales(nstage, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < MI * NI; ++u) {
        const int i = u / NI, j = u % NI;
        if (s % 2)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(fb[1][j]), mx_operand(fa[1][i]),
                                                                      acc[i][j], 4, 4, 2, (int)ub[j], 2, (int)ua[i]);
        else
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(fb[0][j]), mx_operand(fa[0][i]),
                                                                      acc[i][j], 4, 4, 0, (int)ub[j], 0, (int)ua[i]);
        if (s == STEPS - 1) {
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

    // unit finished: write the tile or its partial sum.  Lane l: row l % 32 of each A patch; accumulators
    // 8 r .. 8 r + 7 (r = 0, 1) are columns 16 r + 8 (l / 32) .. +7 of each B patch.
    {
      const int64_t mlim = m_end(C), nlim = n_end(C);
      const int64_t m = (int64_t)C.m0 + arow, n0 = (int64_t)C.n0 + wn * WTN + 8 * h;
      int64_t ccol = 0;
      if constexpr (GROUPED) ccol = C.ccol;
      const bool past = d.past && nsplit == 1;  // (partial sums are read again at once)
      const bool full = vec && (int64_t)C.m0 + BM <= mlim && (int64_t)C.n0 + BN <= nlim;
      if (nsplit > 1 || OUT != 0) {
        const int64_t ldo = nsplit > 1 ? ldp : d.ldc;
        float* o = (nsplit > 1 ? partial + (int64_t)C.split * d.M * ldp : reinterpret_cast<float*>(d.c)) + m * ldo + n0 + ccol;
        const bool add = OUT == 2 && nsplit == 1;
        if (full) {
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
                store_line(s, o4, past && OUT != 2);
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
                if (m + 32 * i >= mlim || n0 + c >= nlim) continue;
                if (vec && n0 + c + 4 <= nlim) {
                  v4f w = {acc[i][j][4 * r], acc[i][j][4 * r + 1], acc[i][j][4 * r + 2], acc[i][j][4 * r + 3]};
                  if (add) w = *reinterpret_cast<v4f*>(p) + w;
                  *reinterpret_cast<v4f*>(p) = w;
                } else {
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    if (n0 + c + k < nlim) p[k] = add ? p[k] + acc[i][j][4 * r + k] : acc[i][j][4 * r + k];
                }
              }
        }
      } else {
        uint16_t* o = reinterpret_cast<uint16_t*>(d.c) + m * d.ldc + n0 + ccol;
        if (full) {
          // a lane's two 16-byte chunks of a patch row: lanes l and l + 16 swap one, so that a store instruction
          // writes 64 contiguous bytes of 16 rows (four lanes each) and not 32 of 32 rows
          uint16_t* s0 = reinterpret_cast<uint16_t*>(d.c) +
                         ((int64_t)C.m0 + wm * WTM + (lane & 15)) * d.ldc + n0 + ccol + (lane & 16);
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
            s0 += 32 * half - 8 * half * d.ldc;
#pragma unroll
            for (int i = 0; i < MI; ++i) {
              v4i x[2], y[2], upper, lower;
#pragma unroll
              for (int j = 0; j < 2; ++j) rows(acc[i][j], x[j], y[j]);
              uint16_t* s = s0 + 32 * i * d.ldc;
              join_halves(x[0], x[1], upper, lower);
              store_line(upper, reinterpret_cast<v4i*>(s), past);
              store_line(lower, reinterpret_cast<v4i*>(s + 8 * d.ldc), past);
              join_halves(y[0], y[1], upper, lower);
              store_line(upper, reinterpret_cast<v4i*>(s + 16 * d.ldc), past);
              store_line(lower, reinterpret_cast<v4i*>(s + 24 * d.ldc), past);
            }
          } else {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
              for (int j = 0; j < NI; ++j) {
                v4i x, y;
                rows(acc[i][j], x, y);
                uint16_t* s = s0 + 32 * i * d.ldc + 32 * j;
                *reinterpret_cast<v4i*>(s) = x;
                *reinterpret_cast<v4i*>(s + 16 * d.ldc) = y;
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
                uint16_t* p = o + 32 * i * d.ldc + c;
                if (m + 32 * i >= mlim || n0 + c >= nlim) continue;
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = pack_bf16x2(acc[i][j][8 * r + 2 * k], acc[i][j][8 * r + 2 * k + 1]);
                if (vec && n0 + c + 8 <= nlim) {
                  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
#pragma unroll
                  for (int k = 0; k < 8; ++k)
                    if (n0 + c + k < nlim) p[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
                }
              }
        }
      }
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    }
    cu += G;
    if (cu >= U) break;
    C = unit_at(cu);
    ckb = C.kb0;
  }
  // no direct-to-LDS load may still be writing when the workgroup's LDS is handed on
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Sum of the split partial sums [nsplit][M][ldp] in split order, converted to the output type (or added to
// it); four columns a thread, the partials' rows being padded to a multiple of four.
template <int OUT>
__global__ __launch_bounds__(256) void mx_reduce_kernel(const float* __restrict__ partial, int nsplit, int64_t M,
                                                        int64_t N, int64_t ldp, void* __restrict__ c, int64_t ldc) {
  const int64_t quads = ldp / 4, total = M * quads;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t m = i / quads, n = 4 * (i - m * quads);
    v4f s = *reinterpret_cast<const v4f*>(partial + m * ldp + n);
    for (int k = 1; k < nsplit; ++k) s += *reinterpret_cast<const v4f*>(partial + ((int64_t)k * M + m) * ldp + n);
    if constexpr (OUT == 0) {
      uint16_t* o = reinterpret_cast<uint16_t*>(c) + m * ldc + n;
      const uint32_t lo = pack_bf16x2(s[0], s[1]), hi = pack_bf16x2(s[2], s[3]);
      if (n + 4 <= N && ((uintptr_t)o & 7) == 0) {
        *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
      } else {
        const uint16_t e[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n + r < N) o[r] = e[r];
      }
    } else {
      float* o = reinterpret_cast<float*>(c) + m * ldc + n;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < N) o[r] = OUT == 2 ? o[r] + s[r] : s[r];
    }
  }
}

template <int BM, int BN, int WGM, int WGN, int STEPS, int NST, int OUT>
static hipError_t launch_tile(const MxDesc& d, const MxGroups& grp, const MxPlan& p, void* ws, int vec,
                              hipStream_t st) {
  const int64_t ldp = (d.N + 3) / 4 * 4;
  const dim3 grid((unsigned)p.grid), block(WGM * WGN * 64);
  if constexpr (OUT != 2) {  // (a grouped product is not added to the output)
    if (grp.offsets) {
      hipLaunchKernelGGL((mx_gemm_kernel<BM, BN, WGM, WGN, STEPS, NST, OUT, true>), grid, block, 0, st, d,
                         (uint32_t)p.tiles_m, (uint32_t)p.tiles_n, 1, (float*)nullptr, ldp, vec,
                         GroupArgs<kGroupRowsMode>{grp.offsets, grp.experts, d.M});
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((mx_gemm_kernel<BM, BN, WGM, WGN, STEPS, NST, OUT, false>), grid, block, 0, st, d,
                     (uint32_t)p.tiles_m, (uint32_t)p.tiles_n, p.split_k, (float*)ws, ldp, vec, GroupArgs<kGroupNone>{});
  return hipGetLastError();
}

template <int OUT>
static hipError_t launch_out(const MxDesc& d, const MxGroups& grp, const MxPlan& p, void* ws, hipStream_t st) {
  const int vec = p.split_k > 1 || (d.ldc * (OUT == 0 ? 2 : 4)) % 16 == 0;
  hipError_t e;
  switch (p.shape) {
    case k256x256: e = launch_tile<256, 256, 2, 4, 4, 2, OUT>(d, grp, p, ws, vec, st); break;
    case k64x64: e = launch_tile<64, 64, 2, 2, 4, 2, OUT>(d, grp, p, ws, vec, st); break;
    default: e = launch_tile<128, 128, 2, 2, 4, 2, OUT>(d, grp, p, ws, vec, st); break;
  }
  if (e != hipSuccess || p.split_k <= 1) return e;
  const int64_t ldp = (d.N + 3) / 4 * 4;
  int64_t blocks = (d.M * (ldp / 4) + 255) / 256;
  blocks = blocks < 8192 ? blocks : 8192;
  hipLaunchKernelGGL((mx_reduce_kernel<OUT>), dim3((unsigned)blocks), dim3(256), 0, st, (const float*)ws, p.split_k,
                     d.M, d.N, ldp, d.c, d.ldc);
  return hipGetLastError();
}

hipError_t launch_mx_gemm(const MxDesc& d, const MxGroups& grp, const MxPlan& p, void* ws, hipStream_t st) {
  if (d.out_t == 0) return launch_out<0>(d, grp, p, ws, st);
  return d.out_t == 1 ? launch_out<1>(d, grp, p, ws, st) : launch_out<2>(d, grp, p, ws, st);
}

}  // namespace fp8bq
