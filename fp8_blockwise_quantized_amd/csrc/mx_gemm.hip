// MXFP4 product for many rows: C[m, n] = sum_k A[m, k] B[n, k], tiles staged in LDS.
//
// Mathematics: the MFMA multiplies the two block scales into each 32-long partial sum itself
// (v_mfma_scale_f32_32x32x64_f8f6f4, two blocks per operand row), so the whole contraction accumulates in one
// set of FP32 registers and nothing is folded afterwards.
//
// Bound by the matrix pipes at large sizes (a lane of four instructions of this kind reaches 7.1 PFLOP/s on
// the card): LDS then has to deliver 1 KB per 32-row patch and 64-long step.  A wave tile of 128 x 64 needs 6
// patch reads for 8 MFMAs of 32 cycles, three quarters of the LDS bandwidth with eight waves.
//
// Layout.  A stage holds 256 values (128 bytes) of the tile's rows of A and B and the two scale words of each
// row.  Tiles arrive by direct global->LDS loads into a ring of two stages; 16-byte chunks are XOR-swizzled by
// row as in the FP8 kernel.  The MFMA's first operand is the B patch: lane l ends with row l % 32 of the A
// patch and 16 of the B patch's 32 columns.  B patch rows are permuted so that those 16 are consecutive
// (16 (l / 32) .. +15): the two lanes of an output row write 64 contiguous bytes of BF16.
//
// A lane's operand is block l / 32 of a 64-long step; it shifts the row's scale word by 8 (l / 32) once per
// 128-long stretch, and the instruction's byte select (0 or 2) picks the step.  The words of a contraction's
// last stretch are masked past the last block (zero bytes, 2^-127 on both sides: the product of whatever codes
// lie there vanishes below FP32's range).
//
// Workgroups are persistent and the ring runs on across tiles, as in the FP8 kernel.
#include "gemm_kernel.hpp"
#include "mx_common.hpp"

namespace fp8bq {

constexpr int kMxStage = 256;  // values per stage

// B patch: MFMA row rho is tile row 16 ((rho / 4) % 2) + 4 (rho / 8) + rho % 4; rho of tile row n:
__device__ __forceinline__ int mx_rho(int n) { return 8 * ((n >> 2) & 3) + 4 * ((n >> 4) & 1) + (n & 3); }
__device__ __forceinline__ int mx_row_of_rho(int rho) {
  return 16 * ((rho >> 2) & 1) + 4 * (rho >> 3) + (rho & 3);
}

template <int BM, int BN, int NW>
struct MxTile {
  static constexpr int kB = BM * 128;
  static constexpr int kSA = (BM + BN) * 128;  // scale words [2][BM], then [2][BN]
  static constexpr int kSB = kSA + 2 * BM * 4;
  static constexpr int kStage = kSB + 2 * BN * 4;
  static constexpr int kBlocks = 4 * 2 * kStage + 4 * 8 * kMaxExperts <= 160 * 1024 ? 4
                                 : 2 * 2 * kStage + 2 * 8 * kMaxExperts <= 160 * 1024 ? 2 : 1;  // workgroups per CU
  // waves per SIMD that the launch bound keeps registers for
  static constexpr int kMinWaves = kBlocks * NW / 4;
};

template <int BM, int BN, int WGM, int WGN, int OUT, bool GROUPED>
__global__ __launch_bounds__(WGM* WGN * 64, (MxTile<BM, BN, WGM * WGN>::kMinWaves)) void mx_gemm_kernel(
    MxDesc d, uint32_t tiles_m, uint32_t tiles_n, int nsplit, float* __restrict__ partial, int64_t ldp, int vec,
    GroupArgs<GROUPED ? kGroupRowsMode : kGroupNone> grp) {
  constexpr int NW = WGM * WGN;
  using Tile = MxTile<BM, BN, NW>;
  constexpr int WTM = BM / WGM, WTN = BN / WGN;
  constexpr int MI = WTM / 32, NI = WTN / 32;
  constexpr int AL = BM / 8 / NW, BL = BN / 8 / NW;       // 1 KB code loads per wave and stage
  constexpr int SJA = 2 * BM / 64, SJ = SJA + 2 * BN / 64;  // scale jobs of 64 words
  constexpr int SL = SJ / NW;
  constexpr int LOADS = AL + BL + SL;
  static_assert(SJ % NW == 0 && BM / 8 % NW == 0 && BN / 8 % NW == 0, "loads split evenly over the waves");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * Tile::kStage];
  __shared__ uint32_t gunits[GROUPED ? kMaxExperts + 1 : 1];
  __shared__ int gstarts[GROUPED ? kMaxExperts + 1 : 1];

  const int t = threadIdx.x;
  const int lane = t & 63;
  const int wid = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wid / WGN, wn = wid % WGN;
  const int nblk = (int)(d.K / kMxBlock);
  const int nkb = (nblk + 7) / 8;
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
  int64_t sld[SL];  // words between a job's stretches, and its stretch within the stage
  int sword[SL];
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    const int j = wid + NW * i;
    sld[i] = j < SJA ? d.ldsa : d.ldsb;
    sword[i] = j < SJA ? j / (BM / 64) : (j - SJA) / (BN / 64);
  }
  auto set_sources = [&](const UnitT& u) {
    abase = (const uint8_t*)d.a + (int64_t)u.m0 * d.lda;
    bbase = d.b + (int64_t)u.n0 * d.ldb;
    const int64_t mleft = m_end(u) - 1 - u.m0, nleft = n_end(u) - 1 - u.n0;
    abytes = sat32((mleft < BM - 1 ? mleft : BM - 1) * d.lda + d.K / 2);
    bbytes = sat32((nleft < BN - 1 ? nleft : BN - 1) * d.ldb + d.K / 2);
#pragma unroll
    for (int i = 0; i < AL; ++i) {
      const int row = 8 * (wid + NW * i) + (lane >> 3);
      const int64_t r = row < mleft ? row : mleft;
      aoff[i] = (uint32_t)(r * d.lda) + (uint32_t)(((lane & 7) ^ swz(row)) * 16);
    }
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const int row = 8 * (wid + NW * i) + (lane >> 3);
      const int64_t r = row < nleft ? row : nleft;
      boff[i] = (uint32_t)(r * d.ldb) + (uint32_t)(((lane & 7) ^ swz(mx_rho(row))) * 16);
    }
    // scale job j: word p of 64 rows; p = j / (rows / 64) within A's jobs, then B's
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      const int j = wid + NW * i;
      if (j < SJA) {
        const int64_t r = 64 * (j % (BM / 64)) + lane;
        soff[i] = (uint32_t)((r < mleft ? r : mleft) * 4);
        sbase[i] = d.sa + u.m0;
        sbytes[i] = (uint32_t)((mleft < BM - 1 ? mleft : BM - 1) * 4 + 4);
      } else {
        const int64_t r = 64 * ((j - SJA) % (BN / 64)) + lane;
        soff[i] = (uint32_t)((r < nleft ? r : nleft) * 4);
        sbase[i] = d.sb + u.n0;
        sbytes[i] = (uint32_t)((nleft < BN - 1 ? nleft : BN - 1) * 4 + 4);
      }
    }
  };
  const int nwords = (nblk + 3) / 4;
  auto issue_load = [&](int i, uint8_t* stg) {
    if (i < AL) {
      dma16(rsrc_of(abase + (int64_t)lkb * 128, abytes - (uint32_t)lkb * 128), aoff[i], stg + (wid + NW * i) * 1024);
    } else if (i < AL + BL) {
      dma16(rsrc_of(bbase + (int64_t)lkb * 128, bbytes - (uint32_t)lkb * 128), boff[i - AL],
            stg + Tile::kB + (wid + NW * (i - AL)) * 1024);
    } else {
      const int q = i - AL - BL;
      const int word = 2 * lkb + sword[q];
      const bool in = word < nwords;  // (past the last word: zeros)
      dma4(rsrc_of(sbase[q] + (in ? word : 0) * sld[q], in ? sbytes[q] : 0u), soff[q],
           stg + Tile::kSA + 256 * (wid + NW * q));
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
  const int asw = swz(r32), bsw = swz(r32);  // (swz reads row % 16; patch rows start at multiples of 32)
  auto aread = [&](const uint8_t* stg, int i, int step) {
    return *reinterpret_cast<const v4i*>(stg + (arow + 32 * i) * 128 + (((2 * step + h) ^ asw) << 4));
  };
  auto bread = [&](const uint8_t* stg, int j, int step) {
    return *reinterpret_cast<const v4i*>(stg + Tile::kB + (brow + 32 * j) * 128 + (((2 * step + h) ^ bsw) << 4));
  };
  auto sread = [&](const uint8_t* stg, int p, uint32_t (&sa)[MI], uint32_t (&sb)[NI]) {
    const uint32_t* wa = reinterpret_cast<const uint32_t*>(stg + Tile::kSA) + p * BM + arow;
    const uint32_t* wb = reinterpret_cast<const uint32_t*>(stg + Tile::kSB) + p * BN + brow;
#pragma unroll
    for (int i = 0; i < MI; ++i) sa[i] = wa[32 * i];
#pragma unroll
    for (int j = 0; j < NI; ++j) sb[j] = wb[32 * j];
  };
  // keep the bytes of existing blocks and bring the lane's two to bytes 0 and 2
  auto smask = [&](int kb, int p, uint32_t (&sa)[MI], uint32_t (&sb)[NI]) {
    const int left = nblk - 8 * kb - 4 * p;
    const uint32_t mask = left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
#pragma unroll
    for (int i = 0; i < MI; ++i) sa[i] = (sa[i] & mask) >> (8 * h);
#pragma unroll
    for (int j = 0; j < NI; ++j) sb[j] = (sb[j] & mask) >> (8 * h);
  };

  v16f acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  set_sources(L);
  load_stage(smem);
  load_stage(smem + Tile::kStage);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(LOADS) : "memory");
  v4i fa[2][MI], fb[2][NI];
  uint32_t sa[2][MI], sb[2][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i) fa[0][i] = aread(smem, i, 0);
#pragma unroll
  for (int j = 0; j < NI; ++j) fb[0][j] = bread(smem, j, 0);
  sread(smem, 0, sa[0], sb[0]);

  int rd = 0;
  while (true) {
    uint8_t* stage = smem + rd * Tile::kStage;
    uint8_t* nstage = smem + (rd ^ 1) * Tile::kStage;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int cur = s & 1, nxt = cur ^ 1, p = s >> 1;
      if (s == 0 || s == 2) smask(ckb, p, sa[p], sb[p]);
      if (s < 3) {
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[nxt][i] = aread(stage, i, s + 1);
#pragma unroll
        for (int j = 0; j < NI; ++j) fb[nxt][j] = bread(stage, j, s + 1);
        if (s == 1) sread(stage, 1, sa[1], sb[1]);
      } else {
        // everything this wave needs of the stage is in registers; the next stage has landed
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
        for (int i = 0; i < LOADS; ++i) issue_load(i, stage);
#pragma unroll
        for (int i = 0; i < MI; ++i) fa[nxt][i] = aread(nstage, i, 0);
#pragma unroll
        for (int j = 0; j < NI; ++j) fb[nxt][j] = bread(nstage, j, 0);
        sread(nstage, 0, sa[0], sb[0]);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          if (s & 1)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(fb[cur][j]), mx_operand(fa[cur][i]),
                                                                        acc[i][j], 4, 4, 2, (int)sb[p][j], 2,
                                                                        (int)sa[p][i]);
          else
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(fb[cur][j]), mx_operand(fa[cur][i]),
                                                                        acc[i][j], 4, 4, 0, (int)sb[p][j], 0,
                                                                        (int)sa[p][i]);
        }
      __builtin_amdgcn_sched_barrier(0);
    }
    // keep the MFMAs in the step sequence (not sunk past the cursor update's branches)
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) asm volatile("" : "+v"(acc[i][j]));
    advance();
    rd ^= 1;
    if (++ckb < C.kb1) continue;

    // unit finished: write the tile or its partial sum.  Lane l: row l % 32 of each A patch, columns
    // 16 (l / 32) .. +15 of each B patch.
    {
      const int64_t mlim = m_end(C), nlim = n_end(C);
      const int64_t m = (int64_t)C.m0 + arow;
      int64_t ccol = 0;
      if constexpr (GROUPED) ccol = C.ccol;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int64_t row = m + 32 * i;
        if (row >= mlim) continue;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          const int64_t n = (int64_t)C.n0 + wn * WTN + 32 * j + 16 * h;
          const v16f& v = acc[i][j];
          const int64_t left = nlim - n;
          if (left <= 0) continue;
          if (nsplit > 1 || OUT != 0) {
            float* o = nsplit > 1 ? partial + ((int64_t)C.split * d.M + row) * ldp + n
                                  : reinterpret_cast<float*>(d.c) + row * d.ldc + n + ccol;
            if (left >= 16 && (nsplit > 1 || vec)) {
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                v4f w = {v[4 * r], v[4 * r + 1], v[4 * r + 2], v[4 * r + 3]};
                v4f* o4 = reinterpret_cast<v4f*>(o) + r;
                if (OUT == 2 && nsplit == 1) w = *o4 + w;
                *o4 = w;
              }
            } else {
#pragma unroll
              for (int r = 0; r < 16; ++r)
                if (r < left) o[r] = (OUT == 2 && nsplit == 1) ? o[r] + v[r] : v[r];
            }
          } else {
            uint16_t* o = reinterpret_cast<uint16_t*>(d.c) + row * d.ldc + n + ccol;
            uint32_t w[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) w[r] = pack_bf16x2(v[2 * r], v[2 * r + 1]);
            if (left >= 16 && vec) {
              *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4*>(o + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            } else {
#pragma unroll
              for (int r = 0; r < 16; ++r)
                if (r < left) o[r] = (uint16_t)(w[r >> 1] >> (16 * (r & 1)));
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

template <int BM, int BN, int WGM, int WGN, int OUT>
static hipError_t launch_tile(const MxDesc& d, const MxGroups& grp, const MxPlan& p, void* ws, int vec,
                              hipStream_t st) {
  const int64_t ldp = (d.N + 3) / 4 * 4;
  if (grp.offsets)
    hipLaunchKernelGGL((mx_gemm_kernel<BM, BN, WGM, WGN, OUT, true>), dim3((unsigned)p.grid), dim3(WGM * WGN * 64), 0,
                       st, d, (uint32_t)p.tiles_m, (uint32_t)p.tiles_n, 1, (float*)nullptr, ldp, vec,
                       GroupArgs<kGroupRowsMode>{grp.offsets, grp.experts, d.M});
  else
    hipLaunchKernelGGL((mx_gemm_kernel<BM, BN, WGM, WGN, OUT, false>), dim3((unsigned)p.grid), dim3(WGM * WGN * 64), 0,
                       st, d, (uint32_t)p.tiles_m, (uint32_t)p.tiles_n, p.split_k, (float*)ws, ldp, vec,
                       GroupArgs<kGroupNone>{});
  return hipGetLastError();
}

template <int OUT>
static hipError_t launch_out(const MxDesc& d, const MxGroups& grp, const MxPlan& p, void* ws, hipStream_t st) {
  const int vec = (d.ldc * (OUT == 0 ? 2 : 4)) % 16 == 0;
  hipError_t e;
  switch (p.shape) {
    case k256x256: e = launch_tile<256, 256, 2, 4, OUT>(d, grp, p, ws, vec, st); break;
    case k64x64: e = launch_tile<64, 64, 2, 2, OUT>(d, grp, p, ws, vec, st); break;
    default: e = launch_tile<128, 128, 2, 2, OUT>(d, grp, p, ws, vec, st); break;
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
