// Scaled FP8 GEMM kernel for gfx950 (CDNA4): fprop, dgrad and wgrad of the blockwise-quantized linear layer.
//
// The product ("小团队也能预训练！普罗2B：RTX5090训练成本不到5090美元", paragraph
// "FP8发挥RTX 5090的低精度效率优势"; "Puro-2B: Poor Lab's Qwen2-1.5B Trained on RTX 5090 within $5090",
// "方法关键点", bullet "FP8 blockwise 混合精度") is, in the kernel's TN frame,
//     C[m, n] = sum_kb sa(kb, m) * sb(kb, n) * sum_{k in kb} dec(A[m, k]) * dec(B[n, k])
// with FP32 accumulation and BF16 (or FP32) output.  One v_mfma_f32_16x16x128_f8f6f4 covers exactly
// one 128-long scale block of the contraction for a 16x16 output patch, so the kernel issues each
// MFMA with a zero accumulator and folds its result into the running FP32 sum with one FMA per
// output element: acc += mfma * (sa * sb).  Mixed formats (E5M2 gradients x E4M3 weights) are the
// instruction's per-operand format fields.
//
// Operand roles: the MFMA's first operand is the B patch (16 output columns) and its second the A
// patch (16 output rows).  A lane then holds output row (lane % 16) and four output columns of the B
// patch, so the A-side scale is one value per lane and patch.  For fprop and dgrad the B patches'
// rows are permuted so that a lane holds runs of 8 consecutive columns and the 4 lanes of an output
// row hold 32 consecutive columns: the epilogue writes 64 contiguous bytes of BF16 per row and store.
//
// Data movement: per 128-long contraction block the workgroup stages a BM x 128 A tile and a
// BN x 128 B tile in LDS (double-buffered, one barrier per block), with 16-byte chunks XOR-swizzled
// by row so the 16-byte fragment reads of 64 lanes spread over all banks.  Global loads for block
// kb+1 (and its scales) are issued before the MFMAs of block kb.  Workgroup ids are remapped so that
// each XCD (its own L2) works on a contiguous, row-grouped region of output tiles.

#pragma once

#include <type_traits>

#include "device_common.hpp"
#include "group_table.hpp"
#include "launch.hpp"

namespace fp8bq {


// 16-byte chunk swizzle inside a 128-byte LDS row.  It depends on row % 16 only, so every 16-row
// patch has the same per-lane read pattern (one pair of lane offsets serves all patches; the patch
// position goes into the instruction's immediate offset).  Conflict-free for 8-lane phases (rows
// 0-7 and 8-15 each get 8 distinct chunks) and for 16-lane phases over 64 banks (rows of equal
// parity get distinct chunks).
__device__ __forceinline__ int swz(int row) { return (row ^ ((row >> 3) & 1)) & 7; }

constexpr int kGroupRows = 8;  // output tile rows per L2 group
constexpr int kXcds = 8;

// Bijective remap of the hardware workgroup id (dispatched round-robin over the XCDs) to a logical
// tile id so each XCD processes a contiguous range of logical ids, then row-grouped tile ordering.
// 32-bit arithmetic (the planner keeps tile and unit counts below 2^31); the results are wave-uniform
// and kept in scalar registers.
__device__ __forceinline__ void tile_of(uint32_t w, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn) {
  const uint32_t nblk = tiles_m * tiles_n;
  const uint32_t q8 = nblk / kXcds, r8 = nblk % kXcds;
  const uint32_t x = w % kXcds;
  const uint32_t L = x * q8 + (x < r8 ? x : r8) + w / kXcds;
  const uint32_t group = (uint32_t)kGroupRows * tiles_n;
  const uint32_t gid = L / group;
  const uint32_t first = gid * kGroupRows;
  const uint32_t gsz = (tiles_m - first) < (uint32_t)kGroupRows ? (tiles_m - first) : (uint32_t)kGroupRows;
  const uint32_t rem = L - gid * group;
  tm = __builtin_amdgcn_readfirstlane(first + rem % gsz);
  tn = __builtin_amdgcn_readfirstlane(rem / gsz);
}

template <int FA, int FB>
__device__ __forceinline__ v4f mfma_block(const v8i& bpatch, const v8i& apatch) {
  const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
  // cbsz = format of the first operand (B patch), blgp = format of the second (A patch);
  // zero E8M0 scale operands select the unscaled instruction.
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bpatch, apatch, zero, FB, FA, 0, 0, 0, 0);
}

// Byte offsets, within a 16-row patch, of the two 16-byte chunks lane reads: row lane % 16, logical
// chunks 2*(lane/16) and 2*(lane/16)+1 (32 consecutive contraction bytes).
struct PatchLane {
  int lo, hi;
};
__device__ __forceinline__ PatchLane patch_lane(int lane) {
  const int r = lane & 15, s = swz(r), c0 = 2 * (lane >> 4);
  return PatchLane{r * 128 + ((c0 ^ s) << 4), r * 128 + (((c0 + 1) ^ s) << 4)};
}
// B-side patches are permuted: row rho of B patch j (a wave's four patches of 16 output columns)
// is output column 8*(rho/4) + 32*(j/2) + 4*(j%2) + rho%4 of the wave's 64 columns.  Lane l then
// holds, for patches 2t and 2t+1, the 8 consecutive columns 32*t + 8*(l/16) .. +7 of its output row,
// so the four lanes of a row write 64 contiguous bytes per store.  B tile rows get their own chunk
// swizzle: lane l's row 8*(rho/4) + rho%4 (rho = l % 16) takes the swizzle A-side row rho has, so
// every lane of a B-patch read hits exactly the bank of the same lane's A-patch read, and the two
// reads conflict alike on any grouping of lanes into LDS phases (A's pattern is conflict-free).  It
// ignores row bit 2 and bits 5 and up, so it is the same for all four patches (their rows differ by
// 32*(j/2) + 4*(j%2)) and for every wave column.
__device__ __forceinline__ int swzb(int row) { return swz(4 * ((row >> 3) & 3) + (row & 3)); }
__device__ __forceinline__ PatchLane b_patch_lane(int lane) {
  const int rho = lane & 15, r = 8 * (rho >> 2) + (rho & 3), s = swzb(r), c0 = 2 * (lane >> 4);
  return PatchLane{r * 128 + ((c0 ^ s) << 4), r * 128 + (((c0 + 1) ^ s) << 4)};
}
// The MFMA operand of the 16-row patch starting at patch_base (a multiple of 16 rows into a tile).
__device__ __forceinline__ v8i lds_patch(const uint8_t* patch_base, PatchLane pl) {
  const v4i lo = *reinterpret_cast<const v4i*>(patch_base + pl.lo);
  const v4i hi = *reinterpret_cast<const v4i*>(patch_base + pl.hi);
  v8i r = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  return r;
}

typedef __attribute__((address_space(3))) void lds_void;

// Raw buffer descriptor over [base, base + bytes): loads past the end read zeros instead of
// faulting.  Word 3 is the gfx9 raw-buffer format word.
constexpr int kRsrcWord3 = 0x00020000;
__device__ __forceinline__ uint32_t sat32(int64_t bytes) {
  return bytes < 0 ? 0u : (bytes < (int64_t)0xFFFFFFFF ? (uint32_t)bytes : 0xFFFFFFFFu);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, kRsrcWord3);
}

// One 16-byte (or 4-byte) load per lane from byte offset voff of the buffer, written straight into
// LDS at lds_base + 16 * lane (or 4 * lane): buffer_load_dwordx4 / _dword with the lds flag.
// lds_base must be the same for the whole wave.  (Buffer loads rather than global_load_lds: the
// compiler then keeps exact counts for the waits on LDS reads.)
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint8_t* lds_base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds_base, 16, voff, 0, 0, 0);
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint8_t* lds_base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds_base, 4, voff, 0, 0, 0);
}

// One work unit: an output tile and the range of 128-long contraction blocks it sums.
struct Unit {
  int m0, n0;
  int kb0, kb1, split;
};

template <int BM, int BN>
__device__ __forceinline__ Unit unit_of(uint32_t u, uint32_t tiles_m, uint32_t tiles_n, int nsplit, int nkb) {
  const uint32_t T = tiles_m * tiles_n;
  const uint32_t w = u % T;
  const int s = (int)(u / T);
  uint32_t tm, tn;
  tile_of(w, tiles_m, tiles_n, tm, tn);
  Unit r;
  r.m0 = (int)tm * BM;
  r.n0 = (int)tn * BN;
  r.kb0 = __builtin_amdgcn_readfirstlane(s * nkb / nsplit);
  r.kb1 = __builtin_amdgcn_readfirstlane((s + 1) * nkb / nsplit);
  r.split = __builtin_amdgcn_readfirstlane(s);
  return r;
}

// Products grouped by expert.  The tokens of expert e are the rows offsets[e] .. offsets[e+1]-1 of
// the activation side and the experts' weights are stacked, so a work unit is a tile of one expert
// with its own row limits and operand positions; the tile loop is the dense product's.  The expert of
// a unit comes from a table of unit counts that each workgroup builds in LDS from the offsets on the
// device (group_table.hpp), so the host never waits for the counts.
//   kGroupRowsMode  fprop: A rows are an expert's tokens, B rows (and scale blocks) its stacked weights;
//   kGroupWindow    dgrad: A rows are an expert's tokens, the contraction runs over the expert's window
//                   of the columns of W^T [K, E N];
//   kGroupContract  wgrad: the contraction runs over an expert's 128-token blocks (operands quantized
//                   along the tokens, every expert's tokens padded to whole blocks); C is stacked.
// Bound by the matrix pipes at the clock the card's power allows, as the dense products, and by what ragged
// experts add.  32768 tokens, us with the operands from HBM (kernel trace), and one after the other on the same ones
// where that differs: fprop on 64 experts of 2816 x 2048 235-240 (1.6 PFLOP/s; matrix pipes busy 47% of the cycles; a
// tenth of the tiles' rows are past an expert's end); on 32 experts of 2048 x 1408 dgrad 135-141, 102-111 (35%; the dense
// product of that size 100) and wgrad 174-185, 141-149 (32%; dense, contracted in one piece, 125): 32 times the outputs,
// 184 MB, which a workgroup writes at the end of a round while its matrix pipes idle.  wgrad into FP32 there 165-190, added
// to FP32 284-299: the old values are read where they are added, with nothing between to hide it.
enum GroupMode : int { kGroupNone = 0, kGroupRowsMode = 1, kGroupWindow = 2, kGroupContract = 3 };
template <int GM>
struct GroupArgs {
  const int64_t* offsets;  // E + 1 token offsets (device)
  int experts;
  int64_t tokens;  // rows of the activation side; for kGroupContract the padded tokens
};
template <>
struct GroupArgs<kGroupNone> {};
template <>
struct GroupArgs<kGroupContract> {
  const int64_t* offsets;
  int experts;
  int64_t tokens;  // padded tokens
  GroupSplit split;
  uint32_t* split_list;
};

enum GroupPart : int { kPartAll = 0, kPartTall = 1, kPartRest = 2 };

struct GroupUnit : Unit {
  int mend, nend;    // ends of the unit's A rows and B rows
  int bkb;           // contraction blocks by which B's columns are ahead of A's
  int64_t crow;      // output row and column of A row m and B row n: m + crow, n + ccol
  int64_t ccol;
  bool whole;        // else the unit's sum is partial, set `split` of the workspace
};

// The unit u of a grouped product.  Rows: units of all experts in expert order, remapped over the XCDs as in
// tile_of; within an expert the row-grouped tile order.  Contraction: the long experts first, in chunks where they are
// split (group_table_blocks), and a chunk's tiles dealt out over the XCDs (with 8 tile rows, a tile row each), so
// that no XCD has the long ones.  PART: kPartTall or kPartRest take an expert's row tiles of tall_tiles() or the
// one short tile after them.
template <int GM, int BM, int BN, int PART = kPartAll>
__device__ __forceinline__ GroupUnit group_unit_of(uint32_t u, const uint32_t* units, const int* starts, int E,
                                                   int M, int N, int nkb, int lane) {
  const uint32_t tiles_n = (uint32_t)((N + BN - 1) / BN);
  int e;
  uint32_t w;
  GroupEntry entry{0, 1, 0, 0};
  if constexpr (GM == kGroupContract) {
    const uint32_t tiles = tiles_n * (uint32_t)((M + BM - 1) / BM);
    entry = entry_of((uint32_t)__builtin_amdgcn_readfirstlane((int)units[u / tiles]));
    e = entry.expert;
    w = u % tiles;
  } else {
    const uint32_t U = units[E];
    const uint32_t q8 = U / kXcds, r8 = U % kXcds;
    const uint32_t x = u % kXcds;
    const uint32_t Lx = x * q8 + (x < r8 ? x : r8) + u / kXcds;
    e = group_find(units, E, Lx, lane);
    w = Lx - units[e];
  }
  const int s0 = starts[e], s1 = starts[e + 1];
  const uint32_t tiles_m = GM == kGroupContract ? (uint32_t)((M + BM - 1) / BM)
                           : PART == kPartAll   ? (uint32_t)((s1 - s0 + BM - 1) / BM)
                           : PART == kPartTall  ? (uint32_t)tall_tiles(s1 - s0)
                                                : 1u;
  const uint32_t group = (uint32_t)kGroupRows * tiles_n;
  const uint32_t gid = w / group;
  const uint32_t first = gid * kGroupRows;
  const uint32_t gsz = (tiles_m - first) < (uint32_t)kGroupRows ? (tiles_m - first) : (uint32_t)kGroupRows;
  const uint32_t rem = w - gid * group;
  const int tm = __builtin_amdgcn_readfirstlane((int)(first + rem % gsz));
  const int tn = __builtin_amdgcn_readfirstlane((int)(rem / gsz));
  GroupUnit r;
  r.split = entry.set + entry.chunk;
  r.whole = entry.chunks == 1;
  if constexpr (GM == kGroupContract) {
    r.m0 = tm * BM;
    r.mend = M;
    r.kb0 = __builtin_amdgcn_readfirstlane(s0);
    r.kb1 = __builtin_amdgcn_readfirstlane(s1);
    if (entry.chunks > 1) {
      const int b = r.kb0, n = r.kb1 - b;
      r.kb0 = b + n * entry.chunk / entry.chunks;
      r.kb1 = b + n * (entry.chunk + 1) / entry.chunks;
    }
    r.crow = (int64_t)__builtin_amdgcn_readfirstlane(e) * M;
  } else {
    r.m0 = __builtin_amdgcn_readfirstlane(s0 + (PART == kPartRest ? kTall * tall_tiles(s1 - s0) : 0)) + tm * BM;
    r.mend = __builtin_amdgcn_readfirstlane(s1);
    r.kb0 = 0;
    r.kb1 = nkb;
    r.crow = 0;
  }
  const int es = __builtin_amdgcn_readfirstlane(e);
  r.bkb = GM == kGroupWindow ? es * nkb : 0;
  const int nbase = GM == kGroupRowsMode ? es * N : 0;  // (E N < 2^31: checked by the caller)
  r.n0 = nbase + tn * BN;
  r.nend = nbase + N;
  r.ccol = -(int64_t)nbase;
  return r;
}

// OP (fprop / dgrad / wgrad) only names the instance, so profiles attribute time per product.
//
// Persistent workgroups: workgroup b processes work units b, b + G, b + 2G, ... (G = grid size, a
// multiple of 8 when there is more than one round, so every unit of a workgroup maps to its XCD's
// contiguous range in tile_of).  A unit is one BM x BN output tile and a range of contraction blocks
// (all of them, or 1/nsplit when the contraction is split; split units write FP32 partial sums that
// a separate pass adds in a fixed order).  The LDS ring runs continuously across units: the loads
// for a unit's first block are issued while the previous unit's last block is multiplied and its
// tile is written out.
//
// LDS stage layout (NSTAGE stages, a ring): [A tile BM x 128 B][B tile BN x 128 B][A scales BM x f32]
// [B scales: BN x f32 (per-column mode) or one f32 per 128 columns (per-block mode), 64 slots min]
// [256 B sink for padding loads].  Tiles and scales arrive by direct global->LDS loads: wave w fills
// 1 KB chunks w, w+NW, ... (8 rows each); lane l of a chunk fetches the 16 bytes that belong at LDS
// offset 16*l, i.e. row l/8 and physical chunk l%8, whose logical chunk is (l%8) ^ swz(row).  Every
// wave issues the same number of loads per stage (scale jobs are padded with loads into the sink), so
// one s_waitcnt vmcnt(loads per stage) leaves exactly the newest stage in flight.
// Workgroups per CU that the LDS ring allows for a 4-wave tile (the planner's slots per CU: four for
// 64x64, two for 128x128); the launch bound then keeps the registers low enough for that residency.
template <int BM, int BN, int NW, int NSTAGE>
struct StageMinBlocks {
  static constexpr int kStage = (BM + BN) * 128 + BM * 4 + 64 * 4 + 256;  // lower bound of STAGE
  static constexpr int value = NW != 4 ? 1 : 4 * NSTAGE * kStage <= 160 * 1024 ? 4 : 2 * NSTAGE * kStage <= 160 * 1024 ? 2 : 1;
};

template <int BM, int BN, int NSTAGE, int SBM>
constexpr int ring_bytes() {
  constexpr int NSB = SBM == kSbColumn ? BN : ((BN + kGroup - 1) / kGroup);
  return NSTAGE * ((BM + BN) * 128 + BM * 4 + (NSB > 64 ? NSB : 64) * 4 + 256);
}

// The work units first, first + G, ... below U of one tile shape.  smem: the ring, ring_bytes() long; gunits and
// gstarts: the table of a grouped product.
template <int OP, int BM, int BN, int WGM, int WGN, int NSTAGE, int SBM, int FA, int FB, int OUTF32, int GM, int PART>
__device__ __forceinline__ void gemm_tn_units(const GemmDesc& d, uint32_t tiles_m, uint32_t tiles_n, int nsplit,
                                              float* __restrict__ partial, const GroupArgs<GM>& grp, uint8_t* smem,
                                              const uint32_t* gunits, const int* gstarts, uint32_t U, uint32_t first) {
  constexpr int NW = WGM * WGN;
  constexpr bool GROUPED = GM != kGroupNone;
  constexpr int WTM = BM / WGM;
  constexpr int WTN = BN / WGN;
  constexpr int MI = WTM / 16;
  constexpr int NI = WTN / 16;
  constexpr int SA_OFF = (BM + BN) * 128;
  constexpr int NSB = SBM == kSbColumn ? BN : ((BN + kGroup - 1) / kGroup);  // (a 64-wide tile: one block)
  constexpr int SB_OFF = SA_OFF + BM * 4;
  constexpr int SINK_OFF = SB_OFF + (NSB > 64 ? NSB : 64) * 4;
  constexpr int STAGE = SINK_OFF + 256;
  constexpr int ACHUNKS = BM / 8, BCHUNKS = BN / 8;  // 1 KB chunks per stage
  constexpr int SAJOBS = BM / 64;                     // 64 scales per wave job
  constexpr int SBJOBS = NSB > 64 ? NSB / 64 : 1;
  constexpr int SJOBS = SAJOBS + SBJOBS;
  constexpr int JPW = (SJOBS + NW - 1) / NW;          // scale jobs per wave (padded)
  // B patch rows permuted for 16-byte BF16 stores (fprop / dgrad); the per-column-scale product
  // (wgrad), mostly written as FP32 partial sums, keeps natural order (64-byte FP32 runs per row)
  constexpr bool PERM = SBM == kSbBlock128;
  static_assert(!PERM || NI == 4, "the B-side permutation is laid out for 64-column wave tiles");
  constexpr int LOADS = ACHUNKS / NW + BCHUNKS / NW + JPW;  // loads per wave per stage
  static_assert(ACHUNKS % NW == 0 && BCHUNKS % NW == 0, "tile chunks must split evenly over waves");
  static_assert(BM % 64 == 0 && (NSB <= 64 || NSB % 64 == 0), "scale jobs are 64 lanes wide");
  static_assert(SBM != kSbBlock128 || WTN <= 128, "a wave's columns must share one weight block");
  static_assert(SBM != kSbBlock128 || BN % kGroup == 0 || kGroup % BN == 0, "a narrow tile lies in one weight block");
  static_assert(NSTAGE >= 2 && NSTAGE * STAGE <= 160 * 1024, "LDS ring does not fit");
  static_assert(ring_bytes<BM, BN, NSTAGE, SBM>() == NSTAGE * STAGE, "ring size");

  const int t = threadIdx.x;
  const int lane = t & 63;
  const int wid = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wid / WGN, wn = wid % WGN;
  const int64_t M = d.M, N = d.N;
  const int nkb = (int)(d.K / kGroup);
  const uint32_t G = gridDim.x;

  using UnitT = std::conditional_t<GROUPED, GroupUnit, Unit>;
  auto unit_at = [&](uint32_t u) {
    if constexpr (GROUPED)
      return group_unit_of<GM, BM, BN, PART>(u, gunits, gstarts, grp.experts, (int)M, (int)N, nkb, lane);
    else
      return unit_of<BM, BN>(u, tiles_m, tiles_n, nsplit, nkb);
  };
  auto m_end = [&](const UnitT& u) -> int64_t {
    if constexpr (GROUPED) return u.mend; else return M;
  };
  auto n_end = [&](const UnitT& u) -> int64_t {
    if constexpr (GROUPED) return u.nend; else return N;
  };

  if (first >= U) return;
  // load-side cursor: unit lu, block lkb, and this lane's sources for that unit as 32-bit offsets
  // from workgroup-uniform bases (rows past the end are clamped; their results are never stored)
  uint32_t lu = first;
  UnitT L = unit_at(lu);
  int lkb = L.kb0;
  bool lmore = true;
  const uint8_t* abase = d.a;
  const uint8_t* bbase = d.b;
  uint32_t abytes = 0, bbytes = 0;  // from abase / bbase to the end of the tile's last valid row
  uint32_t aoff[ACHUNKS / NW], boff[BCHUNKS / NW];
  const float* gs[JPW];  // scale job q: array base (wave-uniform), per-lane byte offset, kb stride
  int64_t gsk[JPW];
  uint32_t gsbytes[JPW];
  uint32_t gvo[JPW];
  int lso[JPW];
  auto set_sources = [&](const UnitT& u) {
    abase = d.a + (int64_t)u.m0 * d.lda;
    bbase = d.b + (int64_t)u.n0 * d.ldb;
    if constexpr (GM == kGroupWindow) bbase += (int64_t)u.bkb * kGroup;
    const int64_t mlim = m_end(u), nlim = n_end(u);
    const int64_t mleft = mlim - 1 - u.m0, nleft = nlim - 1 - u.n0;
    abytes = sat32((mleft < BM - 1 ? mleft : BM - 1) * d.lda + d.K);
    bbytes = sat32((nleft < BN - 1 ? nleft : BN - 1) * d.ldb + d.K);
#pragma unroll
    for (int i = 0; i < ACHUNKS / NW; ++i) {
      const int row = 8 * (wid + NW * i) + (lane >> 3);
      const int64_t r = row < mleft ? row : mleft;
      aoff[i] = (uint32_t)(r * d.lda) + (uint32_t)(((lane & 7) ^ swz(row)) * 16);
    }
#pragma unroll
    for (int i = 0; i < BCHUNKS / NW; ++i) {
      const int row = 8 * (wid + NW * i) + (lane >> 3);
      const int64_t r = row < nleft ? row : nleft;
      boff[i] = (uint32_t)(r * d.ldb) + (uint32_t)(((lane & 7) ^ (PERM ? swzb(row) : swz(row))) * 16);
    }
    // scale jobs: job j < SAJOBS loads A scales of rows 64j..64j+63, the next SBJOBS the B scales;
    // wave w runs jobs w, w+NW, ...; missing jobs load a valid scale into the sink
#pragma unroll
    for (int q = 0; q < JPW; ++q) {
      const int j = wid + NW * q;
      if (j < SAJOBS) {
        int64_t m = u.m0 + 64 * j + lane;
        m = m < mlim ? m : mlim - 1;
        gs[q] = d.sa;
        gvo[q] = (uint32_t)(m * 4 * d.sa_mstride);
        gsk[q] = d.ldsa;
        gsbytes[q] = d.sa_mstride ? sat32(M * 4) : 4;
        lso[q] = SA_OFF + 256 * j;
      } else if (j < SJOBS) {
        const int v = j - SAJOBS;
        gs[q] = d.sb;
        if constexpr (GM == kGroupWindow) gs[q] += (int64_t)u.bkb * d.sb_kstride;
        if constexpr (SBM == kSbColumn) {
          int64_t n = u.n0 + 64 * v + lane;
          n = n < nlim ? n : nlim - 1;
          gvo[q] = (uint32_t)(n * 4);
          gsbytes[q] = sat32(N * 4);
        } else {
          const int64_t nbl = nlim / kGroup;
          int64_t nb = u.n0 / kGroup + (lane < NSB ? lane : NSB - 1);
          nb = nb < nbl ? nb : nbl - 1;
          gvo[q] = (uint32_t)(nb * d.sb_nstride * 4);
          gsbytes[q] = sat32(((nbl - 1) * d.sb_nstride + 1) * 4);
        }
        gsk[q] = d.sb_kstride;
        lso[q] = SB_OFF + 256 * v;
      } else {
        gs[q] = d.sa;
        gvo[q] = 0;
        gsk[q] = 0;
        gsbytes[q] = 4;
        lso[q] = SINK_OFF;
      }
    }
  };
  // Issue the loads of (lu, lkb) into stg, then advance the cursor.  Once every block has been
  // issued the cursor stays on the last one and further calls load it again into the free slot:
  // every call issues exactly LOADS loads, so one constant s_waitcnt serves every iteration and no
  // branch separates the MFMAs from their folds.  (A slot refilled that way is never read: it would
  // hold a block past the end.)
  // load number i (0 <= i < LOADS) of this wave for the current cursor position
  auto issue_load = [&](int i, uint8_t* stg) {
    if (i < ACHUNKS / NW) {
      dma16(rsrc_of(abase + lkb * kGroup, abytes - (uint32_t)(lkb * kGroup)), aoff[i], stg + (wid + NW * i) * 1024);
    } else if (i < ACHUNKS / NW + BCHUNKS / NW) {
      const int b = i - ACHUNKS / NW;
      dma16(rsrc_of(bbase + lkb * kGroup, bbytes - (uint32_t)(lkb * kGroup)), boff[b],
            stg + BM * 128 + (wid + NW * b) * 1024);
    } else {
      const int q = i - ACHUNKS / NW - BCHUNKS / NW;
      dma4(rsrc_of(gs[q] + (int64_t)lkb * gsk[q], gsbytes[q]), gvo[q], stg + lso[q]);
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
  auto load_next = [&](uint8_t* stg) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) issue_load(i, stg);
    advance();
  };
  // Every wave waits for its own loads of the next block, then the barrier makes them (and the end
  // of all reads of the current block's slot) visible workgroup-wide.  No memory fence: loads of
  // the blocks after the next stay in flight across the barrier.
  auto stage_barrier = [&]() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NSTAGE - 2) * LOADS) : "memory");
  };

  v4f acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};

  set_sources(L);
  // compute-side cursor
  uint32_t cu = lu;
  UnitT C = L;
  int ckb = C.kb0;

  // The side with fewer 16-row patches stays in registers for the whole block ("resident"); the
  // other side is streamed one patch at a time.  MFMA order: streamed patch outer, except for the
  // last TAILN streamed patches (the tail), which alternate (resident patch outer) so that resident
  // patch k is free after MFMA TAILN*k + TAILN-1 of the tail.
  constexpr bool STREAM_B = NI > MI;
  constexpr int NOUT = STREAM_B ? NI : MI;  // streamed patches
  constexpr int NIN = STREAM_B ? MI : NI;   // resident patches
  constexpr int NTILE = MI * NI;
  // MFMA u is folded LAG steps after its issue.  Three steps leave the result complete before the
  // fold reads it (the compiler's VALU-after-MFMA wait states drop from 13 to 3 per block, +2-4% on
  // fprop/dgrad); wgrad, whose fold is twice as long and whose registers are fuller, keeps two.
  constexpr int LAG = SBM == kSbBlock128 ? 3 : 2;
#ifndef FP8BQ_TAILN
#define FP8BQ_TAILN 3
#endif
  constexpr int TAILN = (PERM && NOUT >= 6) ? FP8BQ_TAILN : 2;  // streamed patches in the tail
  constexpr int TAIL0 = (NOUT - TAILN) * NIN;  // first MFMA of the tail
  constexpr int UB = TAIL0 + TAILN - 1;        // step that ends with the stage barrier
  constexpr int NPOST = NTILE + LAG - UB - 1;  // steps after it
  static_assert(NOUT >= TAILN && NPOST >= 1, "tile too small for the pipelined order");
  auto order = [&](int u, int& o, int& k) {
    if (u < TAIL0) {
      o = u / NIN;
      k = u % NIN;
    } else {
      o = NOUT - TAILN + (u - TAIL0) % TAILN;
      k = (u - TAIL0) / TAILN;
    }
  };
  const PatchLane pl = patch_lane(lane);
  const PatchLane plb = PERM ? b_patch_lane(lane) : pl;
  auto apatch = [&](const uint8_t* stg, int i) { return lds_patch(stg + wm * WTM * 128 + 16 * i * 128, pl); };
  auto bpatch = [&](const uint8_t* stg, int j) {
    return lds_patch(stg + BM * 128 + wn * WTN * 128 + (PERM ? (4096 * (j >> 1) + 512 * (j & 1)) : 2048 * j), plb);
  };
  auto streamed = [&](const uint8_t* stg, int o) { return STREAM_B ? bpatch(stg, o) : apatch(stg, o); };
  auto resident = [&](const uint8_t* stg, int k) { return STREAM_B ? apatch(stg, k) : bpatch(stg, k); };
  // Streamed patches are read RA patches ahead of their first MFMA (two where the registers allow).
  constexpr int RA = (PERM && NOUT >= 3) ? 2 : 1;
  // The next block's first reads (its resident patches and first RA streamed patches), in the order
  // the current block's tail frees their registers: read h goes out at tail step 2 + 2h.
  constexpr int NHEAD = NIN + RA;
  auto head_read = [&](const uint8_t* stg, int h, v8i* res, v8i* str) {
    if (h == 0) res[0] = resident(stg, 0);
    else if (h <= RA) str[h - 1] = streamed(stg, h - 1);
    else res[h - RA] = resident(stg, h - RA);
  };

  // prologue: every ring slot's block in flight, the first landed, its first reads issued
  v8i res[NIN], str[NOUT];
#pragma unroll
  for (int s = 0; s < NSTAGE; ++s) load_next(smem + s * STAGE);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((NSTAGE - 1) * LOADS) : "memory");
#pragma unroll
  for (int h = 0; h < NHEAD; ++h) head_read(smem, h, res, str);

  int rd = 0;  // ring slot of the block multiplied this iteration
  while (true) {
    const int nx = rd + 1 == NSTAGE ? 0 : rd + 1;
    const uint8_t* stage = smem + rd * STAGE;
    const uint8_t* nstage = smem + nx * STAGE;

    // Step u issues MFMA u (and the read-ahead of the next streamed patch) and the fold of MFMA
    // u-LAG, whose result is then complete; a scheduling fence closes every step, so the matrix pipe
    // never waits on a fold and at most LAG+1 MFMA results are live.  Step UB ends with the stage
    // barrier: every wave has read all it needs of this block (the tail's operands are in registers)
    // and the next block has landed.  The steps after it refill this block's slot with the block
    // NSTAGE ahead and read the next block's first patches while the tail's MFMAs run.
    const float* ssa = reinterpret_cast<const float*>(stage + SA_OFF);
    const float* ssb = reinterpret_cast<const float*>(stage + SB_OFF);
    float sa_[MI];
#pragma unroll
    for (int i = 0; i < MI; ++i) sa_[i] = ssa[wm * WTM + 16 * i + (lane & 15)];
    float sbv = 0.0f;
    v4f sbc[NI];
    if constexpr (SBM == kSbBlock128) {
      sbv = ssb[(wn * WTN) / kGroup];
    } else {
#pragma unroll
      for (int j = 0; j < NI; ++j)
        sbc[j] = *reinterpret_cast<const v4f*>(ssb + wn * WTN + 16 * j + 4 * (lane >> 4));
    }
    v4f p[NTILE];
    // Several workgroups per CU (one wave of each per SIMD): a wave runs its MFMA steps at raised
    // priority and drops back at the stage barrier, so the workgroups drift out of phase instead of
    // contending for the matrix pipe and the refill at the same time (+6% on a 128x128-tile wgrad;
    // neutral with one workgroup per CU, where it is not used).
    constexpr bool PRIO = StageMinBlocks<BM, BN, NW, NSTAGE>::value >= 2;
    if constexpr (PRIO) __builtin_amdgcn_s_setprio(1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < NTILE + LAG; ++u) {
      if (u < NTILE) {
        int o, k;
        order(u, o, k);
        if (k == 0 && o + RA < NOUT) str[o + RA] = streamed(stage, o + RA);
        p[u] = STREAM_B ? mfma_block<FA, FB>(str[o], res[k]) : mfma_block<FA, FB>(res[k], str[o]);
      }
      if (u == UB) {
        stage_barrier();
        if constexpr (PRIO) __builtin_amdgcn_s_setprio(0);
      }
      if (u > UB) {
        const int t = u - UB - 1;  // post-barrier step 0 .. NPOST-1
#pragma unroll
        for (int i = t * LOADS / NPOST; i < (t + 1) * LOADS / NPOST; ++i) issue_load(i, smem + rd * STAGE);
      }
      if (u >= UB && (u - UB) % 2 == 1 && (u - UB) / 2 < NHEAD) head_read(nstage, (u - UB) / 2, res, str);
      if (u >= LAG) {
        int o, k;
        order(u - LAG, o, k);
        const int v = u - LAG;
        const int i = STREAM_B ? k : o, j = STREAM_B ? o : k;
        if constexpr (SBM == kSbBlock128) {
          const float sc = sa_[i] * sbv;
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[v][r], sc, acc[i][j][r]);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[v][r], sa_[i] * sbc[j][r], acc[i][j][r]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // head reads that did not fit into the steps
#pragma unroll
    for (int h = 0; h < NHEAD; ++h)
      if (UB + 1 + 2 * h >= NTILE + LAG) head_read(nstage, h, res, str);
    // keep the folds in the step sequence (not sunk past the cursor update's branches)
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) asm volatile("" : "+v"(acc[i][j]));
    advance();
    rd = nx;

    if (++ckb < C.kb1) continue;

    // unit finished: write the tile (or its partial sum) and move on.  Lane l holds row l % 16 of
    // each 16-row A patch and, of the wave's 64 columns, 8*(l/16) + 32*(j/2) + 4*(j%2) .. +3 for
    // patch j (permuted B rows) or 16*j + 4*(l/16) .. +3 (natural order); only tiles that reach past
    // M or N check bounds.
    {
      // (the lane's place in the output is worked out here: kept in registers over the loop it cost spills)
      int el = lane;
      asm volatile("" : "+v"(el));
      const int64_t mrow = (int64_t)C.m0 + wm * WTM + (el & 15);
      const int64_t ncol = (int64_t)C.n0 + wn * WTN + (PERM ? 8 : 4) * (el >> 4);
      auto jcol = [](int j) { return PERM ? 32 * (j >> 1) + 4 * (j & 1) : 16 * j; };  // patch j's offset from ncol
      const int64_t mlim = m_end(C), nlim = n_end(C);
      const bool full = (int64_t)C.m0 + BM <= mlim && (int64_t)C.n0 + BN <= nlim;
      int64_t crow = mrow, ccol = ncol;  // output position of (mrow, ncol)
      if constexpr (GROUPED) {
        crow += C.crow;
        ccol += C.ccol;
      }
      bool part = nsplit > 1;  // a partial sum of the contraction
      if constexpr (GM == kGroupContract) {
        part = !C.whole;
        if (part) crow = mrow;
      }
      const bool past = d.past && !part;  // (partial sums are read again at once)
      auto write = [&](auto checked) {
        constexpr bool CHK = decltype(checked)::value;
        if (part || OUTF32) {
          const int64_t ldc = part ? N : d.ldc;
          float* c0 = (part ? partial + (int64_t)C.split * M * N : reinterpret_cast<float*>(d.c)) + crow * ldc + ccol;
          if constexpr (!CHK && !PERM && NI % 2 == 0) {
            // whole lines here too: patches j and j + 1 are 32 consecutive columns
            const int h = (el >> 3) & 1;
            c0 += -8 * h * ldc + 16 * h;
#pragma unroll
            for (int i = 0; i < MI; ++i) {
#pragma unroll
              for (int j = 0; j < NI; j += 2) {
                v4i upper, lower;
                join_halves(__builtin_bit_cast(v4i, acc[i][j]), __builtin_bit_cast(v4i, acc[i][j + 1]), upper, lower);
                v4f* cu = reinterpret_cast<v4f*>(c0 + 16 * i * ldc + 16 * j);
                v4f* cl = reinterpret_cast<v4f*>(c0 + (16 * i + 8) * ldc + 16 * j);
                v4f u = __builtin_bit_cast(v4f, upper), l = __builtin_bit_cast(v4f, lower);
                if (OUTF32 == 2 && !part) {
                  u = *cu + u;
                  l = *cl + l;
                }
                store_line(u, cu, past && OUTF32 != 2);
                store_line(l, cl, past && OUTF32 != 2);
              }
            }
            return;
          }
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            float* ci = c0 + 16 * i * ldc;
#pragma unroll
            for (int j = 0; j < NI; ++j) {
              if (CHK && !(mrow + 16 * i < mlim && ncol + jcol(j) < nlim)) continue;
              v4f* cij = reinterpret_cast<v4f*>(ci + jcol(j));
              if (OUTF32 == 2 && !part)
                *cij = *cij + acc[i][j];
              else
                *cij = acc[i][j];
            }
          }
        } else if constexpr (!CHK && NI == 4) {
          // Whole 128-byte lines, past the caches or not (stores_past_caches).  Of row l % 16 a lane has columns
          // 8 (l / 16) .. +7 of both 32-column halves (in natural order lanes l and l + 16 swap first, so that it has eight
          // consecutive columns there too, and the lane groups 16 (g % 2) + 8 (g / 2)).  us with 64-byte stores, whole
          // lines, and whole lines past the caches: wgrad of 64 experts of 2816 x 2048, 32768 tokens 375 / 378 / 324, 4096 tokens 211 / 211 / 159 (64-byte
          // stores past the caches took more than cached ones there); fprop of 64 such experts 233 / 236 / 229.
          const int g = el >> 4, h = (el >> 3) & 1;
          uint16_t* c0 = reinterpret_cast<uint16_t*>(d.c) + (crow - 8 * h) * d.ldc + ccol + 32 * h;
          if constexpr (!PERM) c0 += -4 * g + 16 * (g & 1) + 8 * (g >> 1);
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            v4i p[2], upper, lower;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const v4f& a = acc[i][2 * t];
              const v4f& b = acc[i][2 * t + 1];
              const uint32_t a0 = pack_bf16x2(a[0], a[1]), a1 = pack_bf16x2(a[2], a[3]);
              const uint32_t b0 = pack_bf16x2(b[0], b[1]), b1 = pack_bf16x2(b[2], b[3]);
              if constexpr (PERM) {
                p[t] = (v4i){(int)a0, (int)a1, (int)b0, (int)b1};
              } else {
                const auto lo = __builtin_amdgcn_permlane16_swap(a0, b0, false, false);
                const auto hi = __builtin_amdgcn_permlane16_swap(a1, b1, false, false);
                p[t] = (v4i){(int)lo[0], (int)hi[0], (int)lo[1], (int)hi[1]};
              }
            }
            join_halves(p[0], p[1], upper, lower);
            store_line(upper, reinterpret_cast<v4i*>(c0 + 16 * i * d.ldc), past);
            store_line(lower, reinterpret_cast<v4i*>(c0 + (16 * i + 8) * d.ldc), past);
          }
        } else if constexpr (PERM) {
          uint16_t* c0 = reinterpret_cast<uint16_t*>(d.c) + crow * d.ldc + ccol;
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            uint16_t* ci = c0 + 16 * i * d.ldc;
#pragma unroll
            for (int t = 0; t < NI / 2; ++t) {
              if (CHK && !(mrow + 16 * i < mlim && ncol + 32 * t < nlim)) continue;
              const v4f& a = acc[i][2 * t];
              const v4f& b = acc[i][2 * t + 1];
              *reinterpret_cast<uint4*>(ci + 32 * t) = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                                                   pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]));
            }
          }
        } else {
          uint16_t* c0 = reinterpret_cast<uint16_t*>(d.c) + crow * d.ldc + ccol;
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            uint16_t* ci = c0 + 16 * i * d.ldc;
#pragma unroll
            for (int j = 0; j < NI; ++j) {
              if (CHK && !(mrow + 16 * i < mlim && ncol + 16 * j < nlim)) continue;
              *reinterpret_cast<uint2*>(ci + 16 * j) =
                  make_uint2(pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3]));
            }
          }
        }
      };
      if (full) {
        write(std::false_type{});
      } else {
        write(std::true_type{});
      }
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
    }
    cu += G;
    if (cu >= U) break;  // (the loads issued after the last block are drained below)
    C = unit_at(cu);
    ckb = C.kb0;
  }
  // no direct-to-LDS load may still be writing when the workgroup's LDS is handed to the next one
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// One tile shape for all units.
template <int OP, int BM, int BN, int WGM, int WGN, int NSTAGE, int SBM, int FA, int FB, int OUTF32, int GM = kGroupNone>
__global__ __launch_bounds__(WGM* WGN * 64, (StageMinBlocks<BM, BN, WGM * WGN, NSTAGE>::value)) void gemm_tn_kernel(
    GemmDesc d, uint32_t tiles_m, uint32_t tiles_n, int nsplit, float* __restrict__ partial, GroupArgs<GM> grp) {
  constexpr int NW = WGM * WGN;
  constexpr bool GROUPED = GM != kGroupNone;
  constexpr int RING = ring_bytes<BM, BN, NSTAGE, SBM>();
  // (the table of a grouped product lies in the same array: a second __shared__ object makes the compiler
  // wait for every LDS-DMA load in flight before each LDS read)
  constexpr int TABLE = GM == kGroupContract ? kContractTableBytes : GROUPED ? kGroupTableBytes : 0;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[RING + TABLE];
  uint32_t* gunits = reinterpret_cast<uint32_t*>(smem + RING);
  int* gstarts = reinterpret_cast<int*>(gunits + (GM == kGroupContract ? kMaxEntries : kMaxExperts) + 1);
  uint32_t U = tiles_m * tiles_n * (uint32_t)nsplit;
  if constexpr (GROUPED) {
    const int lane = threadIdx.x & 63;
    if (threadIdx.x < 64) {
      if constexpr (GM == kGroupContract)
        group_table_blocks(grp.offsets, grp.experts, grp.tokens, grp.split, gstarts, gunits, lane);
      else
        group_table_rows(grp.offsets, grp.experts, grp.tokens, BM, tiles_n, gstarts, gunits, lane);
    }
    __syncthreads();
    // (a step of its own behind the barrier: in the branch above it the compiler took the whole tile loop's uniform
    // values into vector registers where no other step followed the barrier, and spilled 73 of them)
    if constexpr (GM == kGroupContract) {
      if (grp.split.sets > 0 && blockIdx.x == 0 && threadIdx.x < 64) list_split(gunits, grp.split_list, lane);
    }
    if constexpr (GM == kGroupContract)
      U *= __builtin_amdgcn_readfirstlane(gunits[kMaxEntries]);
    else
      U = __builtin_amdgcn_readfirstlane(gunits[grp.experts]);
    if constexpr (GM == kGroupContract && OUTF32 != 2) {
      // an expert without tokens has a zero gradient: its slice of C, spread over the workgroups
      for (int e = 0; e < grp.experts; ++e) {
        if (gstarts[e + 1] != gstarts[e]) continue;
        const int64_t chunks = d.N / (OUTF32 ? 4 : 8);
        for (int64_t i = (int64_t)blockIdx.x * (NW * 64) + threadIdx.x; i < d.M * chunks;
             i += (int64_t)gridDim.x * (NW * 64)) {
          const int64_t r = i / chunks, c = i - r * chunks;
          uint8_t* p = (uint8_t*)d.c + ((int64_t)e * d.M + r) * d.ldc * (OUTF32 ? 4 : 2) + c * 16;
          *reinterpret_cast<uint4*>(p) = make_uint4(0, 0, 0, 0);
        }
      }
    }
  }
  gemm_tn_units<OP, BM, BN, WGM, WGN, NSTAGE, SBM, FA, FB, OUTF32, GM, kPartAll>(d, tiles_m, tiles_n, nsplit, partial,
                                                                                 grp, smem, gunits, gstarts, U,
                                                                                 blockIdx.x);
}

// Grouped rows with 256 x 256 tiles and, for an expert's last rows where at most 128 are left, one 128 x 256 tile:
// a 256-row tile there would multiply more rows that do not exist than rows that do (a quarter of all rows with
// 512 tokens an expert; 32 experts, 32768 tokens, 2048 x 1408: 123 us with 256-row tiles alone, 113 us so).  A
// workgroup takes its tall units, then its short ones, counted on over both lists, so that the short units fill
// the tall list's last round.
template <int OP, int SBM, int FA, int FB, int OUTF32, int GM>
__global__ __launch_bounds__(512, 2) void gemm_tn_grouped_kernel(GemmDesc d, uint32_t tiles_n, GroupArgs<GM> grp) {
  constexpr int RING = ring_bytes<256, 256, 2, SBM>();
  static_assert(ring_bytes<128, 256, 2, SBM>() <= RING, "one array serves both tiles");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[RING + kGroupTableBytes + kGroupTableBytes / 2];
  uint32_t* tall = reinterpret_cast<uint32_t*>(smem + RING);
  uint32_t* rest = tall + kMaxExperts + 1;
  int* starts = reinterpret_cast<int*>(rest + kMaxExperts + 1);
  if (threadIdx.x < 64)
    group_table_two(grp.offsets, grp.experts, grp.tokens, tiles_n, starts, tall, rest, threadIdx.x & 63);
  __syncthreads();
  const uint32_t U1 = __builtin_amdgcn_readfirstlane(tall[grp.experts]);
  const uint32_t U2 = __builtin_amdgcn_readfirstlane(rest[grp.experts]);
  const uint32_t G = gridDim.x;
  gemm_tn_units<OP, 256, 256, 2, 4, 2, SBM, FA, FB, OUTF32, GM, kPartTall>(d, 0, tiles_n, 1, nullptr, grp, smem, tall,
                                                                           starts, U1, blockIdx.x);
  __syncthreads();  // (the ring is filled again)
  const uint32_t past = blockIdx.x < U1 ? (U1 - 1 - blockIdx.x) / G * G + G + blockIdx.x : blockIdx.x;
  gemm_tn_units<OP, 128, 256, 2, 4, 2, SBM, FA, FB, OUTF32, GM, kPartRest>(d, 0, tiles_n, 1, nullptr, grp, smem, rest,
                                                                           starts, U2, past - U1);
}

}  // namespace fp8bq
