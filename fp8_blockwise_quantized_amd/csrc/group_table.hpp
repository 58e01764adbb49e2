// Per-expert tables of the products grouped by expert (device side).
//
// offsets[0..E] (int64, on the device) hold where each expert's tokens begin; the tokens of expert e
// are offsets[e] .. offsets[e+1]-1.  The values come from a router on the device, so a kernel makes them
// safe itself: each is clamped to [0, T] (the padded rows where the contraction runs over the tokens) and to at
// least the one before it, whatever the buffer holds.
// One wave builds the tables in LDS: lane l owns experts 8l .. 8l+7 and two wave scans (a maximum for
// the clamped offsets, a sum for the counts) join the lanes; about a microsecond, most of it the load.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "plan.hpp"

namespace fp8bq {

constexpr int kMaxExperts = 512;
constexpr int kExpertsPerLane = kMaxExperts / 64;
constexpr int kGroupTableBytes = (2 * (kMaxExperts + 1) * 4 + 15) / 16 * 16;  // unit counts and starts
// Contraction over the tokens: a list of (expert, chunk) entries, its length, and starts.
constexpr int kMaxEntries = kMaxExperts + kMaxSets;
constexpr int kContractTableBytes = ((kMaxEntries + 1 + kMaxExperts + 1) * 4 + 15) / 16 * 16;

// Inclusive wave scans by DPP: four shifts within the rows of 16 lanes, then each row's last lane into the
// next row and lane 31 into the upper half.  Lanes without a source take 0, the identity of both operations.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t scan_source(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_scan_add(uint32_t v) {
  v += scan_source<0x111, 0xF>(v);
  v += scan_source<0x112, 0xF>(v);
  v += scan_source<0x114, 0xF>(v);
  v += scan_source<0x118, 0xF>(v);
  v += scan_source<0x142, 0xA>(v);
  v += scan_source<0x143, 0xC>(v);
  return v;
}
__device__ __forceinline__ int wave_scan_max(int v) {  // v >= 0
  const auto up = [&](uint32_t o) { v = (int)o > v ? (int)o : v; };
  up(scan_source<0x111, 0xF>(v));
  up(scan_source<0x112, 0xF>(v));
  up(scan_source<0x114, 0xF>(v));
  up(scan_source<0x118, 0xF>(v));
  up(scan_source<0x142, 0xA>(v));
  up(scan_source<0x143, 0xC>(v));
  return v;
}

// The lane's safe offsets o[i] = offset of expert 8*lane + i, i = 0 .. 8 (T < 2^31); experts past E
// are empty.
__device__ __forceinline__ void group_offsets(const int64_t* offsets, int E, int64_t T, int lane,
                                              int (&o)[kExpertsPerLane + 1]) {
#pragma unroll
  for (int i = 0; i <= kExpertsPerLane; ++i) {
    const int j = kExpertsPerLane * lane + i;
    const int64_t v = offsets[j < E ? j : E];
    o[i] = (int)(v < 0 ? 0 : (v > T ? T : v));
  }
#pragma unroll
  for (int i = 1; i <= kExpertsPerLane; ++i) o[i] = o[i] > o[i - 1] ? o[i] : o[i - 1];
  const int upto = wave_scan_max(o[kExpertsPerLane]);
  int before = __shfl_up(upto, 1);
  before = lane == 0 ? 0 : before;
#pragma unroll
  for (int i = 0; i <= kExpertsPerLane; ++i) o[i] = o[i] > before ? o[i] : before;
}

// Exclusive sums of the lane's counts c[i] over all experts, written to pre[0 .. E] (pre[E] = total).
__device__ __forceinline__ void group_sums(const uint32_t (&c)[kExpertsPerLane], int E, int lane, uint32_t* pre) {
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < kExpertsPerLane; ++i) mine += c[i];
  uint32_t at = wave_scan_add(mine) - mine;
#pragma unroll
  for (int i = 0; i < kExpertsPerLane; ++i) {
    const int j = kExpertsPerLane * lane + i;
    if (j <= E) pre[j] = at;
    at += c[i];
  }
  if (lane == 63 && E == kMaxExperts) pre[E] = at;
}

// starts[e] = first token of expert e, units[e] = tiles of the experts before e, of tile_rows tokens by
// tiles_n columns of tiles.
__device__ __forceinline__ void group_table_rows(const int64_t* offsets, int E, int64_t T, int tile_rows,
                                                 uint32_t tiles_n, int* starts, uint32_t* units, int lane) {
  int o[kExpertsPerLane + 1];
  group_offsets(offsets, E, T, lane, o);
  uint32_t c[kExpertsPerLane];
#pragma unroll
  for (int i = 0; i < kExpertsPerLane; ++i) {
    const int j = kExpertsPerLane * lane + i;
    if (j <= E) starts[j] = o[i];
    c[i] = (uint32_t)((o[i + 1] - o[i] + tile_rows - 1) / tile_rows) * tiles_n;
  }
  if (lane == 63 && E == kMaxExperts) starts[E] = o[kExpertsPerLane];
  group_sums(c, E, lane, units);
}

// Row tiles of an expert's n tokens when its last tile may be short: tall tiles of 256 rows, and one of 128 where
// 1 to 128 rows are left after them.
constexpr int kTall = 256, kShort = 128;
__device__ __forceinline__ int tall_tiles(int n) { return n / kTall + (n % kTall > kShort ? 1 : 0); }
__device__ __forceinline__ int short_tiles(int n) { return n % kTall > 0 && n % kTall <= kShort ? 1 : 0; }

// As group_table_rows for both lists.
__device__ __forceinline__ void group_table_two(const int64_t* offsets, int E, int64_t T, uint32_t tiles_n,
                                                int* starts, uint32_t* tall, uint32_t* rest, int lane) {
  int o[kExpertsPerLane + 1];
  group_offsets(offsets, E, T, lane, o);
  uint32_t a[kExpertsPerLane], b[kExpertsPerLane];
#pragma unroll
  for (int i = 0; i < kExpertsPerLane; ++i) {
    const int j = kExpertsPerLane * lane + i;
    if (j <= E) starts[j] = o[i];
    a[i] = (uint32_t)tall_tiles(o[i + 1] - o[i]) * tiles_n;
    b[i] = (uint32_t)short_tiles(o[i + 1] - o[i]) * tiles_n;
  }
  if (lane == 63 && E == kMaxExperts) starts[E] = o[kExpertsPerLane];
  group_sums(a, E, lane, tall);
  group_sums(b, E, lane, rest);
}

// The lane's counts of 128-token blocks, for tokens padded to whole blocks per expert.
__device__ __forceinline__ void group_block_counts(const int (&o)[kExpertsPerLane + 1],
                                                   uint32_t (&c)[kExpertsPerLane]) {
#pragma unroll
  for (int i = 0; i < kExpertsPerLane; ++i) c[i] = (uint32_t)(o[i + 1] - o[i] + 127) / 128;
}

// The longest contraction, in blocks, that a product over the tokens gives one work unit: longer experts are
// split into chunks of about equal length.  Each lane prices one length with the counts at hand (chunk_time)
// and the cheapest is taken, the longest of equals; the last lane's splits nothing.
__device__ __forceinline__ float group_chunk(const int* starts, int E, int longest, const GroupSplit& split, int lane) {
  const float s = chunk_candidate(lane);
  const float inv = 1.0f / s;
  ChunkSums sums(longest, s);
  for (int e = 0; e < E; ++e) sums.add(starts[e + 1] - starts[e], s, inv);
  uint32_t t = __float_as_uint(chunk_time(sums, split));  // (not negative: the bits are ordered)
  const uint32_t mine = t;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)t, d);
    t = o < t ? o : t;
  }
  const int best = 63 - __clzll((long long)__ballot(mine == t));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(s), best));
}

// One entry of the list: chunk `chunk` of the `chunks` (1: whole) of expert `expert`, whose partial sums begin at set
// `set` of the workspace.
struct GroupEntry {
  int expert, chunks, chunk, set;
};
__device__ __forceinline__ uint32_t pack_entry(int expert, int chunks, int chunk, int set) {
  static_assert(kMaxExperts <= 512 && kMaxSets <= 64, "fields of an entry");
  return (uint32_t)expert | (uint32_t)(chunks - 1) << 9 | (uint32_t)chunk << 15 | (uint32_t)set << 21;
}
__device__ __forceinline__ GroupEntry entry_of(uint32_t v) {
  return GroupEntry{(int)(v & 511), (int)(v >> 9 & 63) + 1, (int)(v >> 15 & 63), (int)(v >> 21 & 63)};
}

// starts[e] = first 128-token block of expert e in the padded layout, at most padded / 128; order[0 .. n) = the chunks
// (GroupEntry) of the experts that have a block, by the bit length of the chunk's block count, most first (in
// expert order within one length); order[kMaxEntries] = n.  Products that contract over the blocks take the long
// chunks first: a last round of long units on few workgroups is what costs most (64 experts with shares from
// 1/5 to 1/300: 614 us in expert order, contiguous per XCD, and 402 us so).
__device__ __forceinline__ void group_table_blocks(const int64_t* offsets, int E, int64_t padded,
                                                   const GroupSplit& split, int* starts, uint32_t* order, int lane) {
  int o[kExpertsPerLane + 1];
  group_offsets(offsets, E, padded, lane, o);
  uint32_t c[kExpertsPerLane];
  group_block_counts(o, c);
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < kExpertsPerLane; ++i) mine += c[i];
  uint32_t at = wave_scan_add(mine) - mine;
  const uint32_t cap = (uint32_t)(padded / 128);
#pragma unroll
  for (int i = 0; i < kExpertsPerLane; ++i) {
    const int j = kExpertsPerLane * lane + i;
    const uint32_t b0 = at < cap ? at : cap;
    at += c[i];
    const uint32_t b1 = at < cap ? at : cap;
    if (j <= E) starts[j] = (int)b0;
    c[i] = b1 - b0;
  }
  if (lane == 63 && E == kMaxExperts) starts[E] = (int)(at < cap ? at : cap);
  int chunks[kExpertsPerLane];
  uint32_t sets = 0;  // partial sums of my experts
#pragma unroll
  for (int i = 0; i < kExpertsPerLane; ++i) chunks[i] = c[i] ? 1 : 0;
  if (split.sets > 0) {
    int longest = 0, used = 0, blocks = 0;
#pragma unroll
    for (int i = 0; i < kExpertsPerLane; ++i) {
      longest = (int)c[i] > longest ? (int)c[i] : longest;
      used += chunks[i];
      blocks += (int)c[i];
    }
    longest = __builtin_amdgcn_readlane(wave_scan_max(longest), 63);
    const uint32_t all = (uint32_t)__builtin_amdgcn_readlane((int)wave_scan_add((uint32_t)(used + blocks)), 63);
    // While the longest is well below a workgroup's share of the blocks, whole experts balance: nothing to choose
    // (the choice takes some 50 instructions an expert).
    if ((float)longest > 0.4f * (float)all * split.tiles / split.slots) {
      const float s = group_chunk(starts, E, longest, split, lane), inv = 1.0f / s;
#pragma unroll
      for (int i = 0; i < kExpertsPerLane; ++i) {
        chunks[i] = c[i] ? chunks_of((int)c[i], s, inv) : 0;
        sets += chunks[i] > 1 ? (uint32_t)chunks[i] : 0u;
      }
    }
  }
  uint32_t set = wave_scan_add(sets) - sets;
  uint32_t first[kExpertsPerLane];
  uint32_t lengths = 0;  // bit l: an expert of mine has chunks of l + 1 bits
#pragma unroll
  for (int i = 0; i < kExpertsPerLane; ++i) {
    first[i] = set;
    if (chunks[i] > 1) {
      set += (uint32_t)chunks[i];
      c[i] /= (uint32_t)chunks[i];
    }
    if (c[i]) lengths |= 1u << (31 - __clz((int)c[i]));
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) lengths |= (uint32_t)__shfl_xor((int)lengths, d);
  uint32_t n = 0;
  while (lengths) {  // (the same in every lane)
    const int l = 31 - __clz((int)lengths);
    lengths &= ~(1u << l);
    uint32_t have = 0;
#pragma unroll
    for (int i = 0; i < kExpertsPerLane; ++i) have += c[i] && 31 - __clz((int)c[i]) == l ? (uint32_t)chunks[i] : 0u;
    const uint32_t upto = wave_scan_add(have);
    uint32_t p = n + upto - have;
#pragma unroll
    for (int i = 0; i < kExpertsPerLane; ++i)
      if (c[i] && 31 - __clz((int)c[i]) == l)
        for (int k = 0; k < chunks[i]; ++k)
          order[p++] = pack_entry(kExpertsPerLane * lane + i, chunks[i], k, chunks[i] > 1 ? (int)first[i] : 0);
    n += (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
  }
  if (lane == 0) order[kMaxEntries] = n;
}

// list[0] = experts that are split, list[1 ..] their first entries.
__device__ __forceinline__ void list_split(const uint32_t* order, uint32_t* list, int lane) {
  static_assert((1 + kMaxSets / 2) * 4 <= (int)kSplitListBytes, "a split expert takes two sets at least");
  const int entries = (int)order[kMaxEntries];
  uint32_t n = 0;
  for (int b = 0; b < entries; b += 64) {
    const uint32_t v = b + lane < entries ? order[b + lane] : 0;
    const GroupEntry e = entry_of(v);
    const bool take = e.chunks > 1 && e.chunk == 0;
    const uint64_t m = __ballot(take);
    if (take) list[1 + n + __popcll(m & (((uint64_t)1 << lane) - 1))] = v;
    n += (uint32_t)__popcll(m);
  }
  if (lane == 0) list[0] = n;
}

// The expert of unit u: pre[e] <= u < pre[e+1], by a count of the experts that end at or before u (all
// 64 lanes take part; the result is the same in each).
__device__ __forceinline__ int group_find(const uint32_t* pre, int E, uint32_t u, int lane) {
  int e = 0;
  for (int b = 0; b < E; b += 64) {
    const int j = b + lane;
    const bool le = j < E && pre[j + 1] <= u;
    e += __popcll(__ballot(le));
  }
  return __builtin_amdgcn_readfirstlane(e);
}

}  // namespace fp8bq
