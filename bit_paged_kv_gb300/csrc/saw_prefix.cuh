// saw_prefix.cuh -- how the shared-prefix pass is cut into work, computed the
// same way by the kernel that writes its partial results and by the decode
// kernel that reads them.
//
// A group's rows are (sequence, q-head of a kv-head) pairs.  A unit is one
// kv-head and one block of seqs_per_block(G) neighbouring sequences of a group
// (at most kPrefixRows rows, two 128-row tiles).  Its keys are tiles of
// kPrefixKeys tokens, T of them; units of a group follow one another kv-head
// by kv-head, groups in order, and all tiles form one line that is cut into
// equal pieces of `chunk` tiles, one per CTA.  Unit u meeting CTA c leaves a
// partial result in slot u + c: walking along the line, u or c grows at every
// cut, so slots never collide, and a unit's slots are consecutive.
#pragma once

#include "saw_device.cuh"
#include "saw_int4.h"

namespace saw {

constexpr int kPrefixRows = 256;   // rows of a unit: two 128-row tiles
constexpr int kPrefixKeys = 128;   // keys per tile

__host__ __device__ constexpr int prefix_seqs_per_block(int group) { return kPrefixRows / group; }

// One group as a lane sees it (unit0, tile0: units and tiles of the groups before).
struct PrefixGroup {
  int first, end;      // sequences
  int tokens;          // whole pages of the prefix, in tokens
  int tiles;           // key tiles of a unit
  int blocks;          // blocks of sequences
  uint32_t unit0, tile0;
};

// Group g's sizes; an inconsistent group has no prefix (and *bad set).
__device__ __forceinline__ PrefixGroup prefix_group(const PrefixSide& s, int g, int page_size,
                                                    int group, int num_seqs, bool* bad) {
  PrefixGroup r{0, 0, 0, 0, 0, 0, 0};
  if (g >= s.num_groups) return r;
  const int lo = s.cu_groups[g], hi = s.cu_groups[g + 1], pre = s.prefix_lens[g];
  if (lo < 0 || hi < lo || hi > num_seqs || pre < 0 || pre > s.max_prefix_len) {
    *bad = true;
    return r;
  }
  r.first = lo;
  r.end = hi;
  r.tokens = pre / page_size * page_size;
  r.tiles = (r.tokens + kPrefixKeys - 1) / kPrefixKeys;
  const int per = prefix_seqs_per_block(group);
  r.blocks = r.tiles > 0 ? (hi - lo + per - 1) / per : 0;
  return r;
}

__device__ __forceinline__ uint32_t warp_scan_u32(uint32_t v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Whole warp: the group that holds sequence `seq` (zero sizes if none does),
// with unit0 and tile0, and the tiles of all groups in *total.  The lane that
// meets an inconsistent group reports it.
__device__ __forceinline__ PrefixGroup prefix_find_seq(const PrefixSide& s, int seq, int page_size,
                                                       int group, int hkv, int num_seqs, int lane,
                                                       int32_t* status, uint32_t* total) {
  PrefixGroup found{0, 0, 0, 0, 0, 0, 0};
  uint32_t units = 0, tiles = 0;
  bool have = false, bad = false;
  for (int g0 = 0; g0 < s.num_groups; g0 += 32) {
    PrefixGroup r = prefix_group(s, g0 + lane, page_size, group, num_seqs, &bad);
    const uint32_t u = uint32_t(r.blocks) * hkv, t = u * r.tiles;
    const uint32_t ui = warp_scan_u32(u, lane), ti = warp_scan_u32(t, lane);
    r.unit0 = units + ui - u;
    r.tile0 = tiles + ti - t;
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, r.first <= seq && seq < r.end);
    if (hit && !have) {
      const int at = __ffs(hit) - 1;
      found.first = __shfl_sync(0xFFFFFFFFu, r.first, at);
      found.end = __shfl_sync(0xFFFFFFFFu, r.end, at);
      found.tokens = __shfl_sync(0xFFFFFFFFu, r.tokens, at);
      found.tiles = __shfl_sync(0xFFFFFFFFu, r.tiles, at);
      found.blocks = __shfl_sync(0xFFFFFFFFu, r.blocks, at);
      found.unit0 = __shfl_sync(0xFFFFFFFFu, r.unit0, at);
      found.tile0 = __shfl_sync(0xFFFFFFFFu, r.tile0, at);
      have = true;
    }
    units += __shfl_sync(0xFFFFFFFFu, ui, 31);
    tiles += __shfl_sync(0xFFFFFFFFu, ti, 31);
  }
  if (bad && seq == 0) report(status, SAW_ERR_DEVICE_INDEX);
  *total = tiles;
  return found;
}

// Tiles per CTA when `total` tiles are shared by `ctas` CTAs.
__device__ __forceinline__ uint32_t prefix_chunk(uint32_t total, int ctas) {
  return (total + uint32_t(ctas) - 1) / uint32_t(ctas);
}

// Partial results: slot s, row tile q, holds numerators as
// [32 groups of 4 dims][128 rows][4] binary32 (the rows of a tile lie side by
// side, so both the writing threads, one per row, and the merge, a few rows,
// touch whole sectors) and (m, l) as [128 rows].
__device__ __forceinline__ int64_t prefix_part_index(int64_t slot, int tile) {
  return (slot * 2 + tile) * (32 * 128);  // in float4
}

}  // namespace saw
