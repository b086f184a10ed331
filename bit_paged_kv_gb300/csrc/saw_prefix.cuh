// saw_prefix.cuh -- how the shared-prefix pass is cut into work, computed the
// same way by the kernel that writes its partial results and by the decode
// kernel that reads them.
//
// A group's rows are (sequence, q-head of a kv-head) pairs.  A unit is one
// kv-head and one block of seqs_per_block(G) neighbouring sequences of a group
// (at most kPrefixRows rows, one tensor-core tile).  Its keys are tiles of
// kPrefixKeys tokens, T of them; units of a group follow one another kv-head
// by kv-head, groups in order, and all tiles form one line that is cut into
// equal pieces of `chunk` tiles, one per CTA.  Unit u meeting CTA c leaves a
// partial result in slot u + c: walking along the line, u or c grows at every
// cut, so slots never collide, and a unit's slots are consecutive.
#pragma once

#include "saw_device.cuh"
#include "saw_int4.h"

namespace saw {

__host__ __device__ constexpr int prefix_seqs_per_block(int group) { return kPrefixRows / group; }

// One group (unit0, tile0: units and tiles of the groups before).
struct PrefixGroup {
  int first, end;      // sequences
  int tokens;          // whole pages of the prefix, in tokens
  int tiles;           // key tiles of a unit
  int blocks;          // blocks of sequences (0 with nothing shared)
  uint32_t unit0, tile0;
};

__device__ __forceinline__ uint32_t warp_scan_u32(uint32_t v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Whole warp: the first group for which pick(group) holds (zero sizes if none
// does), and the tiles of all groups.  A group whose entries are inconsistent
// -- out of range, descending, or reaching back over an earlier one, so that
// the others stay disjoint and their units within the workspace -- shares
// nothing; *bad is set in some lane.
// PLACE false: only the group itself, without unit0, tile0 and *total.
template <bool PLACE, typename Pick>
__device__ __forceinline__ PrefixGroup prefix_scan(const PrefixSide& s, int page_size, int group,
                                                   int hkv, int num_seqs, int lane, Pick pick,
                                                   bool* bad, uint32_t* total) {
  PrefixGroup found{0, 0, 0, 0, 0, 0, 0};
  uint32_t units = 0, tiles = 0;
  int top = 0;  // end of the groups so far
  bool have = false;
  const int per = prefix_seqs_per_block(group);
  for (int g0 = 0; g0 < s.num_groups; g0 += 32) {
    const int g = g0 + lane;
    PrefixGroup r{0, 0, 0, 0, 0, 0, 0};
    int lo = 0, hi = 0, pre = 0;
    if (g < s.num_groups) {
      lo = s.cu_groups[g];
      hi = s.cu_groups[g + 1];
      pre = s.prefix_lens[g];
    }
    int reach = hi;  // furthest end up to this group
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, reach, d);
      if (lane >= d) reach = max(reach, o);
    }
    int before = __shfl_up_sync(0xFFFFFFFFu, reach, 1);
    before = lane == 0 ? top : max(top, before);
    if (lo < before || hi < lo || hi > num_seqs || pre < 0 || pre > s.max_prefix_len) {
      if (g < s.num_groups) *bad = true;
    } else {
      r.first = lo;
      r.end = hi;
      r.tokens = pre / page_size * page_size;
      r.tiles = (r.tokens + kPrefixKeys - 1) / kPrefixKeys;
      r.blocks = r.tiles > 0 ? (hi - lo + per - 1) / per : 0;
    }
    const uint32_t u = uint32_t(r.blocks) * hkv, t = u * r.tiles;
    uint32_t ui = 0, ti = 0;
    if constexpr (PLACE) {
      ui = warp_scan_u32(u, lane);
      ti = warp_scan_u32(t, lane);
      r.unit0 = units + ui - u;
      r.tile0 = tiles + ti - t;
    }
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, pick(r, t));
    if (hit && !have) {
      const int at = __ffs(hit) - 1;
      found.first = __shfl_sync(0xFFFFFFFFu, r.first, at);
      found.end = __shfl_sync(0xFFFFFFFFu, r.end, at);
      found.tokens = __shfl_sync(0xFFFFFFFFu, r.tokens, at);
      found.tiles = __shfl_sync(0xFFFFFFFFu, r.tiles, at);
      found.blocks = __shfl_sync(0xFFFFFFFFu, r.blocks, at);
      if constexpr (PLACE) {
        found.unit0 = __shfl_sync(0xFFFFFFFFu, r.unit0, at);
        found.tile0 = __shfl_sync(0xFFFFFFFFu, r.tile0, at);
      }
      have = true;
    }
    if constexpr (PLACE) {
      units += __shfl_sync(0xFFFFFFFFu, ui, 31);
      tiles += __shfl_sync(0xFFFFFFFFu, ti, 31);
    }
    top = max(top, __shfl_sync(0xFFFFFFFFu, reach, 31));
  }
  *total = tiles;
  return found;
}

// Tiles per CTA when `total` tiles are shared by `ctas` CTAs.
__device__ __forceinline__ uint32_t prefix_chunk(uint32_t total, int ctas) {
  return (total + uint32_t(ctas) - 1) / uint32_t(ctas);
}

// Partial results: slot s holds numerators as [32 groups of 4 dims][128
// rows][4] binary32 (rows lie side by side, so both the writing threads, one
// per row, and the merge, a few rows, touch whole sectors) and (m, l) as
// [128 rows].
__device__ __forceinline__ int64_t prefix_part_index(int64_t slot) {
  return slot * (32 * kPrefixRows);  // in float4
}

}  // namespace saw
