// saw_prefix.cuh -- how the shared-prefix pass is cut into work.
//
// A group's rows are (sequence, q-head of a kv-head) pairs.  A unit is one
// kv-head and one block of seqs_per_block(G) neighbouring sequences of a group
// (at most kPrefixRows rows, one tensor-core tile).  Its keys are T tiles of
// kPrefixKeys tokens, cut into n = ceil(T / chunk) equal parts; part j of unit
// u (units of a group kv-head by kv-head) is number part0 + u n + j, and parts
// go round the CTAs.  `chunk` is the one for which the fullest CTA has least to
// do, a part costing its tiles and kPartCost more: CTAs that took equal pieces
// of one line of tiles had two units to start more often than one.  The prefix
// kernel leaves chunk and every group's part0 for the decode kernel's merge.
#pragma once

#include "saw_device.cuh"
#include "saw_int4.h"

namespace saw {

__host__ __device__ constexpr int prefix_seqs_per_block(int group) { return kPrefixRows / group; }

// One group.
struct PrefixGroup {
  int first, end;      // sequences
  int tokens;          // whole pages of the prefix, in tokens
  int tiles;           // key tiles of a unit
  int blocks;          // blocks of sequences (0 with nothing shared)
  int index;
};

constexpr int kPartCost = 5;  // starting and ending a part, in tiles

__device__ __forceinline__ uint32_t warp_scan_u32(uint32_t v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Whole warp: group g0 + lane (nothing shared beyond the last).  *top, the
// furthest end of the groups before g0, moves on.  A group whose entries are
// inconsistent -- out of range, descending, or reaching back over an earlier
// one, so that the others stay disjoint and their units within the workspace --
// shares nothing; *bad is set in its lane.  The ends of groups out of range or
// descending do not count for the later ones.
__device__ __forceinline__ PrefixGroup prefix_load(const PrefixSide& s, int g0, int page_size, int group,
                                                   int num_seqs, int lane, int* top, bool* bad,
                                                   bool past_l1 = false) {
  const int g = g0 + lane;
  PrefixGroup r{0, 0, 0, 0, 0, g};
  int lo = 0, hi = 0, pre = 0;
  if (g < s.num_groups) {
    auto load = [&](const int32_t* at) { return past_l1 ? __ldcg(at) : *at; };
    lo = load(s.cu_groups + g);
    hi = load(s.cu_groups + g + 1);
    pre = load(s.prefix_lens + g);
  }
  int reach = lo >= 0 && hi >= lo && hi <= num_seqs ? hi : 0;  // furthest end up to this group
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, reach, d);
    if (lane >= d) reach = max(reach, o);
  }
  int before = __shfl_up_sync(0xFFFFFFFFu, reach, 1);
  before = lane == 0 ? *top : max(*top, before);
  if (g < s.num_groups) {
    if (lo < before || hi < lo || hi > num_seqs || pre < 0 || pre > s.max_prefix_len) {
      *bad = true;
    } else {
      const int per = prefix_seqs_per_block(group);
      r.first = lo;
      r.end = hi;
      r.tokens = pre & -page_size;  // (page sizes are powers of two)
      r.tiles = (r.tokens + kPrefixKeys - 1) / kPrefixKeys;
      r.blocks = r.tiles > 0 ? (hi - lo + per - 1) / per : 0;
    }
  }
  *top = max(*top, __shfl_sync(0xFFFFFFFFu, reach, 31));
  return r;
}

__device__ __forceinline__ PrefixGroup prefix_from(const PrefixGroup& r, int lane) {
  PrefixGroup o;
  o.first = __shfl_sync(0xFFFFFFFFu, r.first, lane);
  o.end = __shfl_sync(0xFFFFFFFFu, r.end, lane);
  o.tokens = __shfl_sync(0xFFFFFFFFu, r.tokens, lane);
  o.tiles = __shfl_sync(0xFFFFFFFFu, r.tiles, lane);
  o.blocks = __shfl_sync(0xFFFFFFFFu, r.blocks, lane);
  o.index = __shfl_sync(0xFFFFFFFFu, r.index, lane);
  return o;
}

// Whole warp: the group that holds sequence `seq` (nothing shared if none does).
// all: every group is looked at, for *bad.  past_l1: the entries are taken from
// L2, for a caller ahead of its dependency wait.
__device__ __forceinline__ PrefixGroup prefix_of_seq(const PrefixSide& s, int seq, int page_size, int group,
                                                     int num_seqs, int lane, bool all, bool past_l1, bool* bad) {
  int top = 0;
  PrefixGroup mine{0, 0, 0, 0, 0, 0};
  for (int g0 = 0; g0 < s.num_groups; g0 += 32) {
    const PrefixGroup r = prefix_load(s, g0, page_size, group, num_seqs, lane, &top, bad, past_l1);
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, r.first <= seq && seq < r.end);
    if (hit) mine = prefix_from(r, __ffs(hit) - 1);
    if (hit && !all) break;
  }
  return mine;
}

// Partial results: slot s holds numerators as [32 groups of 4 dims][128
// rows][4] binary32 (rows lie side by side, so both the writing threads, one
// per row, and the merge, a few rows, touch whole sectors) and (m, l) as
// [128 rows].
__device__ __forceinline__ int64_t prefix_part_index(int64_t slot) {
  return slot * (32 * kPrefixRows);  // in float4
}

}  // namespace saw
