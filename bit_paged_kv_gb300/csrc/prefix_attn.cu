// prefix_attn.cu -- the shared-prefix pass of saw_prefix_decode_int4: every
// (sequence, q-head) row of a group against the group's shared INT4 pages, on
// the 5th-generation tensor cores (tcgen05; accumulators in tensor memory).
// It writes unnormalised partial results (m, l, sum p v) that the decode
// kernel's merge takes up (saw_prefix.cuh has the split of the work).
//
// A decode step has one query per sequence, so over its own pages it is bound
// by HBM.  Over shared pages all rows of the group read the same keys: 4 D
// flops per (row, key) against 136 bytes per key, which with 256 rows is far
// on the tensor cores' side.
//
// Mathematics: the codes n enter S = q' n^T as they are (binary16 subnormals,
// exact), q' -- the rotated q times a power of two -- as binary16 hi + lo
// parts, so a score is t = s_k (q'.n) + z_k sum(q') to about 2^-22 of its
// terms, as in the decode.  V^ = n s_V + z_V is dequantized and rounded once
// to binary16 (no coarser than the 16-bit rows the cache was made from), p
// too: O += P V^ in binary32, where sum(p s n) + sum(p z) would cancel.
// Softmax in base 2 in binary32 with a running reference m that moves (and
// rescales O and l) only when a row's maximum has outgrown it by more than
// 2^8: p <= 2^8 stays far inside binary16, and the merge's normalisation makes
// the choice of m invisible.
//
// Twelve warps, specialised:
//   0-3    softmax: thread r owns row r (tensor-memory lane r) and its 128
//          scores in registers; p goes back over the scores' columns as the A
//          operand of P V
//   4-7    V expanders: one key per thread; 8-9: K expanders, two keys each
//   10     producer: bulk copies of codes and metadata, one lane each
//   11     MMA: one elected lane issues the products of tile i + 1's scores
//          before tile i's P V, so that the softmax of tile i runs behind them
// The 512 tensor-memory columns hold two score tiles (the second one makes the
// overlap), O, and q' hi and lo: the score products read only K from shared
// memory.  Operands there are unswizzled 8-row x 16-byte core matrices, two
// tiles each of K and V.  An expander writes each 8 dims in the order 0 4 1 5
// 2 6 3 7, the order in which masking a word of codes yields pairs; q' is
// stored in that order and the output columns are put back when written.
// Every wait is bounded to about a second.
#include <type_traits>

#include "saw_device.cuh"
#include "saw_int4.h"
#include "saw_prefix.cuh"
#include "saw_quant_row.cuh"
#include "saw_tcgen05.cuh"

namespace saw {
namespace {

constexpr int kThreads = 384;
constexpr int kSoftWarps = 4;
constexpr int kWarpV = 4, kWarpK = 8, kWarpProd = 10, kWarpMma = 11;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kKeys = kPrefixKeys;
static_assert(kPrefixRows == 128 && kKeys == 128, "one row per softmax thread, one key per V expander thread");

constexpr int kOpBytes = 128 * 128 * 2;            // one operand tile
constexpr int kRawV = kKeys * 64, kRawKM = 2 * kKeys * 64, kRawVM = kRawKM + kKeys * 4;
constexpr int kRawBytes = kRawVM + kKeys * 4;      // 17408
constexpr int kRawStages = 4;
constexpr int kMetas = 4;                          // tiles of (s_k, z_k) for the softmax
constexpr int kMetaBytes = kKeys * 8 + 16;         // s[128], z[128], valid 16-key slices
constexpr int kOffK = 0, kOffV = kOffK + 2 * kOpBytes;
constexpr int kOffRaw = kOffV + 2 * kOpBytes;
constexpr int kOffMeta = kOffRaw + kRawStages * kRawBytes;
constexpr int kOffOk = kOffMeta + kMetas * kMetaBytes;  // valid 16-key slices of the raw stages
constexpr int kOffBar = kOffOk + 4 * kRawStages;
enum { kRawFull = 0, kRawEmpty = kRawFull + kRawStages, kKFull = kRawEmpty + kRawStages, kKEmpty = kKFull + 2,
       kVFull = kKEmpty + 2, kPvDone = kVFull + 2, kMetaFull = kPvDone + 2, kSFull = kMetaFull + kMetas,
       kPFull = kSFull + 2, kQFull = kPFull + 2, kMmaDone, kBars };
constexpr int kOffTmem = kOffBar + kBars * 8;
constexpr int kSmem = kOffTmem + 16;
static_assert(kOffBar % 8 == 0 && kOffMeta % 16 == 0 && kSmem <= 227 * 1024, "shared memory");
constexpr uint32_t kColO = 256, kColQh = 384, kColQl = 448;

// ------------------------------------------------------------ PTX pieces

__device__ __forceinline__ void umma_ts_elect(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc))
      : "memory");
}
__device__ __forceinline__ void commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void arrive_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
// 32 tensor-memory columns of this thread's lane, without waiting
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
        "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// keeps uses of loaded registers behind the wait above
__device__ __forceinline__ void pin32(float* v) {
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                 "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]),
                 "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]),
                 "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]),
                 "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A wait of one warp; after a failure every later wait returns at once.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, bool& failed) {
  if (failed) return false;
  failed = !__all_sync(kAll, mbar_wait_bounded(bar, parity));
  return !failed;
}

// ------------------------------------------------------------ work list

struct Segment {
  int kvh;
  int leader;        // the group's first sequence, whose table row is read
  int seq0, rows;    // first sequence of the block; its (sequence, head) rows (at most 128)
  int tile, tiles;   // key tiles of the prefix to do
  int tokens;        // tokens of the whole prefix
  int64_t slot;
};

// Walks this CTA's tiles segment by segment; every warp walks for itself.
struct Walk {
  PrefixGroup g;
  uint32_t at, end;
  bool have;
};

__device__ __forceinline__ uint32_t group_tiles(const PrefixGroup& g, int hkv) {
  return uint32_t(g.blocks) * hkv * g.tiles;
}

// Whole warp: the group whose tiles hold `at`, and the tiles of all groups.
__device__ __forceinline__ PrefixGroup find_tile(const PrefixParams& p, uint32_t at, int lane, uint32_t* total) {
  bool bad = false;  // (reported by the decode kernel)
  return prefix_scan(p.prefix, p.page_size, p.group, p.num_kv_heads, p.num_seqs, lane,
                     [&](const PrefixGroup& r, uint32_t t) { return r.tile0 <= at && at < r.tile0 + t; }, &bad, total);
}

__device__ __forceinline__ Walk start_walk(const PrefixParams& p, int lane) {
  Walk w;
  uint32_t total;
  // the chunk depends on the total, so the first look finds only that
  (void)find_tile(p, 0xFFFFFFFFu, lane, &total);
  const uint32_t chunk = prefix_chunk(total, p.prefix.ctas);
  const uint64_t lo = uint64_t(blockIdx.x) * chunk;
  w.at = uint32_t(min(lo, uint64_t(total)));
  w.end = uint32_t(min(lo + chunk, uint64_t(total)));
  w.have = false;
  return w;
}

__device__ __forceinline__ bool next_segment(const PrefixParams& p, Walk& w, Segment& s, int lane) {
  if (w.at >= w.end) return false;
  if (!w.have || w.at >= w.g.tile0 + group_tiles(w.g, p.num_kv_heads)) {
    uint32_t total;
    w.g = find_tile(p, w.at, lane, &total);
    w.have = true;
    if (w.g.tiles <= 0) return false;  // (cannot be: the line ends with its groups)
  }
  const uint32_t in = w.at - w.g.tile0;
  const uint32_t u = in / uint32_t(w.g.tiles);
  const int per = prefix_seqs_per_block(p.group);
  s.kvh = int(u / uint32_t(w.g.blocks));
  const int blk = int(u - uint32_t(s.kvh) * w.g.blocks);
  s.leader = w.g.first;
  s.seq0 = w.g.first + blk * per;
  s.rows = min(per, w.g.end - s.seq0) * p.group;
  s.tile = int(in - u * uint32_t(w.g.tiles));
  s.tiles = min(w.g.tiles - s.tile, int(w.end - w.at));
  s.tokens = w.g.tokens;
  s.slot = int64_t(w.g.unit0) + u + blockIdx.x;
  w.at += s.tiles;
  return true;
}

// ------------------------------------------------------------ expanders

// Eight codes of a word as four binary16 pairs of dims (0,4) (1,5) (2,6)
// (3,7).  K: the nibble masked in place, n 2^-24 (dims 0, 4, 2, 6) or n 2^-20
// (1, 5, 3, 7), exact; q' carries 2^-4 in the latter.
__device__ __forceinline__ uint4 codes8(uint32_t w) {
  const uint32_t x = w >> 8;
  return make_uint4(w & 0x000F000Fu, w & 0x00F000F0u, x & 0x000F000Fu, x & 0x00F000F0u);
}
// V: n s + z, rounded once.  1024 + n (1024 + 16 n) is the nibble under
// binary16 exponent bits; n follows exactly, then one fma.
__device__ __forceinline__ uint4 dequant8(uint32_t w, __half2 s, __half2 z) {
  const __half2 k1024 = __float2half2_rn(-1024.0f), k16 = __float2half2_rn(0.0625f), k64 = __float2half2_rn(-64.0f);
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = i ? (w >> 8) : w;
    const uint32_t lo = and_or(x, 0x000F000Fu, 0x64006400u), hi = and_or(x, 0x00F000F0u, 0x64006400u);
    const __half2 a = __hadd2(*reinterpret_cast<const __half2*>(&lo), k1024);
    const __half2 b = __hfma2(*reinterpret_cast<const __half2*>(&hi), k16, k64);
    const __half2 va = __hfma2(a, s, z), vb = __hfma2(b, s, z);
    r[2 * i] = *reinterpret_cast<const uint32_t*>(&va);
    r[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&vb);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// The same through binary32, saturated to the largest binary16: rows whose
// scale or zero binary16 does not hold exactly, or that reach beyond it.
__device__ __noinline__ uint4 dequant8_wide(uint32_t w, float s, float z) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = fmaf(float((w >> (4 * i)) & 15u), s, z), b = fmaf(float((w >> (4 * i + 16)) & 15u), s, z);
    r[i] = pack_half2(fminf(fmaxf(a, -65504.0f), 65504.0f), fminf(fmaxf(b, -65504.0f), 65504.0f));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Key n of a raw tensor tile (64 code bytes per key) into an operand tile:
// dims 8u .. 8u+7 at u * 2048 + n * 16.  widen(word) gives the 16 bytes.
template <typename Widen>
__device__ __forceinline__ void expand_key(const uint8_t* codes, bool ok, uint8_t* dst, int n, Widen widen) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    // rotated 16-byte pieces: eight lanes' rows (64 bytes apart) then fall
    // into different banks
    const int piece = (q + (n >> 1)) & 3;
    const uint4 w = *reinterpret_cast<const uint4*>(codes + n * 64 + 16 * piece);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int u = 0; u < 4; ++u)
      *reinterpret_cast<uint4*>(dst + (4 * piece + u) * 2048 + n * 16) = ok ? widen(ws[u]) : make_uint4(0u, 0u, 0u, 0u);
  }
}

// ------------------------------------------------------------ kernel

template <int P, bool F16IN, bool BFM>
__global__ void __launch_bounds__(kThreads, 1) prefix_attn_kernel(const PrefixParams p) {
  pdl_wait_then_release();
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + kOffTmem);
  int* raw_ok = reinterpret_cast<int*>(smem + kOffOk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int b = 0; b < kRawStages; ++b) {
      mbar_init(&bars[kRawFull + b], 1);
      mbar_init(&bars[kRawEmpty + b], 6);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars[kKFull + b], 2);
      mbar_init(&bars[kKEmpty + b], 1);
      mbar_init(&bars[kVFull + b], 4);
      mbar_init(&bars[kPvDone + b], 1);
      mbar_init(&bars[kSFull + b], 1);
      mbar_init(&bars[kPFull + b], kSoftWarps);
    }
    for (int b = 0; b < kMetas; ++b) mbar_init(&bars[kMetaFull + b], 2);
    mbar_init(&bars[kQFull], kSoftWarps);
    mbar_init(&bars[kMmaDone], 1);
    mbar_fence_init();
  }
  if (warp == kWarpMma) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  bool failed = false;
  Segment sg;
  Walk walk = start_walk(p, lane);
  uint32_t it = 0;  // tiles of this CTA so far

  if (warp < kSoftWarps) {
    // ---------------------------------------------------------- softmax
    const int r = 32 * warp + lane;                 // row, tensor-memory lane
    const uint32_t tl = tmem + (uint32_t(32 * warp) << 16);
    while (next_segment(p, walk, sg, lane)) {
      const bool live = r < sg.rows;
      float a, qc;
      {
        // ---- q': rotate, scale by 2^S with max |q'| 2^S < 2^14, store
        float v[128];
        if (live) {
          const int sq = sg.seq0 + r / p.group, h = r % p.group;
          const uint4* src = reinterpret_cast<const uint4*>(
              p.q + (int64_t(sq) * p.num_q_heads + sg.kvh * p.group + h) * kHeadDim);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint4 w = src[k];
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[8 * k + 2 * j] = in_lo(ws[j], F16IN);
              v[8 * k + 2 * j + 1] = in_hi(ws[j], F16IN);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 128; ++i) v[i] = 0.0f;
        }
        if (p.rotate_k) {
#pragma unroll
          for (int s = 1; s < 128; s <<= 1) {
            if (s < p.block_h) {
#pragma unroll
              for (int i = 0; i < 128; ++i)
                if (!(i & s)) {
                  const float x = v[i], y = v[i + s];
                  v[i] = x + y;
                  v[i + s] = x - y;
                }
            }
          }
#pragma unroll
          for (int i = 0; i < 128; ++i) v[i] *= p.c_h;
        }
        float mx = 0.0f, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 128; ++i) {
          mx = fmaxf(mx, fabsf(v[i]));
          sum += v[i];
        }
        const int E = int((__float_as_uint(mx) >> 23) & 0xFFu);
        const int S = min(100, max(-100, 140 - E));
        const float up = __uint_as_float(uint32_t(127 + S) << 23);
        // codes are n 2^-24: t = a (s_k acc + z_k qc)
        a = p.q_scale * __uint_as_float(uint32_t(127 - S) << 23) * 16777216.0f;
        qc = sum * up * 5.9604644775390625e-08f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          uint32_t hw[4], lw[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float f = (j & 1) ? up * 0.0625f : up;
            const float x0 = v[8 * k + j] * f, x1 = v[8 * k + j + 4] * f;
            const __half h0 = __float2half_rn(x0), h1 = __float2half_rn(x1);
            hw[j] = uint32_t(__half_as_ushort(h0)) | (uint32_t(__half_as_ushort(h1)) << 16);
            lw[j] = pack_half2(x0 - __half2float(h0), x1 - __half2float(h1));
          }
          tmem_st4u(tl + kColQh + 4 * k, hw);
          tmem_st4u(tl + kColQl + 4 * k, lw);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      arrive_elect(&bars[kQFull]);

      float m = -INFINITY, l = 0.0f;
      for (int i = 0; i < sg.tiles; ++i, ++it) {
        const int b = it & 1;
        wait_all(&bars[kMetaFull + (it & (kMetas - 1))], (it / kMetas) & 1, failed);
        wait_all(&bars[kSFull + b], (it >> 1) & 1, failed);
        tc_fence_after();
        const uint32_t col = tl + 128 * b;
        float s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_issue(col + 32 * c, s + 32 * c);
        const uint8_t* meta = smem + kOffMeta + (it & (kMetas - 1)) * kMetaBytes;
        const float4* ms = reinterpret_cast<const float4*>(meta);
        const float4* mz = ms + kKeys / 4;
        const int okm = *reinterpret_cast<const int*>(meta + kKeys * 8);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) pin32(s + 32 * c);
        const float2 qc2 = make_float2(qc, qc);
        float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float4 sk = ms[j], zk = mz[j];
          const float2 x = fma2(make_float2(sk.x, sk.y), make_float2(s[4 * j], s[4 * j + 1]),
                                mul2(qc2, make_float2(zk.x, zk.y)));
          const float2 y = fma2(make_float2(sk.z, sk.w), make_float2(s[4 * j + 2], s[4 * j + 3]),
                                mul2(qc2, make_float2(zk.z, zk.w)));
          s[4 * j] = x.x;
          s[4 * j + 1] = x.y;
          s[4 * j + 2] = y.x;
          s[4 * j + 3] = y.y;
        }
        if (okm != 0xFF) {  // keys past the prefix or on a bad page
#pragma unroll
          for (int j = 0; j < 128; ++j)
            if (!((okm >> (j >> 4)) & 1)) s[j] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < 128; j += 8) {
#pragma unroll
          for (int c = 0; c < 4; ++c) top4[c] = max3(top4[c], s[j + 2 * c], s[j + 2 * c + 1]);
        }
        const float top = a * fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
        // move the reference when the maximum outgrew it (first tile: always)
        const bool move = top > m + 8.0f || (m == -INFINITY && top > -INFINITY);
        if (__any_sync(kAll, move)) {
          const float f = move ? ex2(m - top) : 1.0f;  // 0 while m is -inf
          l *= f;
          if (i > 0 && wait_all(&bars[kPvDone + (b ^ 1)], ((it - 1) >> 1) & 1, failed)) {
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              float o[16];
              tmem_ld16(tl + kColO + 16 * c, o);
              uint32_t ow[16];
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                const float2 x = mul2(make_float2(o[j], o[j + 1]), make_float2(f, f));
                ow[j] = __float_as_uint(x.x);
                ow[j + 1] = __float_as_uint(x.y);
              }
              tmem_st16u(tl + kColO + 16 * c, ow);
            }
          }
          if (move) m = top;
        }
        const float nm = m == -INFINITY ? 0.0f : -m;
        const float2 a2 = make_float2(a, a), nm2 = make_float2(nm, nm);
        float2 la = make_float2(0.0f, 0.0f), lb = la;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pw[16];
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const int k = 32 * c + 2 * j;
            const float2 x = fma2(a2, make_float2(s[k], s[k + 1]), nm2);
            const float2 y = fma2(a2, make_float2(s[k + 2], s[k + 3]), nm2);
            const float2 px = make_float2(ex2(x.x), ex2(x.y)), py = make_float2(ex2(y.x), ex2(y.y));
            la = add2(la, px);
            lb = add2(lb, py);
            pw[j] = pack_half2(px.x, px.y);
            pw[j + 1] = pack_half2(py.x, py.y);
          }
          tmem_st16u(col + 16 * c, pw);
        }
        tmem_wait_st();
        l += (la.x + la.y) + (lb.x + lb.y);
        tc_fence_before();
        __syncwarp();
        arrive_elect(&bars[kPFull + b]);
      }
      // ---- the partial result, once the last P V has completed
      wait_all(&bars[kPvDone + ((it - 1) & 1)], ((it - 1) >> 1) & 1, failed);
      tc_fence_after();
      float4* part = reinterpret_cast<float4*>(p.prefix.part) + prefix_part_index(sg.slot) + r;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float o[32];
        tmem_ld32_issue(tl + kColO + 32 * c, o);
        tmem_wait_ld();
        pin32(o);
        if (live) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // columns of 8 dims: 0 4 1 5 2 6 3 7
            __stcg(part + (8 * c + 2 * k) * 128, make_float4(o[8 * k], o[8 * k + 2], o[8 * k + 4], o[8 * k + 6]));
            __stcg(part + (8 * c + 2 * k + 1) * 128, make_float4(o[8 * k + 1], o[8 * k + 3], o[8 * k + 5], o[8 * k + 7]));
          }
        }
      }
      if (live)
        __stcg(reinterpret_cast<float2*>(p.prefix.part_ml) + sg.slot * kPrefixRows + r,
               failed ? make_float2(-INFINITY, 0.0f) : make_float2(m, l));
    }
    if (failed && lane == 0) report(p.dev_status, SAW_ERR_DEVICE_TIMEOUT);
  } else if (warp == kWarpProd) {
    // ---------------------------------------------------------- producer
    constexpr int kChunk = P * 68;
    constexpr int kPages = kKeys / P;               // pages per tile
    while (!failed && next_segment(p, walk, sg, lane)) {
      const int32_t* btab = p.block_tables + int64_t(sg.leader) * p.max_blocks;
      const int n_pages = sg.tokens / P;
      for (int i = 0; i < sg.tiles; ++i, ++it) {
        const int st = it % kRawStages;
        // lane l: page l / 4 of the tile; K codes, V codes, K words, V words
        const int pg = lane >> 2, kind = lane & 3;
        const int lp = (sg.tile + i) * kPages + pg;
        int id = -1;
        if (pg < kPages && lp < n_pages) {
          id = btab[lp];
          if (id < 0 || id >= p.num_pages) {
            if (kind == 0) report(p.dev_status, SAW_ERR_DEVICE_INDEX);
            id = -1;
          }
        }
        const uint32_t have = __ballot_sync(kAll, id >= 0 && kind == 0);  // bit 4 pg
        if (it >= kRawStages && !wait_all(&bars[kRawEmpty + st], ((it / kRawStages) - 1) & 1, failed)) break;
        uint8_t* raw = smem + kOffRaw + st * kRawBytes;
        if (lane == 0) {
          int okm = 0;
#pragma unroll
          for (int g = 0; g < kPages; ++g)
            if ((have >> (4 * g)) & 1) okm |= ((1 << (P / 16)) - 1) << (g * (P / 16));
          raw_ok[st] = okm;
          if (have)
            mbar_arrive_expect_tx(&bars[kRawFull + st], uint32_t(__popc(have)) * (2 * kChunk));
          else
            mbar_arrive(&bars[kRawFull + st]);
        }
        __syncwarp();
        if (id >= 0) {
          const int64_t off = (int64_t(id) * p.num_kv_heads + sg.kvh) * kChunk;
          const uint8_t* src = (kind & 1 ? p.v_cache : p.k_cache) + off + (kind >> 1 ? P * 64 : 0);
          uint8_t* dst = raw + (kind == 0 ? 0 : kind == 1 ? kRawV : kind == 2 ? kRawKM : kRawVM) +
                         pg * (kind >> 1 ? P * 4 : P * 64);
          bulk_g2s(dst, src, kind >> 1 ? P * 4 : P * 64, &bars[kRawFull + st]);
        }
        __syncwarp();
      }
    }
    if (failed && lane == 0) report(p.dev_status, SAW_ERR_DEVICE_TIMEOUT);
    // the CTA must not exit while a copy into its shared memory is in flight
    for (uint32_t i = it > kRawStages ? it - kRawStages : 0; i < it; ++i)
      (void)mbar_wait_bounded(&bars[kRawFull + i % kRawStages], (i / kRawStages) & 1);
  } else if (warp == kWarpMma) {
    // ---------------------------------------------------------- MMA issue
    constexpr uint32_t id_s = umma_idesc_f16(128, kKeys);
    constexpr uint32_t id_o = umma_idesc_f16(128, kHeadDim) | kUmmaBMnMajor;
    const uint32_t k0 = smem_u32(smem + kOffK), v0 = smem_u32(smem + kOffV);
    uint32_t segs = 0;
    auto score = [&](uint32_t t) {  // S of tile t into buffer t & 1
      const int b = t & 1;
      if (!wait_all(&bars[kKFull + b], (t >> 1) & 1, failed)) return;
      tc_fence_after();
      const uint64_t bd = umma_desc(k0 + b * kOpBytes, 2048, 128);
#pragma unroll
      for (int ks = 0; ks < kHeadDim / 16; ++ks)
        umma_ts_elect(tmem + 128 * b, tmem + kColQh + 8 * ks, bd + ks * (4096 >> 4), id_s, ks > 0);
#pragma unroll
      for (int ks = 0; ks < kHeadDim / 16; ++ks)
        umma_ts_elect(tmem + 128 * b, tmem + kColQl + 8 * ks, bd + ks * (4096 >> 4), id_s, true);
      commit_elect(&bars[kSFull + b]);
      commit_elect(&bars[kKEmpty + b]);
    };
    while (!failed && next_segment(p, walk, sg, lane)) {
      if (!wait_all(&bars[kQFull], segs & 1, failed)) break;
      ++segs;
      score(it);
      for (int i = 0; i < sg.tiles && !failed; ++i, ++it) {
        const int b = it & 1;
        if (i + 1 < sg.tiles) score(it + 1);
        wait_all(&bars[kVFull + b], (it >> 1) & 1, failed);
        if (!wait_all(&bars[kPFull + b], (it >> 1) & 1, failed)) break;
        tc_fence_after();
        const uint64_t bd = umma_desc(v0 + b * kOpBytes, 128, 2048);
#pragma unroll
        for (int ks = 0; ks < kKeys / 16; ++ks)
          umma_ts_elect(tmem + kColO, tmem + 128 * b + 8 * ks, bd + ks * (256 >> 4), id_o, i > 0 || ks > 0);
        commit_elect(&bars[kPvDone + b]);
      }
    }
    if (failed && lane == 0) report(p.dev_status, SAW_ERR_DEVICE_TIMEOUT);
    // every MMA has completed before tensor memory is released
    commit_elect(&bars[kMmaDone]);
    (void)mbar_wait_bounded(&bars[kMmaDone], 0);
    __syncwarp();
  } else {
    // ---------------------------------------------------------- expanders
    const bool is_v = warp < kWarpK;
    while (!failed && next_segment(p, walk, sg, lane)) {
      for (int i = 0; i < sg.tiles; ++i, ++it) {
        const int st = it % kRawStages, b = it & 1;
        if (!wait_all(&bars[kRawFull + st], (it / kRawStages) & 1, failed)) break;
        const uint8_t* raw = smem + kOffRaw + st * kRawBytes;
        const int okm = raw_ok[st];
        if (is_v) {
          const int n = tid - 32 * kWarpV;          // key of the tile
          const bool ok = (okm >> (n >> 4)) & 1;
          const uint32_t w = *reinterpret_cast<const uint32_t*>(raw + kRawVM + 4 * n);
          const float sf = meta_lo(w, BFM), zf = meta_hi(w, BFM);
          // every value below binary16's largest; bfloat16 words also exact in
          // it (eight significant bits: from 2^-17 up)
          bool plain = fmaf(15.0f, sf, fabsf(zf)) <= 65504.0f;
          if (BFM) plain = plain && (sf == 0.0f || sf >= 0x1p-17f) && (zf == 0.0f || fabsf(zf) >= 0x1p-17f);
          const __half2 s = __float2half2_rn(sf), z = __float2half2_rn(zf);
          if (it >= 2 && !wait_all(&bars[kPvDone + b], ((it >> 1) - 1) & 1, failed)) break;
          expand_key(raw + kRawV, ok, smem + kOffV + b * kOpBytes, n,
                     [&](uint32_t x) { return plain ? dequant8(x, s, z) : dequant8_wide(x, sf, zf); });
          fence_async_smem();
          __syncwarp();
          arrive_elect(&bars[kVFull + b]);
        } else {
          // K: codes as they are; scales and zeros for the softmax.  Meta slot
          // it % 4 was read for tile it - 4: its P was used by the P V that
          // precedes the scores of tile it - 2, whose end freed this K buffer.
          if (it >= 2 && !wait_all(&bars[kKEmpty + b], ((it >> 1) - 1) & 1, failed)) break;
          uint8_t* meta = smem + kOffMeta + (it & (kMetas - 1)) * kMetaBytes;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int n = tid - 32 * kWarpK + 64 * u;
            const bool ok = (okm >> (n >> 4)) & 1;
            const uint32_t w = *reinterpret_cast<const uint32_t*>(raw + kRawKM + 4 * n);
            reinterpret_cast<float*>(meta)[n] = ok ? meta_lo(w, BFM) : 0.0f;
            reinterpret_cast<float*>(meta)[kKeys + n] = ok ? meta_hi(w, BFM) : 0.0f;
            expand_key(raw, ok, smem + kOffK + b * kOpBytes, n, [](uint32_t x) { return codes8(x); });
          }
          if (tid == 32 * kWarpK) *reinterpret_cast<int*>(meta + kKeys * 8) = okm;
          fence_async_smem();
          __syncwarp();
          arrive_elect(&bars[kKFull + b]);
          arrive_elect(&bars[kMetaFull + (it & (kMetas - 1))]);
        }
        arrive_elect(&bars[kRawEmpty + st]);
      }
    }
    if (failed && lane == 0) report(p.dev_status, SAW_ERR_DEVICE_TIMEOUT);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int P, bool F16IN, bool BFM>
cudaError_t launch_f(const PrefixParams& p, cudaStream_t stream) {
  auto kernel = prefix_attn_kernel<P, F16IN, BFM>;
  cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.prefix.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int P>
cudaError_t launch_p(const PrefixParams& p, cudaStream_t stream) {
  if (p.in_f16) return p.meta_bf16 ? launch_f<P, true, true>(p, stream) : launch_f<P, true, false>(p, stream);
  return p.meta_bf16 ? launch_f<P, false, true>(p, stream) : launch_f<P, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_prefix_attn(const PrefixParams& p, cudaStream_t stream) {
  switch (p.page_size) {
    case 16: return launch_p<16>(p, stream);
    case 32: return launch_p<32>(p, stream);
    case 64: return launch_p<64>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace saw
