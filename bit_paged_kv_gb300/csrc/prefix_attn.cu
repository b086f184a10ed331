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
// exact), q' -- the rotated q times the softmax scale, log2 e and 2^4 -- as
// binary16 hi + lo parts, so a score t = s_k (q'.n) + z_k sum(q') comes out in
// base 2 to about 2^-22 of its terms, as in the decode (|q'| 2^4 saturates at
// 65504, a score of thousands).  V^ = n s_V + z_V is dequantized and rounded once
// to binary16 (no coarser than the 16-bit rows the cache was made from), p
// too: O += P V^ in binary32, where sum(p s n) + sum(p z) would cancel.
// Softmax in base 2 in binary32 with a running reference m, set 7 below the
// row's maximum, that moves (and rescales O and l) only when the maximum has
// come to exceed it by more than 15: p <= 2^15 stays inside binary16, and the
// merge's normalisation makes the choice of m invisible.  The 2^7 are for faint
// keys: l counts p before its rounding, O after, and binary16 ends at 2^-24, so
// a key counts in both down to 2^-32 of the row's heaviest (with m the maximum,
// 2^-25: 100000 such keys would take 0.3 % from the output).
//
// Twenty-four warps, specialised:
//   0-7, 8-15  softmax of even and odd tiles, run a tile apart so that one
//          set's loads and exponentials fill the other's waits.  A warp has 16
//          rows (half of the 32 tensor-memory lanes it can reach), a thread 2
//          rows x 32 keys (the 16 x 256-bit access): whole rows in a warp, so
//          no maximum crosses warps, and the per-key (s_k, z_k) cost 16 shared
//          loads for 64 scores (one row per thread: 64 loads for 128, every
//          lane the same words).  A warp without a row of the block only keeps
//          the barriers' count (28 rows: 80 -> 74 us of 37 requests behind five
//          prompts).  The running reference m of a row passes from set to set in
//          tile order.  p goes back over the scores' columns as
//          the A operand of P V.
//   16-19  V expanders: one key per thread; 20-21: K expanders, two keys each
//   22     producer: the list of work, and bulk copies of whole page chunks
//   23     MMA: one elected lane issues the products of tile i + 1's scores
//          before tile i's P V, so that the softmax of tile i runs behind them
// Latency, not any unit's rate, sets the pace: a set's softmax (2 warps per
// scheduler) and the two products it waits for follow one another.
// Measured (GB300): 64 sequences, 32 q-heads over 8, behind 16384 tokens, 2048
// tiles on 152 SMs, 34 us: 1.3 us a tile (its three products alone 1.0), 9.7 us
// from the start to the first score -- the plan, page ids, first copies and
// first K tile one after the other, all of it code fetched cold -- and 1.1 us for
// a part's results.
// The softmax warps draw registers from the others (96 and 48 a thread).
// The 512 tensor-memory columns hold two score tiles (the second one makes the
// overlap), O, and q' hi and lo: the score products read only K from shared
// memory.  Operands there are unswizzled 8-row x 16-byte core matrices, two
// tiles each of K and V.  An expander writes each 8 dims in the order 0 4 1 5
// 2 6 3 7, the order in which masking a word of codes yields pairs; q' is
// stored in that order and the output columns are put back when written.
// q' is rotated by the tensor cores too: q times H, a matrix of +-1 (the
// identity when K is not rotated) that the V expanders write; both pass
// through the V buffers, which are free between segments.  (By shuffles, a row
// per warp at a time, the rotation took 11000 cycles of cold, dependent code.)
// Every wait is bounded to about a second.
#include <type_traits>

#include "saw_device.cuh"
#include "saw_int4.h"
#include "saw_prefix.cuh"
#include "saw_quant_row.cuh"
#include "saw_tcgen05.cuh"

namespace saw {
namespace {

constexpr int kThreads = 768;
constexpr int kSoftWarps = 16;
constexpr int kWarpV = 16, kWarpK = 20, kWarpProd = 22, kWarpMma = 23;
constexpr int kLaunchRegs = 80, kSoftRegs = 96, kFeedRegs = 48;
static_assert(4 * kSoftRegs + 2 * kFeedRegs == 6 * kLaunchRegs, "register shares of six warpgroups");
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kKeys = kPrefixKeys;
static_assert(kHeadDim == 128, "eight k-steps of 16");
static_assert(kPrefixRows == 128 && kKeys == 128, "four softmax warps per 32 rows, one key per V expander thread");

constexpr int kOpBytes = 128 * 128 * 2;            // one operand tile
constexpr int kRawV = kKeys * 68;                  // raw stage: the pages' K chunks, then their V chunks
constexpr int kRawBytes = 2 * kKeys * 68;          // 17408
constexpr int kRawStages = 4;
constexpr int kMetas = 4;                          // tiles of (s_k, z_k) for the softmax
constexpr int kMetaBytes = kKeys * 8 + 16;         // (s, s, z, z) per key pair, valid 16-key slices
constexpr int kOffK = 0, kOffV = kOffK + 2 * kOpBytes;
constexpr int kOffRaw = kOffV + 2 * kOpBytes;
constexpr int kOffMeta = kOffRaw + kRawStages * kRawBytes;
constexpr int kOffOk = kOffMeta + kMetas * kMetaBytes;  // valid 16-key slices of the raw stages
constexpr int kOffM = kOffOk + 4 * kRawStages;          // f32 [128]: the rows' running references
// (apart: with one tile the set without it writes its (m, l) while the other may
// still be adding up sum(q'))
constexpr int kOffSum = kOffM + 128 * 4;                // f32 [4][128]: parts of sum(q')
constexpr int kOffRow = kOffSum + 4 * 128 * 4;          // f32x2 [2][128]: each set's (m, l) at the end
constexpr int kSegs = 4;                                // segments announced ahead
constexpr int kOffSeg = kOffRow + 2 * 128 * 8;
constexpr int kOffBar = kOffSeg + kSegs * 48;
enum { kRawFull = 0, kRawEmpty = kRawFull + kRawStages, kKFull = kRawEmpty + kRawStages, kKEmpty = kKFull + 2,
       kVFull = kKEmpty + 2, kPvDone = kVFull + 2, kMetaFull = kPvDone + 2, kSFull = kMetaFull + kMetas,
       kPFull = kSFull + 2, kTurn = kPFull + 2, kSegFull = kTurn + 16, kSegEmpty = kSegFull + kSegs, kQIn = kSegEmpty + kSegs, kQRot, kQFull, kMmaDone, kBars };
constexpr int kOffTmem = kOffBar + kBars * 8;
constexpr int kSmem = kOffTmem + 16;
static_assert(kOffBar % 8 == 0 && kOffMeta % 16 == 0 && kOffM % 16 == 0 && kSmem <= 227 * 1024, "shared memory");
constexpr float kRefBelow = 7.0f, kRefMost = 15.0f;  // a row's maximum above its reference
constexpr uint32_t kColO = 256, kColQh = 384, kColQl = 448;

// ------------------------------------------------------------ PTX pieces

// Eight k-steps of one product by one elected lane: D [+]= A B^T, B advancing
// by kStepB per step.  (One asm block: operands are converted to uniform
// registers per instruction, and with an election each the 24 products of a
// tile were 13 KB of code.)
template <int64_t kStepA, int64_t kStepB>
__device__ __forceinline__ void umma_ss8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\t.reg .b64 a64;\n\t"
      "setp.ne.u32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 b, %2;\n\tmov.b64 a64, %1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a64, b, %3, p;\n\t"
      "add.s64 b, b, %5;\n\tadd.s64 a64, a64, %6;\n\tsetp.eq.u32 p, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a64, b, %3, p;\n\t"
      "add.s64 b, b, %5;\n\tadd.s64 a64, a64, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a64, b, %3, p;\n\t"
      "add.s64 b, b, %5;\n\tadd.s64 a64, a64, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a64, b, %3, p;\n\t"
      "add.s64 b, b, %5;\n\tadd.s64 a64, a64, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a64, b, %3, p;\n\t"
      "add.s64 b, b, %5;\n\tadd.s64 a64, a64, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a64, b, %3, p;\n\t"
      "add.s64 b, b, %5;\n\tadd.s64 a64, a64, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a64, b, %3, p;\n\t"
      "add.s64 b, b, %5;\n\tadd.s64 a64, a64, %6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a64, b, %3, p;\n\t"
      "}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc)), "n"(kStepB), "n"(kStepA)
      : "memory");
}
// The same with A in tensor memory (8 columns per step).
template <int64_t kStepB>
__device__ __forceinline__ void umma_ts8(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\t.reg .b32 a32;\n\t"
      "setp.ne.u32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 b, %2;\n\tmov.b32 a32, %1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a32], b, %3, p;\n\t"
      "add.s64 b, b, %5;\n\tadd.s32 a32, a32, 8;\n\tsetp.eq.u32 p, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a32], b, %3, p;\n\t"
      "add.s64 b, b, %5;\n\tadd.s32 a32, a32, 8;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a32], b, %3, p;\n\t"
      "add.s64 b, b, %5;\n\tadd.s32 a32, a32, 8;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a32], b, %3, p;\n\t"
      "add.s64 b, b, %5;\n\tadd.s32 a32, a32, 8;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a32], b, %3, p;\n\t"
      "add.s64 b, b, %5;\n\tadd.s32 a32, a32, 8;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a32], b, %3, p;\n\t"
      "add.s64 b, b, %5;\n\tadd.s32 a32, a32, 8;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a32], b, %3, p;\n\t"
      "add.s64 b, b, %5;\n\tadd.s32 a32, a32, 8;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a32], b, %3, p;\n\t"
      "}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc)), "n"(kStepB)
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
__device__ __forceinline__ void expect_tx_elect(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
      "@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void bulk_elect(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t"
      "@p cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
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
// 16 lanes x 64 columns: register 4k + j of lane 4g + c is row g (j < 2) or g +
// 8, column 8k + 2c + (j & 1) -- the layout of a 16 x 8 accumulator per k.
__device__ __forceinline__ void tmem_ld_16x256_issue(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
        "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
// The same for 16 columns, loaded (and waited for) and stored.
__device__ __forceinline__ void tmem_ld_16x256_x2(uint32_t taddr, float (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st_16x256_x2(uint32_t taddr, const float (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// 16 lanes x 32 columns: register 2k + j of lane 4g + c is row g + 8j, column 4k + c.
__device__ __forceinline__ void tmem_st_16x128(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
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

// Within binary16's finite range; a NaN stays one.
__device__ __forceinline__ float clamp16(float x) {
  asm("{\n\tmax.NaN.f32 %0, %0, %1;\n\tmin.NaN.f32 %0, %0, %2;\n\t}" : "+f"(x) : "f"(-65504.0f), "f"(65504.0f));
  return x;
}

// {x, x} as a register pair, built once instead of per packed instruction.
__device__ __forceinline__ uint64_t twice(float x) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
  return r;
}
// (v0, v1) = s (v0, v1) + (z qs + nm) for a key pair's sz = (s, s, z, z)
__device__ __forceinline__ void score2(float& v0, float& v1, const float4& sz, uint64_t qs, uint64_t nm) {
  asm("{\n\t.reg .b64 v, s, z;\n\t"
      "mov.b64 v, {%0, %1};\n\tmov.b64 s, {%2, %3};\n\tmov.b64 z, {%4, %5};\n\t"
      "fma.rn.f32x2 z, z, %6, %7;\n\tfma.rn.f32x2 v, s, v, z;\n\t"
      "mov.b64 {%0, %1}, v;\n\t}"
      : "+f"(v0), "+f"(v1)
      : "f"(sz.x), "f"(sz.y), "f"(sz.z), "f"(sz.w), "l"(qs), "l"(nm));
}
// Waits of a whole warp; after a failure every later wait returns at once.
// The loop is a handful of instructions (forty such waits with a clock in each
// were a fifth of the kernel's code) and bounded by its count: a try returns
// after the suspend hint at the latest (10 us: the feeding warps park, leaving
// their scheduler's issue slots to the others), or at once without one, 20
// cycles or more a try -- a second, or a few.
template <bool PARK>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, bool& failed) {
  if (failed) return false;
  uint32_t ok;
  if constexpr (PARK) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 n;\n\tmov.b32 n, 0;\n\t"
        "WAIT_AGAIN:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 10000;\n\t"
        "@p bra WAIT_DONE;\n\tadd.u32 n, n, 1;\n\tsetp.lt.u32 q, n, 200000;\n\t@q bra WAIT_AGAIN;\n\t"
        "WAIT_DONE:\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 n;\n\tmov.b32 n, 0;\n\t"
        "WAIT_AGAIN:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra WAIT_DONE;\n\tadd.u32 n, n, 1;\n\tsetp.lt.u32 q, n, 100000000;\n\t@q bra WAIT_AGAIN;\n\t"
        "WAIT_DONE:\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
  }
  failed = !__all_sync(kAll, ok != 0);
  return !failed;
}
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, bool& failed) {
  return wait_warp<false>(bar, parity, failed);
}
__device__ __forceinline__ bool wait_parked(uint64_t* bar, uint32_t parity, bool& failed) {
  return wait_warp<true>(bar, parity, failed);
}

// The four softmax warps that share this thread's 32 rows meet; the AND of
// `ok` over their threads.
__device__ __forceinline__ bool rows_sync(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(uint32_t(ok)), "r"(1 + int((threadIdx.x >> 5) & 3)), "r"(128)
      : "memory");
  return r != 0;
}

// ------------------------------------------------------------ work list

struct __align__(16) Segment {
  int kvh;
  int first, end;    // the group's sequences
  int seq0, rows;    // first sequence of the block; its (sequence, head) rows (at most 128)
  int tile, tiles;   // key tiles of the prefix to do
  int tokens;        // tokens of the whole prefix
  int more;          // 0: no segment, the end
  int64_t slot;
};
static_assert(sizeof(Segment) == 48, "kOffSeg");

// The producer warp finds this CTA's parts and announces them to the other
// warps through a ring in shared memory: one copy of this code (in every role
// it was half of a kernel of 137 KB, and instruction fetches were a fifth of
// all stalls).  With up to 32 groups a lane keeps its group in registers.
struct Work {
  PrefixGroup mine;   // group base + lane
  int base;
  uint32_t chunk;     // tiles per part
  uint32_t next;      // this CTA's next part
  uint32_t before;    // parts of the groups before `base`
  int top;            // furthest end of the groups up to base + 31
};

__device__ __forceinline__ uint32_t group_parts(const PrefixGroup& g, int hkv, uint32_t chunk) {
  return uint32_t(g.blocks) * hkv * ((uint32_t(g.tiles) + chunk - 1) / chunk);
}

// Whole warp: the groups' first 32, and the chunk.  Lanes weigh chunks
// ceil(Tmax / n) for n = 1 .. 64 parts of the longest prefix, two each: rounds
// of the fullest CTA times the cost of a part.  More parts than max(units, 2
// CTAs) are not considered (the workspace holds no more).
__device__ __forceinline__ Work plan_work(const PrefixParams& p, int lane) {
  Work w;
  bool bad = false;  // (reported by the decode kernel)
  int top = 0, tmax = 0;
  w.base = 0;
  w.before = 0;
  for (int g0 = 0; g0 < max(p.prefix.num_groups, 1); g0 += 32) {
    const PrefixGroup r = prefix_load(p.prefix, g0, p.page_size, p.group, p.num_seqs, lane, &top, &bad);
    if (g0 == 0) {
      w.mine = r;
      w.top = top;
    }
    tmax = max(tmax, r.blocks > 0 ? r.tiles : 0);
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) tmax = max(tmax, __shfl_xor_sync(kAll, tmax, d));
  tmax = max(tmax, 1);
  uint32_t c[2], parts[2] = {0, 0}, units = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) c[k] = (uint32_t(tmax) + 2 * lane + k) / (2 * lane + k + 1);
  top = w.top;
  for (int g0 = 0; g0 < p.prefix.num_groups; g0 += 32) {
    PrefixGroup r = w.mine;
    if (g0 > 0) r = prefix_load(p.prefix, g0, p.page_size, p.group, p.num_seqs, lane, &top, &bad);
    const int n = min(32, p.prefix.num_groups - g0);
    for (int g = 0; g < n; ++g) {
      const uint32_t u = uint32_t(__shfl_sync(kAll, r.blocks, g)) * p.num_kv_heads;
      const uint32_t t = uint32_t(__shfl_sync(kAll, r.tiles, g));
      units += u;
#pragma unroll
      for (int k = 0; k < 2; ++k) parts[k] += u * ((t + c[k] - 1) / c[k]);
    }
  }
  uint32_t best = 0xFFFFFFFFu, cost = 0xFFFFFFFFu;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t x = ((parts[k] + p.prefix.ctas - 1) / p.prefix.ctas) * (c[k] + kPartCost);
    const bool fits = parts[k] <= max(units, 2u * p.prefix.ctas);
    if (fits && x < cost) {
      cost = x;
      best = c[k];
    }
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    const uint32_t oc = __shfl_xor_sync(kAll, cost, d), ob = __shfl_xor_sync(kAll, best, d);
    if (oc < cost || (oc == cost && ob > best)) {
      cost = oc;
      best = ob;
    }
  }
  w.chunk = best;
  w.next = blockIdx.x;
  return w;
}

// Whole warp: the next part of this CTA, or false after the last.  CTA 0 also
// leaves the plan for the decode kernel on its way.
__device__ __forceinline__ bool next_segment(const PrefixParams& p, Work& w, Segment& s, int lane) {
  for (;;) {
    const uint32_t n = group_parts(w.mine, p.num_kv_heads, w.chunk);
    const uint32_t upto = w.before + warp_scan_u32(n, lane);
    const uint32_t hit = __ballot_sync(kAll, w.next < upto);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const PrefixGroup g = prefix_from(w.mine, src);
      const uint32_t part = w.next - __shfl_sync(kAll, upto - n, src);
      const uint32_t per_unit = (uint32_t(g.tiles) + w.chunk - 1) / w.chunk;
      const uint32_t u = part / per_unit, j = part - u * per_unit;
      const int per = prefix_seqs_per_block(p.group);
      s.kvh = int(u / uint32_t(g.blocks));
      const int blk = int(u - uint32_t(s.kvh) * g.blocks);
      s.first = g.first;
      s.end = g.end;
      s.seq0 = g.first + blk * per;
      s.rows = min(per, g.end - s.seq0) * p.group;
      s.tile = int(j * uint32_t(g.tiles) / per_unit);
      s.tiles = int((j + 1) * uint32_t(g.tiles) / per_unit) - s.tile;
      s.tokens = g.tokens;
      s.slot = int64_t(w.next);
      w.next += gridDim.x;
      return true;
    }
    // beyond these 32 groups
    w.before = __shfl_sync(kAll, upto, 31);
    w.base += 32;
    if (w.base >= p.prefix.num_groups) return false;
    bool bad = false;
    w.mine = prefix_load(p.prefix, w.base, p.page_size, p.group, p.num_seqs, lane, &w.top, &bad);
  }
}

// CTA 0's producer warp, when its own work is done: the plan.
__device__ __forceinline__ void publish_plan(const PrefixParams& p, uint32_t chunk, int lane) {
  int top = 0;
  bool bad = false;
  uint32_t before = 0;
  if (lane == 0) p.prefix.plan[0] = int(chunk);
  for (int g0 = 0; g0 < p.prefix.num_groups; g0 += 32) {
    const PrefixGroup r = prefix_load(p.prefix, g0, p.page_size, p.group, p.num_seqs, lane, &top, &bad);
    const uint32_t n = group_parts(r, p.num_kv_heads, chunk), upto = before + warp_scan_u32(n, lane);
    if (g0 + lane < p.prefix.num_groups) p.prefix.plan[1 + g0 + lane] = int(upto - n);
    before = __shfl_sync(kAll, upto, 31);
  }
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
__device__ __forceinline__ uint4 dequant8_wide(uint32_t w, float s, float z) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = fmaf(float((w >> (4 * i)) & 15u), s, z), b = fmaf(float((w >> (4 * i + 16)) & 15u), s, z);
    r[i] = pack_half2(fminf(fmaxf(a, -65504.0f), 65504.0f), fminf(fmaxf(b, -65504.0f), 65504.0f));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Key n's 64 code bytes into an operand tile: dims 8u .. 8u+7 at u * 2048 +
// n * 16.  widen(word) gives the 16 bytes.  kUnroll: V one piece at a time (the
// instruction cache: 64 sequences behind 16384 tokens 65.5 us, 66.5 with four),
// K four (it comes first: 37 behind five prompts 73.4 us, 77 with one).
template <int kUnroll, typename Widen>
__device__ __forceinline__ void expand_key(const uint8_t* codes, uint8_t* dst, int n, Widen widen) {
#pragma unroll kUnroll
  for (int q = 0; q < 4; ++q) {
    // rotated 16-byte pieces: eight lanes' rows (64 bytes apart) then fall
    // into different banks
    const int piece = (q + (n >> 1)) & 3;
    const uint4 w = *reinterpret_cast<const uint4*>(codes + 16 * piece);
    uint8_t* d = dst + 4 * piece * 2048 + n * 16;
    *reinterpret_cast<uint4*>(d) = widen(w.x);
    *reinterpret_cast<uint4*>(d + 2048) = widen(w.y);
    *reinterpret_cast<uint4*>(d + 4096) = widen(w.z);
    *reinterpret_cast<uint4*>(d + 6144) = widen(w.w);
  }
}

// Column n of the rotated q -- dim d = 8 (n / 8) + {0 4 1 5 2 6 3 7}[n % 8] --
// as row n of the B operand: H[d][j] = (-1)^popcount(d & j) within blocks of
// h (h = 1: the identity), times 2^-4 in the pairs whose codes are n 2^-20.
template <bool F16IN>
__device__ __forceinline__ void write_hadamard(uint8_t* dst, int n, int h) {
  const int at = n & 7, d = (n & ~7) + ((at >> 1) | ((at & 1) << 2));
  const uint32_t one = ((at >> 1) & 1) ? (F16IN ? 0x2C00u : 0x3D80u) : (F16IN ? 0x3C00u : 0x3F80u);
  uint32_t w[4];  // j & 7 = 0 .. 7
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    uint32_t lo = one | ((__popc(d & (2 * t)) & 1) << 15), hi = one | ((__popc(d & (2 * t + 1) & 7) & 1) << 15);
    if (h == 1) {
      lo = (d & 7) == 2 * t ? one : 0u;
      hi = (d & 7) == 2 * t + 1 ? one : 0u;
    }
    w[t] = lo | (hi << 16);
  }
  const int hb = h < 8 ? 8 : h;  // (h = 1: the group of 8 that holds d)
#pragma unroll 1
  for (int u = 0; u < 16; ++u) {
    const bool in = d / hb == 8 * u / hb;
    const uint32_t flip = h > 1 && (__popc((d >> 3) & u & (hb / 8 - 1)) & 1) ? 0x80008000u : 0u;
    *reinterpret_cast<uint4*>(dst + u * 2048 + n * 16) =
        in ? make_uint4(w[0] ^ flip, w[1] ^ flip, w[2] ^ flip, w[3] ^ flip) : make_uint4(0u, 0u, 0u, 0u);
  }
}

// ------------------------------------------------------------ kernel

template <int P, bool F16IN, bool BFM>
__global__ void __launch_bounds__(kThreads, 1) prefix_attn_kernel(const PrefixParams p) {
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
      mbar_init(&bars[kPFull + b], kSoftWarps / 2);
    }
    for (int b = 0; b < 16; ++b) mbar_init(&bars[kTurn + b], 1);
    for (int b = 0; b < kMetas; ++b) mbar_init(&bars[kMetaFull + b], 2);
    for (int b = 0; b < kSegs; ++b) {
      mbar_init(&bars[kSegFull + b], 1);
      mbar_init(&bars[kSegEmpty + b], kThreads / 32 - 1);
    }
    mbar_init(&bars[kQIn], kSoftWarps + 4);
    mbar_init(&bars[kQRot], 1);
    mbar_init(&bars[kQFull], kSoftWarps);
    mbar_init(&bars[kMmaDone], 1);
    mbar_fence_init();
  }
  if (warp == kWarpMma) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  pdl_wait_then_release();  // nothing above reads what another kernel writes
  bool failed = false;
  uint32_t it = 0;    // tiles of this CTA so far
  uint32_t segs = 0;  // and segments
  Segment* ring = reinterpret_cast<Segment*>(smem + kOffSeg);
  // the next announced segment, taken (every warp but the producer's)
  auto take = [&](Segment& s) {
    const int e = segs % kSegs;
    if (!wait_all(&bars[kSegFull + e], (segs / kSegs) & 1, failed)) return false;
    s = ring[e];
    __syncwarp();
    arrive_elect(&bars[kSegEmpty + e]);
    return s.more != 0;
  };

  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ---------------------------------------------------------- softmax
    const int par = warp >> 3;                      // tiles of this parity
    const int quart = warp >> 2;                    // columns 32 quart .. of q' and O
    const int r = 32 * (warp & 3) + lane;           // tensor-memory lane
    const int g = lane >> 2, c = lane & 3;
    const int r2 = 32 * (warp & 3) + 16 * (quart & 1) + g;  // lanes r2, r2 + 8 of this thread's scores
    // The block's rows lie 16 by 16 in the lane quarters (and so schedulers) in
    // turn: rows 16 b .. are the lanes 32 (b % 4) + 16 (b / 4) ...
    const int row = 16 * (warp & 3) + 64 * (lane >> 4) + (lane & 15);
    const int row2 = 16 * (warp & 3) + 64 * (quart & 1);  // first row of the 16 this warp scores
    const uint32_t tl = tmem + (uint32_t(32 * (warp & 3)) << 16);
    const uint32_t ts = tl + (uint32_t(16 * (quart & 1)) << 16);
    float* rowm = reinterpret_cast<float*>(smem + kOffM);
    uint64_t* turn = &bars[kTurn + 2 * (warp & 7)];  // [parity]: that tile's m is in rowm
    float* rowsum = reinterpret_cast<float*>(smem + kOffSum);
    float2* rowx = reinterpret_cast<float2*>(smem + kOffRow);
    bool agreed = false;  // on a failure, all four
    for (Segment sg; take(sg);) {
      // ---- q: this thread's quarter row into the A operand (V buffer 0)
      const bool live = row < sg.rows;
      {
        uint4 w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = make_uint4(0u, 0u, 0u, 0u);
        if (live) {
          const int sq = sg.seq0 + row / p.group, h = row % p.group;
          const uint4* src = reinterpret_cast<const uint4*>(
                                 p.q + (int64_t(sq) * p.num_q_heads + sg.kvh * p.group + h) * kHeadDim) + 4 * quart;
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = src[k];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(smem + kOffV + (4 * quart + k) * 2048 + r * 16) = w[k];
      }
      fence_async_smem();
      tc_fence_before();  // (the last segment's O has been read)
      __syncwarp();
      arrive_elect(&bars[kQIn]);
      // ---- the rotated row: softmax scale and 2^4, hi and lo parts
      wait_all(&bars[kQRot], segs & 1, failed);
      tc_fence_after();
      {
        const float f = (p.rotate_k ? p.c_h : 1.0f) * p.q_scale * 16.0f;
        float sum = 0.0f;
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          float x[16];
          tmem_ld16(tl + kColO + 32 * quart + 16 * k, x);
          uint32_t hw[8], lw[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            // (pairs 1 and 3 of each 8 columns carry 2^-4)
            const float y0 = clamp16(x[2 * j] * f), y1 = clamp16(x[2 * j + 1] * f);
            sum += (y0 + y1) * ((j & 1) ? 1.0f : 0.0625f);
            const __half h0 = __float2half_rn(y0), h1 = __float2half_rn(y1);
            hw[j] = uint32_t(__half_as_ushort(h0)) | (uint32_t(__half_as_ushort(h1)) << 16);
            lw[j] = pack_half2(y0 - __half2float(h0), y1 - __half2float(h1));
          }
          tmem_st8u(tl + kColQh + 16 * quart + 8 * k, hw);
          tmem_st8u(tl + kColQl + 16 * quart + 8 * k, lw);
        }
        tmem_wait_st();
        rowsum[quart * 128 + r] = sum;
      }
      ++segs;
      tc_fence_before();
      __syncwarp();
      arrive_elect(&bars[kQFull]);
      failed = !rows_sync(!failed);  // rowsum
      uint64_t qs[2];  // a row's sum(q'), twice
      float m[2];      // and reference
      float2 l[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) x += rowsum[k * 128 + r2 + 8 * i];
        qs[i] = twice(x);
        m[i] = 0.0f;
        l[i] = make_float2(0.0f, 0.0f);
      }

      const uint32_t first = it, end = it + sg.tiles;
      const uint32_t at_s = ts + 128 * par;
      const bool idle = row2 >= sg.rows;  // no row of this warp's: it only keeps the barriers' count
      for (it = first + ((first ^ par) & 1); it < end; it += 2) {
        if (idle) {
          wait_all(&bars[kSFull + par], (it >> 1) & 1, failed);
          arrive_elect(&turn[par]);
          arrive_elect(&bars[kPFull + par]);
          continue;
        }
        wait_all(&bars[kMetaFull + (it & (kMetas - 1))], (it / kMetas) & 1, failed);
        wait_all(&bars[kSFull + par], (it >> 1) & 1, failed);
        tc_fence_after();
        float s[64];  // [4 k + 2 i + column]: scores, minus m
        tmem_ld_16x256_issue(at_s, s);
        tmem_ld_16x256_issue(at_s + 64, s + 32);
        const uint8_t* meta = smem + kOffMeta + (it & (kMetas - 1)) * kMetaBytes;
        const float4* msz = reinterpret_cast<const float4*>(meta) + c;  // (s, s, z, z) of a key pair
        uint64_t nm[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) nm[i] = twice(-m[i]);
        tmem_wait_ld();
        pin32(s);
        pin32(s + 32);
        float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float4 sz = msz[4 * k];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float* v = &s[4 * k + 2 * i];
            score2(v[0], v[1], sz, qs[i], nm[i]);
            t4[2 * i + (k & 1)] = max3(t4[2 * i + (k & 1)], v[0], v[1]);
          }
        }
        const int okm = *reinterpret_cast<const int*>(meta + kKeys * 8);
        if (okm != 0xFF) {  // keys past the prefix or on a bad page
#pragma unroll
          for (int i = 0; i < 4; ++i) t4[i] = -INFINITY;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const bool in = (okm >> (k >> 1)) & 1;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float* v = &s[4 * k + 2 * i];
              v[0] = in ? v[0] : -INFINITY;
              v[1] = in ? v[1] : -INFINITY;
              t4[2 * i] = max3(t4[2 * i], v[0], v[1]);
            }
          }
        }
        float top[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[i] = fmaxf(t4[2 * i], t4[2 * i + 1]);
          top[i] = fmaxf(top[i], __shfl_xor_sync(kAll, top[i], 1));
          top[i] = fmaxf(top[i], __shfl_xor_sync(kAll, top[i], 2));
        }
        // ---- the reference: the other set may have moved it in the tile
        // before, and this tile moves it when its maximum outgrew it (the first
        // tile to its maximum).  Both are rare, so the scores above are taken
        // against the one known here, and shifted if it was not the last word.
        // In rowm -inf says that no key has counted yet (unreadable pages may
        // open a part); m is 0 then, and the row has neither l nor O.
        if (it > first) wait_all(&turn[par ^ 1], ((it - 1) >> 1) & 1, failed);
        float now[2];
        bool move = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          now[i] = it > first ? rowm[r2 + 8 * i] : -INFINITY;
          move = move || now[i] != m[i] || top[i] > kRefMost;
        }
        if (__any_sync(kAll, move)) {
          float f[2], sh[2];
          bool grow = it == first, any[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float at = m[i] + top[i];  // this tile's maximum
            const bool g1 = at > now[i] + kRefMost;
            const float to = g1 ? at - kRefBelow : now[i] > -INFINITY ? now[i] : 0.0f;
            // (nothing to scale yet: 1; the shift to a first reference below
            // -127 would be infinite, and 0 times it NaN)
            f[i] = now[i] > -INFINITY ? ex2(now[i] - to) : 1.0f;
            sh[i] = m[i] - to;
            const float fl = ex2(fminf(sh[i], 0.0f));
            l[i] = mul2(l[i], make_float2(fl, fl));
            m[i] = to;
            grow = grow || g1;
            any[i] = g1 || now[i] > -INFINITY;
          }
#pragma unroll
          for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              s[4 * k + 2 * i] += sh[i];
              s[4 * k + 2 * i + 1] += sh[i];
            }
          if (__any_sync(kAll, grow)) {
            if (it > first && wait_all(&bars[kPvDone + (par ^ 1)], ((it - 1) >> 1) & 1, failed)) {
              tc_fence_after();
#pragma unroll 1
              for (int q = 0; q < 8; ++q) {
                float o[8];
                tmem_ld_16x256_x2(ts + kColO + 16 * q, o);
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                  for (int j = 0; j < 4; ++j) o[4 * k + j] *= f[j >> 1];
                tmem_st_16x256_x2(ts + kColO + 16 * q, o);
              }
            }
            if (c == 0) {
#pragma unroll
              for (int i = 0; i < 2; ++i) rowm[r2 + 8 * i] = any[i] ? m[i] : -INFINITY;
            }
          }
        }
        __syncwarp();
        arrive_elect(&turn[par]);
#pragma unroll
        for (int kq = 0; kq < 2; ++kq) {
          uint32_t pw[16];
#pragma unroll
          for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float* v = &s[32 * kq + 4 * k + 2 * i];
              const float2 e = make_float2(ex2(v[0]), ex2(v[1]));
              l[i] = add2(l[i], e);
              pw[2 * k + i] = pack_half2(e.x, e.y);
            }
          tmem_st_16x128(at_s + 32 * kq, pw);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        arrive_elect(&bars[kPFull + par]);
      }
      it = end;
      // ---- the partial result, once the last P V has completed
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v = l[i].x + l[i].y;
        v += __shfl_xor_sync(kAll, v, 1);
        v += __shfl_xor_sync(kAll, v, 2);
        if (c == 0) rowx[par * 128 + r2 + 8 * i] = make_float2(m[i], v);
      }
      wait_all(&bars[kPvDone + ((it - 1) & 1)], ((it - 1) >> 1) & 1, failed);
      failed = !rows_sync(!failed);
      tc_fence_after();
      {
        float4* part = reinterpret_cast<float4*>(p.prefix.part) + prefix_part_index(sg.slot) + 8 * quart * 128 + row;
        float o[32];
        tmem_ld32_issue(tl + kColO + 32 * quart, o);
        tmem_wait_ld();
        pin32(o);
        if (live) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // columns of 8 dims: 0 4 1 5 2 6 3 7
            __stcg(part + 2 * k * 128, make_float4(o[8 * k], o[8 * k + 2], o[8 * k + 4], o[8 * k + 6]));
            __stcg(part + (2 * k + 1) * 128, make_float4(o[8 * k + 1], o[8 * k + 3], o[8 * k + 5], o[8 * k + 7]));
          }
        }
      }
      if (live && quart == 0) {
        // rowm is the reference that O refers to; nothing counted: m = -inf
        // (a q with a NaN never sets it, and its l, a NaN, goes on to the merge)
        const float2 x = rowx[r], y = rowx[128 + r];
        const float mm = rowm[r];
        const float ll = (x.y != 0.0f ? x.y * ex2(x.x - mm) : 0.0f) + (y.y != 0.0f ? y.y * ex2(y.x - mm) : 0.0f);
        __stcg(reinterpret_cast<float2*>(p.prefix.part_ml) + sg.slot * kPrefixRows + row,
               failed || ll == 0.0f ? make_float2(-INFINITY, 0.0f) : make_float2(mm, ll));
      }
      failed = !rows_sync(!failed);  // rowx has been read
      agreed = failed;
    }
    // One of the four warps that meet may have given up waiting for a segment
    // that another still got: those that end here without having agreed to
    // meet as often as the other does in that segment, so that it ends too.
    if (!agreed) {
#pragma unroll 1
      for (int i = 0; i < 3; ++i) (void)rows_sync(!failed);
    }
    if (failed && lane == 0) report(p.dev_status, SAW_ERR_DEVICE_TIMEOUT);
  } else {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFeedRegs));
  if (warp == kWarpProd) {
    // ---------------------------------------------------------- producer
    constexpr int kChunk = P * 68;
    constexpr int kPages = kKeys / P;               // pages per tile
    constexpr int kAhead = 32 / kPages;             // tiles whose page ids a warp holds
    Work work = plan_work(p, lane);
    const uint32_t chunk = work.chunk;
    for (bool more = true; more && !failed; ++segs) {
      Segment sg{};
      more = next_segment(p, work, sg, lane);
      sg.more = more;
      const int e = segs % kSegs;
      if (segs >= kSegs && !wait_parked(&bars[kSegEmpty + e], ((segs / kSegs) - 1) & 1, failed)) break;
      if (lane == 0) ring[e] = sg;
      __syncwarp();
      arrive_elect(&bars[kSegFull + e]);
      if (!more) break;
      // the pages' ids from the table row of the group's first sequence that
      // has the prefix and is served (the row of one that is idle or refused
      // for its length may hold anything; none: nothing to read)
      int reader = -1;
      for (int s0 = sg.first; s0 < sg.end && reader < 0; s0 += 32) {
        const int len = s0 + lane < sg.end ? p.seq_lens[s0 + lane] : 0;
        const uint32_t has = __ballot_sync(
            kAll, len >= sg.tokens && len <= p.max_seq_len && len - sg.tokens <= p.max_own_len);
        if (has) reader = s0 + __ffs(has) - 1;
      }
      const int32_t* btab = p.block_tables + int64_t(max(reader, 0)) * p.max_blocks;
      const int n_pages = reader < 0 ? 0 : sg.tokens / P;
      int ids = -1;
      for (int i = 0; i < sg.tiles; ++i, ++it) {
        const int st = it % kRawStages;
        if (i % kAhead == 0) {  // one page per lane
          const int lp = (sg.tile + i) * kPages + lane;
          ids = -1;
          if (lp < n_pages && lp < (sg.tile + sg.tiles) * kPages) {
            ids = btab[lp];
            if (ids < 0 || ids >= p.num_pages) {
              report(p.dev_status, SAW_ERR_DEVICE_INDEX);
              ids = -1;
            }
          }
        }
        // (lane g of the tile's pages says whether page g is there)
        const int id_l = __shfl_sync(kAll, ids, (i % kAhead) * kPages + (lane % kPages));
        const uint32_t have = __ballot_sync(kAll, id_l >= 0 && lane < kPages);
        if (it >= kRawStages && !wait_parked(&bars[kRawEmpty + st], ((it / kRawStages) - 1) & 1, failed)) break;
        const uint32_t raw = smem_u32(smem + kOffRaw + st * kRawBytes);
        const uint32_t bar = smem_u32(&bars[kRawFull + st]);
        if (lane == 0) {
          int okm = 0;
#pragma unroll
          for (int g = 0; g < kPages; ++g)
            if ((have >> g) & 1) okm |= ((1 << (P / 16)) - 1) << (g * (P / 16));
          raw_ok[st] = okm;
          if (!have) mbar_arrive(&bars[kRawFull + st]);
        }
        __syncwarp();
        // a page's chunk (codes and metadata) per copy, issued by one elected
        // lane of the converged warp: the copy takes uniform registers, and 32
        // lanes issuing their own cost 6000 cycles a tile
        if (have) {
          expect_tx_elect(bar, uint32_t(__popc(have)) * (2 * kChunk));
#pragma unroll
          for (int g = 0; g < kPages; ++g) {
            if (!((have >> g) & 1)) continue;
            const int id = __shfl_sync(kAll, id_l, g);
            const int64_t off = (int64_t(id) * p.num_kv_heads + sg.kvh) * kChunk;
            bulk_elect(raw + g * kChunk, p.k_cache + off, kChunk, bar);
            bulk_elect(raw + kRawV + g * kChunk, p.v_cache + off, kChunk, bar);
          }
        }
        __syncwarp();
      }
    }
    if (blockIdx.x == 0) publish_plan(p, chunk, lane);
  } else if (warp == kWarpMma) {
    // ---------------------------------------------------------- MMA issue
    constexpr uint32_t id_s = umma_idesc_f16(128, kKeys);
    constexpr uint32_t id_o = umma_idesc_f16(128, kHeadDim) | kUmmaBMnMajor;
    const uint32_t k0 = smem_u32(smem + kOffK), v0 = smem_u32(smem + kOffV);
    auto score = [&](uint32_t t) {  // S of tile t into buffer t & 1
      const int b = t & 1;
      if (!wait_all(&bars[kKFull + b], (t >> 1) & 1, failed)) return;
      tc_fence_after();
      const uint64_t bd = umma_desc(k0 + b * kOpBytes, 2048, 128);
      umma_ts8<(4096 >> 4)>(tmem + 128 * b, tmem + kColQh, bd, id_s, false);
      umma_ts8<(4096 >> 4)>(tmem + 128 * b, tmem + kColQl, bd, id_s, true);
      commit_elect(&bars[kSFull + b]);
      commit_elect(&bars[kKEmpty + b]);
    };
    // q' = q H^T in the input type
    constexpr uint32_t id_q = umma_idesc_f16(128, kHeadDim) | (F16IN ? 0u : (1u << 7) | (1u << 10));
    for (Segment sg; take(sg);) {
      if (!wait_all(&bars[kQIn], segs & 1, failed)) break;
      tc_fence_after();
      {
        const uint64_t ad = umma_desc(v0, 2048, 128), bd = umma_desc(v0 + kOpBytes, 2048, 128);
        umma_ss8<(4096 >> 4), (4096 >> 4)>(tmem + kColO, ad, bd, id_q, false);
        commit_elect(&bars[kQRot]);
      }
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
        umma_ts8<(256 >> 4)>(tmem + kColO, tmem + 128 * b, bd, id_o, i > 0);
        commit_elect(&bars[kPvDone + b]);
      }
    }
  } else {
    // ---------------------------------------------------------- expanders
    const bool is_v = warp < kWarpK;
    if (is_v) {
      write_hadamard<F16IN>(smem + kOffV + kOpBytes, tid - 32 * kWarpV, p.rotate_k ? p.block_h : 1);
      fence_async_smem();
      __syncwarp();
    }
    for (Segment sg; take(sg); ++segs) {
      if (is_v) {
        // the rotation matrix, once the last segment is done with the buffers
        // (the first one's was written before it was known)
        if (segs > 0) {
          if (!wait_parked(&bars[kPvDone + ((it - 1) & 1)], ((it - 1) >> 1) & 1, failed)) break;
          write_hadamard<F16IN>(smem + kOffV + kOpBytes, tid - 32 * kWarpV, p.rotate_k ? p.block_h : 1);
          fence_async_smem();
          __syncwarp();
        }
        arrive_elect(&bars[kQIn]);
        if (!wait_parked(&bars[kQFull], segs & 1, failed)) break;
      }
      for (int i = 0; i < sg.tiles; ++i, ++it) {
        const int st = it % kRawStages, b = it & 1;
        if (!wait_parked(&bars[kRawFull + st], (it / kRawStages) & 1, failed)) break;
        const uint8_t* raw = smem + kOffRaw + st * kRawBytes;
        const int okm = raw_ok[st];
        if (is_v) {
          const int n = tid - 32 * kWarpV;          // key of the tile
          const bool ok = (okm >> (n >> 4)) & 1;
          const uint8_t* chunk = raw + kRawV + (n / P) * (P * 68);
          const uint8_t* codes = chunk + (n % P) * 64;
          const uint32_t w = *reinterpret_cast<const uint32_t*>(chunk + P * 64 + 4 * (n % P));
          const float sf = meta_lo(w, BFM), zf = meta_hi(w, BFM);
          // every value below binary16's largest; bfloat16 words also exact in
          // it (eight significant bits: from 2^-17 up)
          bool plain = fmaf(15.0f, sf, fabsf(zf)) <= 65504.0f;
          if (BFM) plain = plain && (sf == 0.0f || sf >= 0x1p-17f) && (zf == 0.0f || fabsf(zf) >= 0x1p-17f);
          const __half2 s = __float2half2_rn(sf), z = __float2half2_rn(zf);
          if (it >= 2 && !wait_parked(&bars[kPvDone + b], ((it >> 1) - 1) & 1, failed)) break;
          uint8_t* dst = smem + kOffV + b * kOpBytes;
          if (__all_sync(kAll, plain && ok))
            expand_key<1>(codes, dst, n, [&](uint32_t x) { return dequant8(x, s, z); });
          else  // (a key past the prefix or on a bad page: zeros, whatever lies there)
            expand_key<1>(codes, dst, n, [&](uint32_t x) {
              return ok ? dequant8_wide(x, sf, zf) : make_uint4(0u, 0u, 0u, 0u);
            });
          fence_async_smem();
          __syncwarp();
          arrive_elect(&bars[kVFull + b]);
        } else {
          // K: codes as they are; scales and zeros for the softmax.  Meta slot
          // it % 4 was read for tile it - 4: its P was used by the P V that
          // precedes the scores of tile it - 2, whose end freed this K buffer.
          if (it >= 2 && !wait_parked(&bars[kKEmpty + b], ((it >> 1) - 1) & 1, failed)) break;
          uint8_t* meta = smem + kOffMeta + (it & (kMetas - 1)) * kMetaBytes;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int n = tid - 32 * kWarpK + 64 * u;
            const bool ok = (okm >> (n >> 4)) & 1;
            const uint8_t* chunk = raw + (n / P) * (P * 68);
            const uint32_t w = *reinterpret_cast<const uint32_t*>(chunk + P * 64 + 4 * (n % P));
            float* sz = reinterpret_cast<float*>(meta) + 4 * (n >> 1) + (n & 1);  // (s, s, z, z) of a key pair
            sz[0] = ok ? meta_lo(w, BFM) * 1048576.0f : 0.0f;  // 2^24 of the codes, 2^-4 of q'
            sz[2] = ok ? meta_hi(w, BFM) : 0.0f;
            // (codes of a key that does not count: any number, its score is masked)
            expand_key<4>(chunk + (n % P) * 64, smem + kOffK + b * kOpBytes, n, [](uint32_t x) { return codes8(x); });
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
  }
  if (failed && lane == 0) report(p.dev_status, SAW_ERR_DEVICE_TIMEOUT);
  if (warp == kWarpProd) {
    // the CTA must not exit while a copy into its shared memory is in flight
    for (uint32_t i = it > kRawStages ? it - kRawStages : 0; i < it; ++i)
      (void)mbar_wait_bounded(&bars[kRawFull + i % kRawStages], (i / kRawStages) & 1);
  } else if (warp == kWarpMma) {
    // every MMA has completed before tensor memory is released
    commit_elect(&bars[kMmaDone]);
    (void)mbar_wait_bounded(&bars[kMmaDone], 0);
  }
  __syncwarp();
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
  // the softmax warps' larger share is drawn from the launch's registers: with
  // fewer than kLaunchRegs a thread it would never be granted
  static const bool regs_ok = [&] {
    cudaFuncAttributes at{};
    return cudaFuncGetAttributes(&at, kernel) == cudaSuccess && at.numRegs == kLaunchRegs;
  }();
  if (!regs_ok) return cudaErrorLaunchOutOfResources;
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
