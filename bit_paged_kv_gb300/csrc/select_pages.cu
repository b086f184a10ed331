// select_pages.cu -- the pages that each kv-head's queries attend over: a
// score from the page's mean key (page_summary.cu), then the best of them.
//
// q' = (1/sqrt h) H q in binary32 by the append's butterfly; m_d = rint(q'_d /
// (max|q'| / 127)) are whole numbers.  With a summary's codes n, scale s and
// zero z, I = sum m n and J = sum m are exact whole numbers, and
//   score = max over the group's heads of RN(qs RN(RN(s I) + RN(z J))),
// qs = RN(max|q'| / 127): every step is exact or one rounding, so the lists are
// determined.  Ties go to the lower page.  The softmax scale and the part of
// the score that all pages share do not change the order.
//
// I on the tensor cores: 16 pages on M, the group's heads on N, dims on K, the
// codes masked in place into binary16 subnormals (n 2^-24, or n 2^-20 where m
// carries 2^-4), m as binary16.  |I| <= 127 15 D < 2^24 in units of 2^-24, so
// the binary32 sums are exact in any order.
//
// One CTA takes one (sequence, kv-head), or a cluster of them a run of its pages
// each; the pages' keys stay in shared memory.  A warp scores 32 pages at a time,
// the next 64's rows under way meanwhile.  The last entry of the list comes from one
// histogram of the scores between their extremes (radix digits of the keys would
// put nearly all of them in a few bins) and a ranking of the keys in its bin;
// where that bin holds too many (ties, far outliers), digit by digit.
//
// Bound: many pages, by the scoring, 26.8 us of 32.7 at 16 x 131072 tokens (10.6 at the
// measured copy rate): the latency of the rows' copies at the warps that fit, whose
// first stall is long_scoreboard, with issue at 38 % and DRAM at 2.0 TB/s; a page costs
// a kv-head three 32-byte sectors in two places.  Whole rows by bulk copies of 544 bytes,
// a cluster per sequence with its kv-heads' keys dealt to owners, took 136 us, two
// kv-heads to a CTA 44.  Choosing behind it is a chain of rounds: extremes, histogram,
// ranking, list; with few pages most of the time (1 x 32768 tokens 8.5 us, 3.7 of them
// the scoring; all keys to one CTA of the cluster, with fewer barriers, 9.5).  By digits:
// 13.0 and 42.4 us where scores are equal.
#include <algorithm>

#include <cooperative_groups.h>

#include "saw_device.cuh"
#include "saw_int4.h"
#include "saw_quant_row.cuh"

namespace saw {
namespace {

namespace cg = cooperative_groups;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kTile = 16;                            // pages per MMA
constexpr int kStrip = 32;                           // pages per warp and step: two MMA tiles
constexpr int kRing = 2;                             // strips under way per warp
constexpr int kCands = 128;                          // a CTA's keys in the threshold's bin
constexpr int kAllCands = 512;                       // the cluster's, ranked against one another
// Pages that a CTA takes before more join it, and more units than leave SMs idle.
// (1 x 32768 tokens 8.5 us, in clusters of four 10.3, of two 12.0.)  A cluster's
// barriers cost more than the SMs that it adds are worth soon: 16 x 32768, 128
// units, 12.4 us alone, in pairs 14.4, in fours 20.8; 8 x 131072, 64 units, in pairs
// 27.7, in fours 24.4, in eights 26.5.
constexpr int kAlone = 256;
// CTA shapes.  4 warps, eight per SM, for short lists, so that more units are under
// way (256 sequences of 62 to 256 pages 21.6 us, with 8 warps 25.8); 16 warps for few
// long ones (16 x 131072 tokens 33.0 us, with 8 warps 42); else 8 warps with what
// registers the units leave (32 x 65536, 256 units, two per SM 28.1 us, with the
// registers of three 37, of four 38.5; 64 x 16384, 512 units, 17.8, 14.1, 15.7).
constexpr int kSmall = 512, kLong = 1024;
constexpr int kMaxCtas = 8;                          // per cluster
constexpr int kMaxChunk = kSelectMaxPages / kMaxCtas;  // pages per CTA
static_assert(kMaxChunk % kStrip == 0, "whole strips");
constexpr int kMaxAlone = 16384;                     // pages of a 16-warp CTA
// a strip in shared memory: 32 rows of codes, then the 16 bytes that hold each
// row's word (copied past L1: 64 x 16384 tokens 15.8 us, by words through it 17.4)
__host__ __device__ constexpr int strip_bytes(int D) { return kStrip * (D / 2 + 16); }
__host__ __device__ constexpr int ring_bytes(int D, int warps) { return warps * kRing * strip_bytes(D); }

__device__ __forceinline__ void async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// The larger, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// Larger scores have larger keys; -0 counts as +0.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ float score_of(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Column h of a kv-head's queries by a warp: m into qh (the MMA's B fragments),
// qs and J; a column without a head has m = 0 and a NaN for qs, whose scores are
// passed over.
template <int D>
__device__ __forceinline__ void prepare_head(const SelectParams& p, int seq, int kvh, int h, int lane, __half* qh,
                                             float* qs_out, float* j_out) {
  constexpr int kE = D / 32;
  const int G = p.group;
  float x[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) x[e] = 0.0f;
  if (h < G) {
    const uint16_t* src = p.q + (int64_t(seq) * p.num_q_heads + kvh * G + h) * D + kE * lane;
#pragma unroll
    for (int e = 0; e < kE; e += 2) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(src + e);
      x[e] = in_lo(w, p.in_f16 != 0);
      x[e + 1] = in_hi(w, p.in_f16 != 0);
    }
    if (p.rotate_k) {
#pragma unroll
      for (int s = 1; s < kE; s <<= 1)
#pragma unroll
        for (int e = 0; e < kE; ++e)
          if (!(e & s)) {
            const float a = x[e], b = x[e + s];
            x[e] = __fadd_rn(a, b);
            x[e + s] = __fsub_rn(a, b);
          }
      for (int s = kE; s < p.block_h; s <<= 1) {
        const bool upper = (lane & (s / kE)) != 0;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const float o = __shfl_xor_sync(kAll, x[e], s / kE);
          x[e] = upper ? __fsub_rn(o, x[e]) : __fadd_rn(x[e], o);
        }
      }
#pragma unroll
      for (int e = 0; e < kE; ++e) x[e] = __fmul_rn(x[e], p.c_h);
    }
  }
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < kE; ++e) top = max_nan(top, fabsf(x[e]));
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) top = max_nan(top, __shfl_xor_sync(kAll, top, d));
  const float qs = __fdiv_rn(top, 127.0f);
  const float r = qs < 0x1p-126f ? 0.0f : __frcp_rn(qs);
  int sum = 0;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const int m = min(max(__float2int_rn(__fmul_rn(x[e], r)), -127), 127);
    sum += m;
    // element d: thread-in-group d / (D/4); of its 32-bit words of codes
    // word (d mod D/4) / 8, nibble j = d mod 8: byte j / 2, of bytes (0, 2) in
    // k-step 2 word, (1, 3) in 2 word + 1; odd nibbles are the high ones
    const int d = kE * lane + e, o = d % (D / 4), j = o & 7;
    const int t = 2 * (o >> 3) + ((j >> 1) & 1);
    qh[((t * 32 + h * 4 + d / (D / 4)) * 4) + (j & 1) * 2 + ((j >> 2) & 1)] =
        __float2half_rn(float(m) * ((j & 1) ? 0.0625f : 1.0f));
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
  if (lane == 0) {
    *qs_out = h < G ? qs : __uint_as_float(0x7FC00000u);
    *j_out = float(sum);
  }
}

// The scores of a strip of 32 pages for a kv-head, page `lane`'s in this lane:
// rows of codes `stride` bytes apart, their words `word_stride` apart.  b, qs, jj:
// this lane's part of the queries.
template <int D, bool BFM>
__device__ __forceinline__ float score_strip(const uint8_t* codes, int stride, const uint8_t* words, int word_stride,
                                             const uint32_t (&b)[D / 16][2], const float2& qs, const float2& jj,
                                             int lane) {
  constexpr int kW = D / 32;                         // words of a row per thread-in-group
  const int g = lane >> 2, c = lane & 3;
  float v[4];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    uint32_t x[kW], y[kW];                           // rows g and g + 8 of the tile
    const uint8_t* src = codes + (kTile * t + g) * stride + c * (D / 8);
    if constexpr (kW == 2) {
      const uint2 a = *reinterpret_cast<const uint2*>(src), e = *reinterpret_cast<const uint2*>(src + 8 * stride);
      x[0] = a.x; x[1] = a.y;
      y[0] = e.x; y[1] = e.y;
    } else {
#pragma unroll
      for (int k = 0; k < kW; k += 4) {
        const uint4 a = *reinterpret_cast<const uint4*>(src + 4 * k);
        const uint4 e = *reinterpret_cast<const uint4*>(src + 8 * stride + 4 * k);
        x[k] = a.x; x[k + 1] = a.y; x[k + 2] = a.z; x[k + 3] = a.w;
        y[k] = e.x; y[k + 1] = e.y; y[k + 2] = e.z; y[k + 3] = e.w;
      }
    }
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kW; ++k)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const uint32_t xx = hh ? x[k] >> 8 : x[k], yy = hh ? y[k] >> 8 : y[k];
        const uint32_t a[4] = {xx & 0x000F000Fu, yy & 0x000F000Fu, xx & 0x00F000F0u, yy & 0x00F000F0u};
        mma_16816(d, a, b[2 * k + hh][0], b[2 * k + hh][1]);
      }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t m = *reinterpret_cast<const uint32_t*>(words + (kTile * t + 8 * u + g) * word_stride);
      float s = meta_lo(m, BFM);
      const float z = meta_hi(m, BFM);
      // I = 2^24 d, exactly; a binary16 scale takes the factor as well.  (Scalar
      // steps: packed products and packed sums get fused by the assembler.)
      float i0 = d[2 * u], i1 = d[2 * u + 1];
      if constexpr (BFM) {
        i0 *= 0x1p24f;
        i1 *= 0x1p24f;
      } else {
        s *= 0x1p24f;
      }
      const float2 r = mul2(qs, make_float2(__fadd_rn(__fmul_rn(s, i0), __fmul_rn(z, jj.x)),
                                            __fadd_rn(__fmul_rn(s, i1), __fmul_rn(z, jj.y))));
      v[2 * t + u] = fmaxf(r.x, r.y);                // (fmaxf passes over a NaN)
    }
  }
  // over the thread-in-group: c is left with row g + 8 c
  const bool odd = c & 1, high = c & 2;
  const float a = fmaxf(odd ? v[1] : v[0], __shfl_xor_sync(kAll, odd ? v[0] : v[1], 1));
  const float e = fmaxf(odd ? v[3] : v[2], __shfl_xor_sync(kAll, odd ? v[2] : v[3], 1));
  float best = fmaxf(high ? e : a, __shfl_xor_sync(kAll, high ? a : e, 2));
  best = fmaxf(best, -INFINITY);
  // page g + 8 c of the strip is at lane 4 g + c
  return __shfl_sync(kAll, best, 4 * (lane & 7) + (lane >> 3));
}

struct Cand {
  uint32_t key;
  int32_t index;                                     // among the sequence's scored pages
};
template <int W>
struct Shared {
  static constexpr int kBins = W >= 8 ? 1024 : 512;
  alignas(16) uint32_t hist[kBins];
  alignas(8) float range[2];                         // this CTA's finite scores
  float qs[kMaxGroup], j[kMaxGroup];
  float least[W], most[W];                           // each warp's finite scores
  uint32_t above;                                    // this CTA's keys in larger bins
  uint32_t cands;
  Cand cand[kCands], all[W == 8 ? kAllCands : 1];    // (clusters are of 8 warps)
  uint32_t run[W], sum[W];                           // of the warps: entries of the list; scratch
  uint32_t listed[kMaxCtas];                         // of the cluster's CTAs: entries of the list
  uint32_t bin, want, key;
  int32_t index;
};

// Of nb bins the one that holds the wanted-th largest key, and how many are wanted
// of it; the bins are the sums over the cluster's histograms.
template <int W, class Count>
__device__ __forceinline__ void find_bin(Shared<W>& sh, int nb, uint32_t wanted, int tid, Count&& count_of) {
  const int warp = tid >> 5, lane = tid & 31;
  // this thread's bins: top, top - 1, ..  (16 warps: some threads have none of 256)
  const int per = (nb + 32 * W - 1) / (32 * W), top = nb - 1 - tid * per;
  uint32_t sum = 0;
  for (int j = 0; j < per && j <= top; ++j) sum += count_of(top - j);
  uint32_t above = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(kAll, above, d);
    if (lane >= d) above += o;
  }
  if (lane == 31) sh.sum[warp] = above;
  above -= sum;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) above += w < warp ? sh.sum[w] : 0u;
  if (above < wanted && wanted <= above + sum) {     // (one thread)
    for (int j = 0; j < per && j <= top; ++j) {
      const uint32_t v = count_of(top - j);
      if (wanted <= above + v) {
        sh.bin = uint32_t(top - j);
        sh.want = wanted - above;
        break;
      }
      above += v;
    }
  }
  __syncthreads();
}

template <int D, bool BFM, int W, int PER_SM>
__global__ void __launch_bounds__(32 * W, PER_SM) select_pages_kernel(const SelectParams p) {
  pdl_wait_then_release();
  constexpr int kThr = 32 * W, kBins = Shared<W>::kBins;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  auto sync_all = [&] {
    if (ctas > 1) cluster.sync();
    else __syncthreads();
  };
  constexpr int kKS = D / 16;                        // k-steps
  extern __shared__ __align__(16) uint8_t dyn[];     // each warp's ring, then keys [chunk]
  uint32_t* keys = reinterpret_cast<uint32_t*>(dyn + ring_bytes(D, W));
  __shared__ Shared<W> sh;
  __shared__ __align__(16) __half qh[kKS * 32 * 4];  // m in the B-fragment order
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = lane & 3;
  const int kvh = blockIdx.y, seq = blockIdx.z;
  const int hkv = p.num_kv_heads;
  int L = p.seq_lens[seq];
  if (L < 0 || L > p.max_seq_len) {
    if (rank == 0 && kvh == 0 && tid == 0) report(p.dev_status, SAW_ERR_DEVICE_INDEX);
    L = 0;
  }
  const int n = (L + p.page_size - 1) >> p.page_shift;
  const int take = p.max_selected;
  const int32_t* bt = p.block_tables + int64_t(seq) * p.max_blocks;
  const int64_t row = (int64_t(seq) * hkv + kvh) * take;
  int32_t* tables = p.sel_tables + row;
  int32_t* pages = p.sel_pages ? p.sel_pages + row : nullptr;
  auto put = [&](int at, int e) {
    tables[at] = e >= 0 ? bt[e] : -1;
    if (pages) pages[at] = e;
  };
  if (rank == 0 && tid == 0)
    p.sel_lens[int64_t(seq) * hkv + kvh] = n <= take ? L : take * p.page_size - (n * p.page_size - L);
  if (n <= take) {                                   // (the same in every CTA of the cluster)
    for (int i = rank * kThr + tid; i < take; i += ctas * kThr) put(i, i < n ? i : -1);
    return;
  }
  const int lo = p.first_pages, mid = n - p.last_pages - lo;  // by score: pages lo .. lo + mid - 1
  const int want = take - p.first_pages - p.last_pages;
  if (want == 0) {
    for (int i = rank * kThr + tid; i < take; i += ctas * kThr) put(i, i < lo ? i : n - take + i);
    return;
  }

  // ---- this CTA's run of the pages; its first strips' rows start here
  const int chunk = ((mid + ctas - 1) / ctas + kStrip - 1) / kStrip * kStrip;
  const int begin = min(rank * chunk, mid), count = min(mid - begin, chunk);
  const int32_t* run = bt + lo + begin;
  const int64_t stride = summary_stride(hkv, D);
  const uint8_t* codes = p.summary + kvh * (D / 2);
  const uint8_t* words = p.summary + hkv * (D / 2) + (4 * kvh & ~15);
  uint8_t* ring = dyn + warp * (kRing * strip_bytes(D));
  constexpr int kStep = W * kStrip;
  // this lane's page of the strip at i0 (-1: none, or bad)
  auto page_of = [&](int i0) { return i0 + lane < count ? run[i0 + lane] : -1; };
  // Starts the copies of a strip's rows; a page that is not there has the first
  // one that is.  Returns whether this lane's is.
  auto issue = [&](int id, int stage) {
    const bool ok = uint32_t(id) < uint32_t(p.num_pages);
    const uint32_t there = __ballot_sync(kAll, ok);
    if (there != 0) {
      const int any = __shfl_sync(kAll, id, __ffs(int(there)) - 1);
      if (!ok) id = any;
      uint8_t* dst = ring + stage * strip_bytes(D);
      constexpr int kParts = D / 32;                 // 16-byte parts of a row
#pragma unroll
      for (int u = 0; u < kParts; ++u) {
        const int at = 32 * u + lane;                // of the strip's parts
        const int64_t off = __shfl_sync(kAll, id, at / kParts) * stride;
        async16(dst + 16 * at, codes + off + 16 * (at % kParts));
      }
      async16(dst + kStrip * (D / 2) + 16 * lane, words + id * stride);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return ok;
  };
  bool ok0 = issue(page_of(warp * kStrip), 0), ok1 = issue(page_of(warp * kStrip + kStep), 1);
  int next = page_of(warp * kStrip + 2 * kStep);

  // (meanwhile) what is always listed
  for (int i = rank * kThr + tid; i < take - want; i += ctas * kThr)
    if (i < lo) put(i, i);
    else put(want + i, n - p.last_pages + i - lo);

  // ---- m, qs and J of the group's heads
  for (int h = warp; h < kMaxGroup; h += W) prepare_head<D>(p, seq, kvh, h, lane, qh, &sh.qs[h], &sh.j[h]);
  for (int i = tid; i < kBins; i += kThr) sh.hist[i] = 0;
  if (tid == 0) sh.cands = 0;
  __syncthreads();
  uint32_t b[kKS][2];
#pragma unroll
  for (int t = 0; t < kKS; ++t) {
    const uint2 v = reinterpret_cast<const uint2*>(qh)[t * 32 + lane];
    b[t][0] = v.x;
    b[t][1] = v.y;
  }
  const float2 qs = make_float2(sh.qs[2 * c], sh.qs[2 * c + 1]), jj = make_float2(sh.j[2 * c], sh.j[2 * c + 1]);

  // ---- keys
  bool bad = false;
  float least = INFINITY, most = -INFINITY;
  for (int i0 = warp * kStrip, stage = 0; i0 < count; i0 += kStep, stage ^= 1) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
    __syncwarp();
    const uint8_t* st = ring + stage * strip_bytes(D);
    float best = score_strip<D, BFM>(st, D / 2, st + kStrip * (D / 2) + (4 * kvh & 15), 16, b, qs, jj, lane);
    if (!ok0) best = -INFINITY;
    const int i = i0 + lane;
    if (i < count) {
      bad = bad || !ok0;
      keys[i] = key_of(best);
      if (fabsf(best) < INFINITY) {
        least = fminf(least, best);
        most = fmaxf(most, best);
      }
    }
    ok0 = ok1;
    __syncwarp();                                    // the strip is read: its place takes the next but one
    ok1 = issue(next, stage);
    next = page_of(i0 + 3 * kStep);
  }
  if (bad) report(p.dev_status, SAW_ERR_DEVICE_INDEX);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    least = fminf(least, __shfl_xor_sync(kAll, least, d));
    most = fmaxf(most, __shfl_xor_sync(kAll, most, d));
  }
  if (lane == 0) {
    sh.least[warp] = least;
    sh.most[warp] = most;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) {
    least = fminf(least, sh.least[w]);
    most = fmaxf(most, sh.most[w]);
  }
  if (ctas > 1) {
    if (tid == 0) {
      sh.range[0] = least;
      sh.range[1] = most;
    }
    cluster.sync();
    // (here and below: every CTA's word under way before the first is used)
    float2 o[kMaxCtas];
#pragma unroll
    for (int r = 0; r < kMaxCtas; ++r) o[r] = *reinterpret_cast<const float2*>(cluster.map_shared_rank(sh.range, min(r, ctas - 1)));
#pragma unroll
    for (int r = 0; r < kMaxCtas; ++r) {
      least = fminf(least, o[r].x);
      most = fmaxf(most, o[r].y);
    }
  }

  // ---- the last entry of the list by (key, lower page): sh.key and sh.index; and
  // the entries of each warp's run and of each CTA
  const int part = ((count + W - 1) / W + 31) / 32 * 32;  // a warp's run
  const int w0 = min(warp * part, count), w1 = min(w0 + part, count);
  const float scale = float(kBins - 1) / (most - least);
  bool done = false;
  if (most > least && most - least < INFINITY && scale < INFINITY) {  // (not: one value, or none that is finite)
    // A score's bin grows with the score: a difference and a product, each rounded
    // monotonously.
    auto bin_of = [&](uint32_t key) {
      return min(__float2int_rz(fmaxf(__fmul_rn(__fsub_rn(score_of(key), least), scale), 0.0f)), kBins - 1);
    };
#pragma unroll 4
    for (int i = tid; i < count; i += kThr) atomicAdd(&sh.hist[bin_of(keys[i])], 1u);
    sync_all();
    if (ctas == 1) {
      find_bin<W>(sh, kBins, uint32_t(want), tid, [&](int i) { return sh.hist[i]; });
    } else {
      // (a thread's bins, the sum over the cluster)
      constexpr int kPer = kBins / kThr;
      uint32_t v[kPer] = {};
      if constexpr (kPer == 4) {
        uint4 o[kMaxCtas];
#pragma unroll
        for (int r = 0; r < kMaxCtas; ++r)
          o[r] = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(sh.hist, min(r, ctas - 1)) + kBins - kPer * (tid + 1));
#pragma unroll
        for (int r = 0; r < kMaxCtas; ++r) {
          const uint32_t in = r < ctas ? 0xFFFFFFFFu : 0u;
          v[0] += o[r].x & in;
          v[1] += o[r].y & in;
          v[2] += o[r].z & in;
          v[3] += o[r].w & in;
        }
      }
      const int top = kBins - 1 - tid * kPer;
      find_bin<W>(sh, kBins, uint32_t(want), tid, [&](int i) {
        uint32_t x = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) x = top - i == j ? v[kPer - 1 - j] : x;
        return x;
      });
    }
    const int bin = int(sh.bin);
    const uint32_t need = sh.want;
    uint32_t above = 0;
#pragma unroll 2
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t k = i < w1 ? keys[i] : 0u;
      const int at = i < w1 ? bin_of(k) : -1;
      above += __popc(__ballot_sync(kAll, at > bin));
      if (at == bin) {
        const uint32_t x = atomicAdd(&sh.cands, 1u);
        if (x < kCands) sh.cand[x] = Cand{k, begin + i};
      }
    }
    if (lane == 0) sh.run[warp] = above;
    __syncthreads();
    uint32_t m = 0;
    bool fits = true;
    if (ctas == 1) {
      m = sh.cands;
      fits = m <= kCands;
    } else {
      if (tid == 0) {
        uint32_t x = 0;
        for (int w = 0; w < W; ++w) x += sh.run[w];
        sh.above = x;
      }
      cluster.sync();
      // warp r takes CTA r's candidates
      uint32_t cnt[kMaxCtas];
#pragma unroll
      for (int r = 0; r < kMaxCtas; ++r) cnt[r] = *cluster.map_shared_rank(&sh.cands, min(r, ctas - 1));
      if (tid < ctas) sh.listed[tid] = *cluster.map_shared_rank(&sh.above, tid);
      uint32_t at = 0, mine = 0;
#pragma unroll
      for (int r = 0; r < kMaxCtas; ++r) {
        if (r >= ctas) cnt[r] = 0;
        fits = fits && cnt[r] <= kCands;
        if (r == warp) {
          at = m;
          mine = cnt[r];
        }
        m += cnt[r];
      }
      fits = fits && m <= kAllCands;
      static_assert(W != 8 || W == kMaxCtas, "a warp per CTA of the cluster");
      if (fits && mine > 0) {
        const Cand* o = cluster.map_shared_rank(sh.cand, warp);
        for (uint32_t i = lane; i < mine; i += 32) sh.all[at + i] = o[i];
      }
      __syncthreads();
    }
    done = fits;                                     // (the same in every CTA)
    if (done) {
      const Cand* from = ctas == 1 ? sh.cand : sh.all;
      for (uint32_t x = tid; x < m; x += kThr) {
        const Cand a = from[x];
        uint32_t before = 0;
#pragma unroll 4
        for (uint32_t y = 0; y < m; ++y) {
          const Cand o = from[y];
          before += o.key > a.key || (o.key == a.key && o.index < a.index);
        }
        if (before < need) {
          if (ctas > 1) atomicAdd(&sh.listed[a.index / chunk], 1u);
          if (a.index >= begin && a.index < begin + count) atomicAdd(&sh.run[(a.index - begin) / part], 1u);
        }
        if (before == need - 1) {
          sh.key = a.key;
          sh.index = a.index;
        }
      }
      __syncthreads();
    }
  }
  if (!done) {
    // digit by digit
    uint32_t prefix = 0, mask = 0, need = uint32_t(want);
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      sync_all();                                    // the cluster is past its reads of the histograms
      for (int i = tid; i < 256; i += kThr) sh.hist[i] = 0;
      __syncthreads();
      for (int i0 = 32 * warp; i0 < count; i0 += kThr) {
        const uint32_t k = i0 + lane < count ? keys[i0 + lane] : 0u;
        const bool in = i0 + lane < count && (k & mask) == prefix;
        // one count per digit and warp: equal keys would queue up
        const uint32_t digit = in ? (k >> shift) & 255u : 256u;
        const uint32_t same = __match_any_sync(kAll, digit);
        if (in && lane == __ffs(int(same)) - 1) atomicAdd(&sh.hist[digit], uint32_t(__popc(same)));
      }
      sync_all();
      find_bin<W>(sh, 256, need, tid, [&](int i) {
        uint32_t x = 0;
        for (int r = 0; r < ctas; ++r) x += cluster.map_shared_rank(sh.hist, r)[i];
        return x;
      });
      prefix |= sh.bin << shift;
      mask |= 255u << shift;
      need = sh.want;
    }
    // the need-th of the keys equal to it, then the entries
    uint32_t eq = 0, gt = 0;
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const uint32_t k = i0 + lane < w1 ? keys[i0 + lane] : 0u;
      gt += __popc(__ballot_sync(kAll, i0 + lane < w1 && k > prefix));
      eq += __popc(__ballot_sync(kAll, i0 + lane < w1 && k == prefix));
    }
    __syncthreads();
    if (lane == 0) {
      sh.run[warp] = gt;
      sh.sum[warp] = eq;
    }
    if (tid == 0) {
      sh.key = prefix;
      sh.index = -1;
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t x = 0, y = 0;
      for (int w = 0; w < W; ++w) {
        x += sh.run[w];
        y += sh.sum[w];
      }
      sh.above = x;
      sh.cands = y;                                  // (this CTA's equal ones)
    }
    sync_all();
    uint32_t before = 0, left = need;
    for (int r = 0; r < ctas; ++r) {
      const uint32_t x = *cluster.map_shared_rank(&sh.above, r), y = *cluster.map_shared_rank(&sh.cands, r);
      if (tid == r) sh.listed[r] = x + min(y, left);
      if (r < rank) before += y;
      left -= min(y, left);
    }
    for (int w = 0; w < warp; ++w) before += sh.sum[w];
    const uint32_t taken = min(need > before ? need - before : 0u, eq);  // of this warp's equal ones
    if (lane == 0) sh.run[warp] += taken;
    // this CTA's last equal entry: its equal pages up to there are listed
    uint32_t seen = 0;
    for (int i0 = w0; taken > 0 && i0 < w1; i0 += 32) {
      const bool is = i0 + lane < w1 && keys[i0 + lane] == prefix;
      const uint32_t all = __ballot_sync(kAll, is);
      if (is && seen + __popc(all & ((2u << lane) - 1u)) == taken) atomicMax(&sh.index, begin + i0 + lane);
      seen += __popc(all);
    }
    __syncthreads();
  }

  // ---- the list.  (A CTA's memory stays until the cluster has read it.)
  if (ctas > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const uint32_t last = sh.key;
  const int last_at = sh.index - begin;
  uint32_t at = 0;
  if (ctas > 1)
#pragma unroll
    for (int r = 0; r < kMaxCtas; ++r) at += r < rank ? sh.listed[r] : 0u;
  for (int w = 0; w < warp; ++w) at += sh.run[w];
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < w1 ? keys[i] : 0u;
    const bool in = i < w1 && (k > last || (k == last && i <= last_at));
    const uint32_t all = __ballot_sync(kAll, in);
    if (in) put(lo + int(at) + __popc(all & ((1u << lane) - 1u)), lo + begin + i);
    at += __popc(all);
  }
  __syncwarp();
  if (ctas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int D, bool BFM, int W, int PER_SM>
cudaError_t launch_select_w(const SelectParams& p, int ctas, cudaStream_t stream) {
  const int max_pages = std::max((p.max_seq_len + p.page_size - 1) / p.page_size, 1);
  const int chunk = ((max_pages + ctas - 1) / ctas + kStrip - 1) / kStrip * kStrip;
  auto kernel = select_pages_kernel<D, BFM, W, PER_SM>;
  // (the most that any call needs, so that no thread lowers another's)
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               ring_bytes(D, W) + (W == 16 ? kMaxAlone : kMaxChunk) * 4);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas), unsigned(p.num_kv_heads), unsigned(p.num_seqs));
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = size_t(ring_bytes(D, W) + chunk * 4);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(ctas);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, bool BFM>
cudaError_t launch_select(const SelectParams& p, int sms, cudaStream_t stream) {
  const int max_pages = (p.max_seq_len + p.page_size - 1) / p.page_size;
  const int64_t units = int64_t(p.num_seqs) * p.num_kv_heads;
  constexpr int kWide = D == 256 ? 2 : 1;            // (its rows and queries take twice the registers)
  if (units > 2 * int64_t(sms) && max_pages <= kSmall) return launch_select_w<D, BFM, 4, 8 / kWide>(p, 1, stream);
  int ctas = 1;
  while (ctas < kMaxCtas && (ctas == 1 ? 3 * units <= 2 * int64_t(sms) : units * ctas <= sms) && max_pages > ctas * kAlone)
    ctas *= 2;
  while (max_pages > ctas * kMaxChunk) ctas *= 2;
  if (ctas == 1 && units <= sms && max_pages > kLong && max_pages <= kMaxAlone)
    return launch_select_w<D, BFM, 16, 1>(p, 1, stream);
  if (units * ctas <= 2 * int64_t(sms)) return launch_select_w<D, BFM, 8, 2>(p, ctas, stream);
  return launch_select_w<D, BFM, 8, kWide == 2 ? 2 : 3>(p, ctas, stream);
}

}  // namespace

cudaError_t launch_select_pages(const SelectParams& p, int sms, cudaStream_t stream) {
  switch (p.head_dim) {
    case 64: return p.meta_bf16 ? launch_select<64, true>(p, sms, stream) : launch_select<64, false>(p, sms, stream);
    case 128: return p.meta_bf16 ? launch_select<128, true>(p, sms, stream) : launch_select<128, false>(p, sms, stream);
    case 256: return p.meta_bf16 ? launch_select<256, true>(p, sms, stream) : launch_select<256, false>(p, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace saw
