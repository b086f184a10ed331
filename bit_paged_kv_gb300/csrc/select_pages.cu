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
// the next 64's rows under way meanwhile.  The threshold comes from one
// histogram of the scores between their extremes (radix digits of the keys would
// put nearly all of them in a few bins) and a ranking of the keys in its bin;
// where that bin holds too many (ties, far outliers), digit by digit.
#include <cooperative_groups.h>

#include "saw_device.cuh"
#include "saw_int4.h"
#include "saw_quant_row.cuh"

namespace saw {
namespace {

namespace cg = cooperative_groups;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int ctas_per_sm(int D) { return D == 256 ? 2 : 4; }
constexpr int kAlone = 512;                          // pages that a CTA takes before more join it
constexpr int kBins = 1024;
constexpr int kCands = 256;                          // keys ranked against one another
constexpr int kTile = 16;                            // pages per MMA
constexpr int kStrip = 32;                           // pages per warp and step: two MMA tiles
constexpr int kMaxChunk = kSelectMaxPages / 8;       // pages per CTA
static_assert(kMaxChunk % kStrip == 0, "whole strips");
constexpr int kRing = 2;                             // strips under way per warp
// a strip in shared memory: 32 rows of codes, 32 words
__host__ __device__ constexpr int strip_bytes(int D) { return kStrip * (D / 2 + 4); }
__host__ __device__ constexpr int ring_bytes(int D) { return kWarps * kRing * strip_bytes(D); }

__device__ __forceinline__ void async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
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

struct Shared {
  alignas(16) uint32_t hist[kBins];                  // (read four bins at a time)
  float qs[kMaxGroup], j[kMaxGroup];
  float least[kWarps], most[kWarps];                 // each warp's finite scores
  float range[2];                                    // this CTA's
  uint32_t cands, cand[kCands];                      // this CTA's keys in the threshold's bin
  uint32_t all[kCands];                              // the cluster's
  uint32_t count[2];                                 // this CTA's keys above the threshold, and equal to it
  uint32_t warp_count[kWarps][2];
  uint32_t bin, want, key;
};

// Thread t's share of a histogram's bins, largest first: the bin that holds the
// want-th largest key, and how many are wanted of that bin.  v: its N bins.
template <int N>
__device__ __forceinline__ void find_bin(Shared& sh, const uint32_t (&v)[N], uint32_t want, int tid) {
  const int warp = tid >> 5, lane = tid & 31;
  uint32_t sum = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) sum += v[j];
  uint32_t above = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(kAll, above, d);
    if (lane >= d) above += o;
  }
  if (lane == 31) sh.warp_count[warp][0] = above;
  above -= sum;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) above += w < warp ? sh.warp_count[w][0] : 0u;
  if (above < want && want <= above + sum) {         // (one thread)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (above < want && want <= above + v[j]) {
        sh.bin = uint32_t(kThreads * N - 1 - N * tid - j);
        sh.want = want - above;
      }
      above += v[j];
    }
  }
  __syncthreads();
}

template <int D, bool BFM>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D))
    select_pages_kernel(const SelectParams p, int chunk) {
  pdl_wait_then_release();
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  auto sync_all = [&] {
    if (ctas > 1) cluster.sync();
    else __syncthreads();
  };
  constexpr int kKS = D / 16;                        // k-steps
  constexpr int kE = D / 32;
  constexpr int kW = D / 32;                         // words of a row per thread-in-group
  extern __shared__ __align__(16) uint8_t dyn[];     // each warp's ring, then keys [chunk]
  uint32_t* keys = reinterpret_cast<uint32_t*>(dyn + ring_bytes(D));
  __shared__ Shared sh;
  __shared__ __align__(16) __half qh[kKS * 32 * 4];  // m in the B-fragment order
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int kvh = blockIdx.y, seq = blockIdx.z;
  const int hkv = p.num_kv_heads, G = p.group;
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
    for (int i = rank * kThreads + tid; i < take; i += ctas * kThreads) put(i, i < n ? i : -1);
    return;
  }
  const int lo = p.first_pages, mid = n - p.last_pages - lo;  // by score: pages lo .. lo + mid - 1
  const int want = take - p.first_pages - p.last_pages;
  for (int i = rank * kThreads + tid; i < take - want; i += ctas * kThreads)
    if (i < lo) put(i, i);
    else put(want + i, n - p.last_pages + i - lo);
  if (want == 0) return;

  // ---- this CTA's run of the pages; its first strips' rows start here
  const int begin = min(rank * chunk, mid), count = min(mid - begin, chunk);
  const int32_t* run = bt + lo + begin;
  const int64_t stride = summary_stride(hkv, D);
  const uint8_t* codes = p.summary + kvh * (D / 2);
  const uint8_t* words = p.summary + hkv * (D / 2) + 4 * kvh;
  uint8_t* ring = dyn + warp * (kRing * strip_bytes(D));
  constexpr int kStep = kWarps * kStrip;
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
      async4(dst + kStrip * (D / 2) + 4 * lane, words + id * stride);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return ok;
  };
  bool ok0 = issue(page_of(warp * kStrip), 0), ok1 = issue(page_of(warp * kStrip + kStep), 1);
  int next = page_of(warp * kStrip + 2 * kStep);

  // ---- m, qs and J of the group's heads
  for (int h = warp; h < kMaxGroup; h += kWarps) {
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
      sh.qs[h] = h < G ? qs : __uint_as_float(0x7FC00000u);  // (a NaN's scores are passed over)
      sh.j[h] = float(sum);
    }
  }
  for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
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
  auto score = [&](int i0, int stage, bool ok) {
    const uint8_t* st = ring + stage * strip_bytes(D);
    float v[4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t x[kW], y[kW];                         // rows g and g + 8 of the tile
      const uint8_t* src = st + (kTile * t + g) * (D / 2) + c * (D / 8);
      if constexpr (kW == 2) {
        const uint2 a = *reinterpret_cast<const uint2*>(src), e = *reinterpret_cast<const uint2*>(src + 8 * (D / 2));
        x[0] = a.x; x[1] = a.y;
        y[0] = e.x; y[1] = e.y;
      } else {
#pragma unroll
        for (int k = 0; k < kW; k += 4) {
          const uint4 a = *reinterpret_cast<const uint4*>(src + 4 * k);
          const uint4 e = *reinterpret_cast<const uint4*>(src + 8 * (D / 2) + 4 * k);
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
        const uint32_t m = reinterpret_cast<const uint32_t*>(st + kStrip * (D / 2))[kTile * t + 8 * u + g];
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
        const float2 x = mul2(qs, make_float2(__fadd_rn(__fmul_rn(s, i0), __fmul_rn(z, jj.x)),
                                              __fadd_rn(__fmul_rn(s, i1), __fmul_rn(z, jj.y))));
        v[2 * t + u] = fmaxf(x.x, x.y);              // (fmaxf passes over a NaN)
      }
    }
    // over the thread-in-group: c is left with row g + 8 c
    const bool odd = c & 1, high = c & 2;
    const float a = fmaxf(odd ? v[1] : v[0], __shfl_xor_sync(kAll, odd ? v[0] : v[1], 1));
    const float e = fmaxf(odd ? v[3] : v[2], __shfl_xor_sync(kAll, odd ? v[2] : v[3], 1));
    float best = fmaxf(high ? e : a, __shfl_xor_sync(kAll, high ? a : e, 2));
    best = fmaxf(best, -INFINITY);
    // lane's own page's score (lane = g + 8 c of the strip is at lane 4 g + c)
    best = __shfl_sync(kAll, best, 4 * (lane & 7) + (lane >> 3));
    if (!ok) best = -INFINITY;
    const int i = i0 + lane;
    if (i < count) {
      bad = bad || !ok;
      keys[i] = key_of(best);
      if (fabsf(best) < INFINITY) {
        least = fminf(least, best);
        most = fmaxf(most, best);
      }
    }
  };
  for (int i0 = warp * kStrip, stage = 0; i0 < count; i0 += kStep, stage ^= 1) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
    __syncwarp();
    score(i0, stage, ok0);
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
  for (int w = 0; w < kWarps; ++w) {
    least = fminf(least, sh.least[w]);
    most = fmaxf(most, sh.most[w]);
  }
  if (ctas > 1) {
    if (tid == 0) {
      sh.range[0] = least;
      sh.range[1] = most;
    }
    cluster.sync();
    for (int r = 0; r < ctas; ++r) {
      const float* o = cluster.map_shared_rank(sh.range, r);
      least = fminf(least, o[0]);
      most = fmaxf(most, o[1]);
    }
  }

  // ---- the threshold: the want-th largest key of the cluster.  A score's bin
  // grows with the score: a difference and a product, each rounded monotonously.
  const float scale = float(kBins - 1) / (most - least);
  bool done = false;
  uint32_t prefix = 0, need = uint32_t(want);
  if (most - least < INFINITY && scale < INFINITY) {  // (not: one value, or none that is finite)
    auto bin_of = [&](uint32_t key) {
      return min(__float2int_rz(fmaxf(__fmul_rn(__fsub_rn(score_of(key), least), scale), 0.0f)), kBins - 1);
    };
    for (int i = tid; i < count; i += kThreads) atomicAdd(&sh.hist[bin_of(keys[i])], 1u);
    sync_all();
    constexpr int kPer = kBins / kThreads;
    uint32_t v[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = 0;
    for (int r = 0; r < ctas; ++r) {
      const uint4 h = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(sh.hist, r) + kBins - kPer * (tid + 1));
      static_assert(kPer == 4, "a thread's bins in one load");
      v[0] += h.w; v[1] += h.z; v[2] += h.y; v[3] += h.x;
    }
    find_bin(sh, v, need, tid);
    const int bin = int(sh.bin);
    need = sh.want;
    for (int i = tid; i < count; i += kThreads) {
      const uint32_t k = keys[i];
      if (bin_of(k) == bin) {
        const uint32_t at = atomicAdd(&sh.cands, 1u);
        if (at < kCands) sh.cand[at] = k;
      }
    }
    sync_all();
    uint32_t n_all = 0;
    for (int r = 0; r < ctas; ++r) {
      const uint32_t m = *cluster.map_shared_rank(&sh.cands, r);
      const uint32_t* o = cluster.map_shared_rank(sh.cand, r);
      for (uint32_t i = tid; i < m && n_all + i < kCands; i += kThreads) sh.all[n_all + i] = o[i];
      n_all += m;
    }
    __syncthreads();
    done = n_all <= kCands;
    if (done) {
      if (tid < int(n_all)) {
        const uint32_t k = sh.all[tid];
        uint32_t gt = 0, eq = 0;
        for (uint32_t i = 0; i < n_all; ++i) {
          gt += sh.all[i] > k;
          eq += sh.all[i] == k;
        }
        if (gt < need && need <= gt + eq) {          // (equal keys write the same)
          sh.key = k;
          sh.want = need - gt;
        }
      }
      __syncthreads();
      prefix = sh.key;
      need = sh.want;
    } else {
      need = uint32_t(want);
    }
  }
  if (!done) {
    // (every CTA of the cluster is past its reads of the others' histograms)
    uint32_t mask = 0;
    for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
    __syncthreads();
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      static_assert(kBins == 4 * 256 && kThreads == 256, "a histogram per pass, a bin per thread");
      uint32_t* hist = sh.hist + 256 * pass;
      for (int i0 = 0; i0 < count; i0 += kThreads) {
        const uint32_t k = i0 + tid < count ? keys[i0 + tid] : 0u;
        const bool in = i0 + tid < count && (k & mask) == prefix;
        // one count per digit and warp: equal keys would queue up
        const uint32_t digit = in ? (k >> shift) & 255u : 256u;
        const uint32_t same = __match_any_sync(kAll, digit);
        if (in && lane == __ffs(int(same)) - 1) atomicAdd(&hist[digit], uint32_t(__popc(same)));
      }
      sync_all();
      uint32_t v[1] = {0};
      for (int r = 0; r < ctas; ++r) v[0] += cluster.map_shared_rank(hist, r)[255 - tid];
      find_bin(sh, v, need, tid);
      prefix |= sh.bin << shift;
      mask |= 255u << shift;
      need = sh.want;
      __syncthreads();
    }
  }

  // ---- the list: keys above the threshold, and `need` of those equal to it,
  // the lower pages first
  const int part = ((count + kWarps - 1) / kWarps + 31) / 32 * 32;  // a warp's run
  const int w0 = min(warp * part, count), w1 = min(w0 + part, count);
  uint32_t gt = 0, eq = 0;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const uint32_t k = i0 + lane < w1 ? keys[i0 + lane] : 0u;
    gt += __popc(__ballot_sync(kAll, k > prefix));
    eq += __popc(__ballot_sync(kAll, i0 + lane < w1 && k == prefix));
  }
  if (lane == 0) {
    sh.warp_count[warp][0] = gt;
    sh.warp_count[warp][1] = eq;
  }
  __syncthreads();
  if (tid < 2) {
    uint32_t s = 0;
    for (int w = 0; w < kWarps; ++w) s += sh.warp_count[w][tid];
    sh.count[tid] = s;
  }
  gt = eq = 0;
  if (ctas > 1) {
    cluster.sync();
    for (int r = 0; r < rank; ++r) {
      const uint32_t* o = cluster.map_shared_rank(sh.count, r);
      gt += o[0];
      eq += o[1];
    }
  }
  for (int w = 0; w < warp; ++w) {
    gt += sh.warp_count[w][0];
    eq += sh.warp_count[w][1];
  }
  if (ctas > 1) cluster.sync();  // no CTA ends while another reads its memory
  const uint32_t below = (1u << lane) - 1u;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const uint32_t k = i0 + lane < w1 ? keys[i0 + lane] : 0u;
    const bool is_eq = i0 + lane < w1 && k == prefix;
    const uint32_t bg = __ballot_sync(kAll, k > prefix), be = __ballot_sync(kAll, is_eq);
    const uint32_t g0 = gt + __popc(bg & below), e0 = eq + __popc(be & below);
    if (k > prefix || (is_eq && e0 < need)) put(lo + int(g0 + min(e0, need)), lo + begin + i0 + lane);
    gt += __popc(bg);
    eq += __popc(be);
  }
}

template <int D, bool BFM>
cudaError_t launch_select(const SelectParams& p, int sms, cudaStream_t stream) {
  const int max_pages = (p.max_seq_len + p.page_size - 1) / p.page_size;
  const int64_t units = int64_t(p.num_seqs) * p.num_kv_heads;
  int ctas = 1;
  while (ctas < 8 && 2 * units * ctas <= int64_t(sms) * ctas_per_sm(D) && max_pages > ctas * kAlone) ctas *= 2;
  while (max_pages > ctas * kMaxChunk) ctas *= 2;
  const int mid = max_pages > 0 ? max_pages : 1;
  const int chunk = ((mid + ctas - 1) / ctas + kStrip - 1) / kStrip * kStrip;
  auto kernel = select_pages_kernel<D, BFM>;
  const int smem = ring_bytes(D) + chunk * 4;
  // (the most that any call needs, so that no thread lowers another's)
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               ring_bytes(D) + kMaxChunk * 4);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas), unsigned(p.num_kv_heads), unsigned(p.num_seqs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(smem);
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
  return cudaLaunchKernelEx(&cfg, kernel, p, chunk);
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
