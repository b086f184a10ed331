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
// A cluster of CTAs takes one (sequence, kv-head); each scores its run of the
// pages and keeps their keys in shared memory.  The threshold is found digit by
// digit from histograms that the CTAs read from one another, then every CTA
// writes its part of the list in order.
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
constexpr int kBins = 256;
constexpr int kTile = 16;                            // pages per MMA
constexpr int kMaxChunk = kSelectMaxPages / 8;       // pages per CTA
static_assert(kMaxChunk % kTile == 0, "whole tiles");

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

struct Shared {
  float qs[kMaxGroup], j[kMaxGroup];
  uint32_t hist[4][kBins];
  uint32_t count[2];                                 // this CTA's keys above the threshold, and equal to it
  uint32_t warp_count[kWarps][2];
  uint32_t digit, want;
};

template <int D, bool BFM>
__global__ void __launch_bounds__(kThreads) select_pages_kernel(const SelectParams p, int chunk) {
  pdl_wait_then_release();
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  constexpr int kKS = D / 16;                        // k-steps
  constexpr int kE = D / 32;
  constexpr int kW = D / 32;                         // words of a row per thread-in-group
  extern __shared__ __align__(16) uint32_t keys[];   // [chunk]
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
      sh.qs[h] = qs;
      sh.j[h] = float(sum);
    }
  }
  for (int i = tid; i < 4 * kBins; i += kThreads) sh.hist[i / kBins][i % kBins] = 0;
  __syncthreads();
  uint32_t b[kKS][2];
#pragma unroll
  for (int t = 0; t < kKS; ++t) {
    const uint2 v = reinterpret_cast<const uint2*>(qh)[t * 32 + lane];
    b[t][0] = v.x;
    b[t][1] = v.y;
  }
  const float qs0 = sh.qs[2 * c], qs1 = sh.qs[2 * c + 1], j0 = sh.j[2 * c], j1 = sh.j[2 * c + 1];

  // ---- keys of this CTA's run of the pages
  const int begin = min(rank * chunk, mid), count = min(mid - begin, chunk);
  const int64_t stride = summary_stride(hkv, D);
  bool bad = false;
  for (int t0 = warp * kTile; t0 < count; t0 += kWarps * kTile) {
    uint32_t w[2][kW], meta[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = t0 + g + 8 * u;
      const int id = i < count ? bt[lo + begin + i] : -1;
      const bool ok = id >= 0 && id < p.num_pages;
      bad = bad || (i < count && !ok);
      const uint8_t* s = p.summary + id * stride;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(s + kvh * (D / 2)) + kW * c;
#pragma unroll
      for (int k = 0; k < kW; ++k) w[u][k] = ok ? src[k] : 0u;
      // (NaN: counts as -infinity)
      meta[u] = ok ? *reinterpret_cast<const uint32_t*>(s + hkv * (D / 2) + 4 * kvh) : 0xFFFFFFFFu;
    }
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kW; ++k)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const uint32_t x = hh ? w[0][k] >> 8 : w[0][k], y = hh ? w[1][k] >> 8 : w[1][k];
        const uint32_t a[4] = {x & 0x000F000Fu, y & 0x000F000Fu, x & 0x00F000F0u, y & 0x00F000F0u};
        mma_16816(d, a, b[2 * k + hh][0], b[2 * k + hh][1]);
      }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float s = meta_lo(meta[u], BFM), z = meta_hi(meta[u], BFM);
      const float i0 = __fmul_rn(d[2 * u], 0x1p24f), i1 = __fmul_rn(d[2 * u + 1], 0x1p24f);
      float best = -INFINITY;                        // (fmaxf passes over NaN)
      if (2 * c < G) best = fmaxf(best, __fmul_rn(qs0, __fadd_rn(__fmul_rn(s, i0), __fmul_rn(z, j0))));
      if (2 * c + 1 < G) best = fmaxf(best, __fmul_rn(qs1, __fadd_rn(__fmul_rn(s, i1), __fmul_rn(z, j1))));
      best = fmaxf(best, __shfl_xor_sync(kAll, best, 1));
      best = fmaxf(best, __shfl_xor_sync(kAll, best, 2));
      const int i = t0 + g + 8 * u;
      if (c == 0 && i < count) keys[i] = key_of(best);
    }
  }
  if (bad) report(p.dev_status, SAW_ERR_DEVICE_INDEX);
  __syncthreads();

  // ---- the threshold: the want-th largest key of the cluster, digit by digit
  uint32_t prefix = 0, mask = 0, need = uint32_t(want);
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int i = tid; i < count; i += kThreads) {
      const uint32_t k = keys[i];
      if ((k & mask) == prefix) atomicAdd(&sh.hist[pass][(k >> shift) & 255u], 1u);
    }
    cluster.sync();
    if (warp == 0) {
      // eight bins per lane, from the top; lane 0 has the largest digits
      uint32_t v[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0;
      for (int r = 0; r < ctas; ++r) {
        const uint32_t* h = cluster.map_shared_rank(sh.hist[pass], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += h[255 - 8 * lane - j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += v[j];
      uint32_t above = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(kAll, above, d);
        if (lane >= d) above += o;
      }
      above -= sum;                                  // keys in larger digits
      if (above < need && need <= above + sum) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (above < need && need <= above + v[j]) {
            sh.digit = uint32_t(255 - 8 * lane - j);
            sh.want = need - above;
          }
          above += v[j];
        }
      }
    }
    __syncthreads();
    prefix |= sh.digit << shift;
    mask |= 255u << shift;
    need = sh.want;
    __syncthreads();
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
  cluster.sync();
  gt = eq = 0;
  for (int r = 0; r < rank; ++r) {
    const uint32_t* o = cluster.map_shared_rank(sh.count, r);
    gt += o[0];
    eq += o[1];
  }
  for (int w = 0; w < warp; ++w) {
    gt += sh.warp_count[w][0];
    eq += sh.warp_count[w][1];
  }
  cluster.sync();  // no CTA ends while another reads its memory
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
  while (ctas < 8 && units * ctas < sms && max_pages > ctas * 256) ctas *= 2;
  while (max_pages > ctas * kMaxChunk) ctas *= 2;
  const int mid = max_pages > 0 ? max_pages : 1;
  const int chunk = ((mid + ctas - 1) / ctas + kTile - 1) / kTile * kTile;
  auto kernel = select_pages_kernel<D, BFM>;
  const int smem = chunk * 4;
  // (the most that any call needs, so that no thread lowers another's)
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxChunk * 4);
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
  cfg.numAttrs = 2;
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
