// page_summary.cu -- the mean key of every page that a step completed, held
// like a cache row.
//
// Page e of a sequence, kv-head h, keys k_t = n_t s_t + z_t in the cache's
// (rotated) domain: A_d = sum_t n_td s_t and Z = sum_t z_t, each the even
// tokens in order plus the odd tokens in order; mean_d = RN(RN(A_d + Z) / P),
// quantized by the append's rule.  n s is exact in binary32 (4 by at most 11
// bits), so fma(n, s, A) rounds once like a product and a sum, and every step
// is one rounding: the bytes are determined.
#include <algorithm>

#include "saw_device.cuh"
#include "saw_int4.h"
#include "saw_quant_row.cuh"

namespace saw {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kWarps = 8;

// A warp sums one kv-head's page (head_dim 64: two kv-heads', a half-warp
// each).  A lane owns 8 dims, one 32-bit word of codes per token; D / 8 lanes
// hold a row, and the halves of what is left take the even and the odd tokens
// (head_dim 256: every lane takes both).
template <int D, int P, bool BFM>
__global__ void __launch_bounds__(32 * kWarps) page_summary_kernel(const SummaryParams p) {
  pdl_wait_then_release();
  constexpr int kRow = D / 8;                        // lanes per row
  constexpr int kHeads = D == 64 ? 2 : 1;            // kv-heads per warp
  constexpr bool kBoth = D == 256;                   // a lane takes even and odd tokens
  constexpr int kChunk = P * (D / 2 + 4);
  const int lane = threadIdx.x & 31;
  const int seq = blockIdx.y;
  const int L = p.seq_lens[seq];
  const int fresh = p.new_lens ? p.new_lens[seq] : L;
  if (L < 0 || fresh < 0 || L > (int64_t(p.max_blocks) << p.page_shift) || min(fresh, L) > p.max_new_len) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report(p.dev_status, SAW_ERR_DEVICE_INDEX);
    return;
  }
  const int first = (L - min(fresh, L)) >> p.page_shift, end = L >> p.page_shift;
  const int hkv = p.num_kv_heads;
  const int per = (hkv + kHeads - 1) / kHeads;       // warps per page
  const int64_t i = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (i >= int64_t(end - first) * per) return;
  const int page = first + int(i / per);
  const int head = int(i % per) * kHeads + (kHeads == 2 ? lane >> 4 : 0);
  const int id = p.block_tables[int64_t(seq) * p.max_blocks + page];
  if (id < 0 || id >= p.num_pages) {
    if (lane == 0) report(p.dev_status, SAW_ERR_DEVICE_INDEX);
    return;
  }
  const int r = lane & (kRow - 1);                   // word of the row
  const int odd = kBoth ? 0 : (lane / kRow) & 1;
  const uint8_t* chunk = p.k_cache + (int64_t(id) * hkv + min(head, hkv - 1)) * kChunk;
  constexpr int kSums = kBoth ? 2 : 1;
  float a[kSums][8], z[kSums];
#pragma unroll
  for (int u = 0; u < kSums; ++u) {
    z[u] = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) a[u][j] = 0.0f;
  }
#pragma unroll
  for (int t = 0; t < P; t += 2) {
#pragma unroll
    for (int u = 0; u < kSums; ++u) {
      const int tok = t + (kBoth ? u : odd);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(chunk + tok * (D / 2) + 4 * r);
      const uint32_t m = *reinterpret_cast<const uint32_t*>(chunk + P * (D / 2) + 4 * tok);
      const float s = meta_lo(m, BFM);
      z[u] = __fadd_rn(z[u], meta_hi(m, BFM));
#pragma unroll
      for (int j = 0; j < 8; ++j) a[u][j] = __fmaf_rn(float((w >> (4 * j)) & 15u), s, a[u][j]);
    }
  }
  float y[8], zz;
  if constexpr (kBoth) {
    zz = __fadd_rn(z[0], z[1]);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = __fadd_rn(a[0][j], a[1][j]);
  } else {
    zz = __fadd_rn(z[0], __shfl_xor_sync(kAll, z[0], kRow));
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = __fadd_rn(a[0][j], __shfl_xor_sync(kAll, a[0][j], kRow));
  }
  float mn = INFINITY, mx = -INFINITY;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    y[j] = __fmul_rn(__fadd_rn(y[j], zz), 1.0f / P);
    mn = fminf(mn, y[j]);
    mx = fmaxf(mx, y[j]);
  }
#pragma unroll
  for (int d = 1; d < kRow; d <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(kAll, mn, d));
    mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, d));
  }
  const RowMeta m = row_meta(mn, mx, BFM);
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int q = __float2int_rn(__fmul_rn(__fsub_rn(y[j], m.z), m.rcp));
    w |= uint32_t(min(max(q, 0), 15)) << (4 * j);
  }
  if (odd || head >= hkv) return;
  uint8_t* out = p.summary + id * summary_stride(hkv, D);
  reinterpret_cast<uint32_t*>(out + head * (D / 2))[r] = w;
  if (r == 0) *reinterpret_cast<uint32_t*>(out + hkv * (D / 2) + 4 * head) = uint32_t(m.sb) | (uint32_t(m.zb) << 16);
}

template <int D, int P>
cudaError_t launch_page(const SummaryParams& p, cudaStream_t stream) {
  const int per = (p.num_kv_heads + (D == 64 ? 1 : 0)) / (D == 64 ? 2 : 1);
  // a step of n tokens completes at most ceil(n / P) pages
  const int64_t warps = std::max<int64_t>((int64_t(p.max_new_len) + P - 1) / P, 1) * per;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((warps + kWarps - 1) / kWarps), unsigned(p.num_seqs));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.meta_bf16 ? cudaLaunchKernelEx(&cfg, page_summary_kernel<D, P, true>, p)
                     : cudaLaunchKernelEx(&cfg, page_summary_kernel<D, P, false>, p);
}

template <int D>
cudaError_t launch_dim(const SummaryParams& p, cudaStream_t stream) {
  switch (p.page_size) {
    case 16: return launch_page<D, 16>(p, stream);
    case 32: return launch_page<D, 32>(p, stream);
    case 64: return launch_page<D, 64>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_page_summary(const SummaryParams& p, int, cudaStream_t stream) {
  switch (p.head_dim) {
    case 64: return launch_dim<64>(p, stream);
    case 128: return launch_dim<128>(p, stream);
    case 256: return launch_dim<256>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace saw
