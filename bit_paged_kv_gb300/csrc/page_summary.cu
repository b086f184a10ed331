// page_summary.cu -- the mean key of every page that a step completed, held
// like a cache row.
//
// Page e of a sequence, kv-head h, keys k_t = n_t s_t + z_t in the cache's
// (rotated) domain: A_d = sum_t n_td s_t and Z = sum_t z_t, each the even
// tokens in order plus the odd tokens in order; mean_d = RN(RN(A_d + Z) / P),
// quantized by the append's rule.  n s is exact in binary32 (4 by at most 11
// bits), so fma(n, s, A) rounds once like a product and a sum, and every step
// is one rounding: the bytes are determined.
//
// The codes need no conversion (which runs at a quarter of the issue rate): a
// nibble left in place in a word of zeros is the binary32 16^j n 2^-149, up to j =
// 5 (bit 23 is the first exponent's, whose step is the subnormals').  s 2^111 is
// finite for every binary16 s, and the sums, kept times 16^j 2^-38, round as the
// plain ones do.  bfloat16 scales leave no room for that: there the nibble goes
// under the exponent of 2^23, which is taken off again.
//
// Bound: issue, 65 % of the slots where the pages are many, with the ALU pipe at 62 %:
// of 16.1 M warp instructions at 131072 tokens 4.2 M are the masks, one per code on a
// pipe of half rate, 2.1 M the fused steps, about 2 M loads and the words' conversion,
// the others what follows a sum.  131072 tokens, 8 kv-heads, D 128 (76 MB): 22.2 us
// (11.1 at the measured copy rate), bfloat16 words 32.9, four times as many tokens 74;
// with conversions 37, one kv-head a warp 26.  64-token pages 21.1 us.
#include <algorithm>

#include "saw_device.cuh"
#include "saw_int4.h"
#include "saw_quant_row.cuh"

namespace saw {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kWarps = 4;                            // (131072 tokens 22.2 us, with eight 24.7)
// Groups of kv-heads per warp, one after another: 131072 tokens 30.0 us with one, 24.5
// with two, 22.3 with four and with eight, four times as many 109, 85.7, 74.3, 74.3,
// bfloat16 words 37.9, 33.7, 32.9, 32.8; 32768 tokens, where warps are few, 7.5 with any.
// (A ring in shared memory filled by bulk copies instead of registers: 26.3 us, 37
// chunks of 64-token pages 18.6 against 11.9.)
constexpr int kMaxPasses = 4;

// a[j] += n_j s for the eight codes of a word; not BFM: s comes times 2^111 and
// the sums are times 16^place_of(j) 2^-38.
__host__ __device__ constexpr int place_of(int j) { return j < 6 ? j : j - 2; }
template <bool BFM>
__device__ __forceinline__ void add8(uint32_t w, float s, float2* a) {
  const uint32_t up = w >> 8;
  auto value = [&](int j) {
    return BFM ? ((w >> (4 * j)) & 15u) | 0x4B000000u : (j < 6 ? w : up) & (15u << (4 * place_of(j)));
  };
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float2 n = make_float2(__uint_as_float(value(2 * j)), __uint_as_float(value(2 * j + 1)));
    if constexpr (BFM) n = add2(n, make_float2(-0x1p23f, -0x1p23f));
    a[j] = fma2(n, make_float2(s, s), a[j]);
  }
}

// A lane owns kWords 32-bit words of codes per token (two, at head_dim 64 one),
// half of a row's lanes take the even tokens and half the odd ones; a warp sums
// two kv-heads' pages, at head_dim 256 one's.  Then a lane finishes half of its
// dims: one of its words, or half of its one.  A warp goes through `passes` groups
// of kv-heads of a page in batches of 16 tokens, the next batch under way.
template <int D, int P, bool BFM>
__global__ void __launch_bounds__(32 * kWarps) page_summary_kernel(const SummaryParams p, int passes) {
  pdl_wait_then_release();
  constexpr int kWords = D == 64 ? 1 : 2;
  constexpr int kRow = D / 8 / kWords;               // lanes per row of a token
  constexpr int kHeads = 16 / kRow;                  // kv-heads per warp
  constexpr int kChunk = P * (D / 2 + 4);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seq = blockIdx.y;
  const int L = p.seq_lens[seq];
  const int fresh = p.new_lens ? p.new_lens[seq] : L;
  if (L < 0 || fresh < 0 || L > (int64_t(p.max_blocks) << p.page_shift) || min(fresh, L) > p.max_new_len) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report(p.dev_status, SAW_ERR_DEVICE_INDEX);
    return;
  }
  const int first = (L - min(fresh, L)) >> p.page_shift, end = L >> p.page_shift;
  const int hkv = p.num_kv_heads;
  const int groups = (hkv + kHeads - 1) / kHeads;
  const uint32_t per = uint32_t((groups + passes - 1) / passes);  // warps per page
  const uint32_t i = blockIdx.x * kWarps + warp;
  if (i >= uint32_t(end - first) * per) return;
  const int page = first + int(i / per);
  const int group0 = int(i % per) * passes;
  const int id = p.block_tables[int64_t(seq) * p.max_blocks + page];
  if (id < 0 || id >= p.num_pages) {
    if (lane == 0) report(p.dev_status, SAW_ERR_DEVICE_INDEX);
    return;
  }
  const int r = lane & (kRow - 1);                   // lane of the row
  const int odd = (lane / kRow) & 1;
  const int sub = lane / (2 * kRow);                 // kv-head of the group
  constexpr int kBatch = 8, kBatches = P / 2 / kBatch;  // tokens of this lane
  struct Batch {
    uint32_t w[kBatch][kWords], m[kBatch];
  };
  const uint8_t* pages = p.k_cache + int64_t(id) * hkv * kChunk;
  auto load = [&](int k, Batch& x) {                 // batch k of this warp
    const int head = min((group0 + k / kBatches) * kHeads + sub, hkv - 1);
    const uint8_t* chunk = pages + int64_t(head) * kChunk;
    const uint8_t* code = chunk + (k % kBatches) * (kBatch * D) + odd * (D / 2) + 4 * kWords * r;
    const uint32_t* word = reinterpret_cast<const uint32_t*>(chunk + P * (D / 2)) + (k % kBatches) * (2 * kBatch) + odd;
#pragma unroll
    for (int t = 0; t < kBatch; ++t) {
      const uint8_t* src = code + t * D;
      if constexpr (kWords == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(src);
        x.w[t][0] = v.x;
        x.w[t][kWords - 1] = v.y;
      } else {
        x.w[t][0] = *reinterpret_cast<const uint32_t*>(src);
      }
      x.m[t] = word[2 * t];
    }
  };
  float2 a[kWords][4] = {};
  float z = 0.0f;
  auto sum_of = [&](int u, int j) { return j & 1 ? a[u][j >> 1].y : a[u][j >> 1].x; };
  auto add = [&](int k, const Batch& x) {
    if (k % kBatches == 0) {
#pragma unroll
      for (int u = 0; u < kWords; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) a[u][j] = make_float2(0.0f, 0.0f);
      z = 0.0f;
    }
#pragma unroll
    for (int t = 0; t < kBatch; ++t) {
      z = __fadd_rn(z, meta_hi(x.m[t], BFM));
      const float s = BFM ? meta_lo(x.m[t], BFM) : meta_lo(x.m[t], BFM) * 0x1p111f;
#pragma unroll
      for (int u = 0; u < kWords; ++u) add8<BFM>(x.w[t][u], s, a[u]);
    }
    if (k % kBatches != kBatches - 1) return;
    // even + odd; this lane keeps word `odd`, or half `odd` of its word
    constexpr int kMine = 4 * kWords;
    float y[kMine], mn = INFINITY, mx = -INFINITY;
    z = __fadd_rn(z, __shfl_xor_sync(kAll, z, kRow));
    if constexpr (!BFM) z *= 1.0f / P;
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int jo = kWords == 2 ? j : 4 + j;        // the other half's nibble
      const float lo = sum_of(0, j), hi = sum_of(kWords - 1, jo);
      const float x = __fadd_rn(odd ? hi : lo, __shfl_xor_sync(kAll, odd ? lo : hi, kRow));
      if constexpr (BFM) {
        y[j] = __fmul_rn(__fadd_rn(x, z), 1.0f / P);
      } else {
        // powers of two, far from either end of binary32's range: one rounding,
        // that of A + Z
        constexpr float kUnit = 0x1p38f / P;
        const float one = kUnit / float(1 << (4 * place_of(j))), two = kUnit / float(1 << (4 * place_of(jo)));
        y[j] = __fmaf_rn(x, kWords == 2 || !odd ? one : two, z);
      }
      mn = fminf(mn, y[j]);
      mx = fmaxf(mx, y[j]);
    }
#pragma unroll
    for (int d = 1; d < 2 * kRow; d <<= 1) {
      mn = fminf(mn, __shfl_xor_sync(kAll, mn, d));
      mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, d));
    }
    const RowMeta m = row_meta(mn, mx, BFM);
    // rounded half to even below 2^23's exponent, whose bits the sum of the words
    // takes 16^j times (clamping first is the same)
    uint32_t w = 0u - 0x4B000000u * (kMine == 8 ? 0x11111111u : 0x1111u);
    const bool clamp = __any_sync(kAll, !m.fast);
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      float q = __fmul_rn(__fsub_rn(y[j], m.z), m.rcp);
      if (clamp) q = fminf(fmaxf(q, 0.0f), 15.0f);
      w += __float_as_uint(__fadd_rn(q, 0x1p23f)) << (4 * j);
    }
    const int head = (group0 + k / kBatches) * kHeads + sub;
    if (head < hkv) {
      uint8_t* out = p.summary + id * summary_stride(hkv, D);
      uint8_t* row = out + head * (D / 2) + 4 * kWords * r + 2 * kWords * odd;
      if constexpr (kWords == 2) *reinterpret_cast<uint32_t*>(row) = w;
      else *reinterpret_cast<uint16_t*>(row) = uint16_t(w);
      if (r == 0 && !odd)
        *reinterpret_cast<uint32_t*>(out + hkv * (D / 2) + 4 * head) = uint32_t(m.sb) | (uint32_t(m.zb) << 16);
    }
  };
  const int n = min(passes, groups - group0) * kBatches;
  Batch x[2];
  load(0, x[0]);
#pragma unroll 1
  for (int k = 0; k < n; k += 2) {
    if (k + 1 < n) load(k + 1, x[1]);
    add(k, x[0]);
    if (k + 1 >= n) break;
    if (k + 2 < n) load(k + 2, x[0]);
    add(k + 1, x[1]);
  }
}

template <int D, int P>
cudaError_t launch_page(const SummaryParams& p, int sms, cudaStream_t stream) {
  constexpr int kHeads = D == 256 ? 1 : 2;
  const int groups = (p.num_kv_heads + kHeads - 1) / kHeads;
  // a step of n tokens completes at most ceil(n / P) pages
  const int64_t pages = std::max<int64_t>((int64_t(p.max_new_len) + P - 1) / P, 1);
  // more groups per warp where that leaves warps enough
  int passes = 1;
  while (passes < kMaxPasses && passes < groups && pages * groups * p.num_seqs >= int64_t(2 * passes) * 32 * sms) passes *= 2;
  const int64_t warps = pages * ((groups + passes - 1) / passes);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((warps + kWarps - 1) / kWarps), unsigned(p.num_seqs));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.meta_bf16 ? cudaLaunchKernelEx(&cfg, page_summary_kernel<D, P, true>, p, passes)
                     : cudaLaunchKernelEx(&cfg, page_summary_kernel<D, P, false>, p, passes);
}

template <int D>
cudaError_t launch_dim(const SummaryParams& p, int sms, cudaStream_t stream) {
  switch (p.page_size) {
    case 16: return launch_page<D, 16>(p, sms, stream);
    case 32: return launch_page<D, 32>(p, sms, stream);
    case 64: return launch_page<D, 64>(p, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_page_summary(const SummaryParams& p, int sms, cudaStream_t stream) {
  switch (p.head_dim) {
    case 64: return launch_dim<64>(p, sms, stream);
    case 128: return launch_dim<128>(p, sms, stream);
    case 256: return launch_dim<256>(p, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace saw
