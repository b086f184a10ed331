// rope_append.cu -- rotary positions on q and k fused with the rotated,
// quantized append of k and v, and the table of cosines and sines it reads.
//
// Rotary: the first r = rope_dim elements of a head are r/2 pairs; pair i of
// a token at position p is turned by the angle p w_i:
//   y0 = RN(RN(x0 c) - RN(x1 s)),  y1 = RN(RN(x1 c) + RN(x0 s)),
// in binary32, products rounded separately, so the result is fixed to the
// bit by the table.  Pairs are (i, i + r/2) or, interleaved, (2i, 2i + 1).
// k goes on in binary32 into the append's butterfly and quantizer (the rule
// of saw_quantize_append from "widen to binary32" on); q is rounded once, to
// the input type.
#include <numeric>
#include <type_traits>

#include "saw_device.cuh"
#include "saw_int4.h"
#include "saw_quant_row.cuh"

namespace saw {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t pack_bf162(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ------------------------------------------------------------ table
//
// The angle of position p is p w_i / 2 pi turns.  turns_i arrives as a 64-bit
// binary fraction (of a binary64: a relative error of 2^-52, which moves the
// angle by p w_i 2^-52 radians), so p * turns_i modulo 2^64 is the angle modulo
// one turn; its top two bits, rounded, are the quarter, the rest an angle within
// 1/8 turn that binary32 holds to 2^-27 turns.  There the Taylor series of sine
// (to x^9) and cosine (to x^10) are within 2^-29, two pairs per packed
// instruction.
//
// Bound: HBM writes; 131072 x 128 floats (67 MB) in 10.9 us, 6.1 TB/s, 9.9 us
// at the measured copy rate.  With sincospif, bound by issue, 17.4 us.
constexpr int kTableThreads = 256;

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(const RopeTableParams p) {
  pdl_wait_then_release();
  __shared__ uint64_t turns[kRopeMaxPairs];
  for (int i = threadIdx.x; i < p.pairs; i += kTableThreads) turns[i] = p.turns[i];
  __syncthreads();
  const uint32_t quads = p.pairs / 4;  // four pairs per thread
  const uint32_t rows = gridDim.x * kTableThreads / quads;  // positions in flight
  const uint32_t me = blockIdx.x * kTableThreads + threadIdx.x;
  const uint32_t i0 = me % quads * 4;
  uint64_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = turns[i0 + k];
  if (me >= rows * quads) return;
  for (int64_t pos = me / quads; pos < p.max_pos; pos += rows) {
    float cv[4], sv[4];
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      uint32_t q[2];
      float2 x;  // radians, |x| <= pi / 4
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t hi = uint32_t((uint64_t(pos) * w[k + j]) >> 32);
        q[j] = (hi + 0x20000000u) >> 30;
        const float f = float(int32_t(hi - (q[j] << 30)));
        (j ? x.y : x.x) = f * 1.4629180792671596e-09f;  // 2 pi 2^-32
      }
      const float2 t = mul2(x, x);
      float2 s = fma2(t, both(2.7557319e-6f), both(-1.9841270e-4f));
      s = fma2(t, s, both(8.3333333e-3f));
      s = fma2(t, s, both(-1.6666667e-1f));
      s = fma2(mul2(t, x), s, x);
      float2 c = fma2(t, both(-2.7557319e-7f), both(2.4801587e-5f));
      c = fma2(t, c, both(-1.3888889e-3f));
      c = fma2(t, c, both(4.1666667e-2f));
      c = fma2(t, c, both(-0.5f));
      c = fma2(t, c, both(1.0f));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float sj = j ? s.y : s.x, cj = j ? c.y : c.x;
        const bool odd = q[j] & 1;
        const uint32_t a = __float_as_uint(odd ? sj : cj), b = __float_as_uint(odd ? cj : sj);
        // cosine negative in quarters 1 and 2, sine in 2 and 3
        cv[k + j] = __uint_as_float(a ^ (((q[j] + 1) & 2) << 30)) * p.att;
        sv[k + j] = __uint_as_float(b ^ ((q[j] & 2) << 30)) * p.att;
      }
    }
    float* row = p.cos_sin + pos * (2 * p.pairs);
    *reinterpret_cast<float4*>(row + i0) = make_float4(cv[0], cv[1], cv[2], cv[3]);
    *reinterpret_cast<float4*>(row + p.pairs + i0) = make_float4(sv[0], sv[1], sv[2], sv[3]);
  }
}

// ------------------------------------------------------------ one row per warp
//
// Lane l holds elements E l .. E l + E - 1 (E = D / 32).  Any size, layout and
// stride; the bulk kernel takes over for large batches.  Bound by latency: one
// token, 32 and 8 heads, 2.6 us, a launch and three dependent loads.
constexpr int kRowWarps = 4;

template <int D>
__device__ __forceinline__ void load_row(const uint16_t* src, bool f16, float (&x)[D / 32]) {
  constexpr int E = D / 32;
  if constexpr (E == 2) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(src);
    x[0] = in_lo(w, f16);
    x[1] = in_hi(w, f16);
  } else {
    uint32_t ws[E / 2];
    if constexpr (E == 4) {
      const uint2 w = *reinterpret_cast<const uint2*>(src);
      ws[0] = w.x;
      ws[1] = w.y;
    } else {
      const uint4 w = *reinterpret_cast<const uint4*>(src);
      ws[0] = w.x;
      ws[1] = w.y;
      ws[2] = w.z;
      ws[3] = w.w;
    }
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      x[2 * j] = in_lo(ws[j], f16);
      x[2 * j + 1] = in_hi(ws[j], f16);
    }
  }
}

// Turns the lane's elements in place.  cs: the token's row of the table.
template <int D>
__device__ __forceinline__ void turn_row(float (&x)[D / 32], const float* cs, int r, bool inter,
                                         int lane) {
  constexpr int E = D / 32;
  const int half = r >> 1;
  const int d0 = E * lane;
  if (inter) {
    if (d0 < r) {
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const int i = (d0 + e) >> 1;
        const float c = __ldg(cs + i), s = __ldg(cs + half + i);
        const float a = x[e], b = x[e + 1];
        x[e] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
        x[e + 1] = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
      }
    }
  } else {
    // the partner element sits `half` elements away, half / E lanes (r is a
    // multiple of 16, so half is one of E)
    const bool low = d0 < half, in = d0 < r;
    const int hop = half / E;
    const int from = in ? (low ? lane + hop : lane - hop) : lane;
    const int i0 = low ? d0 : d0 - half;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float o = __shfl_sync(kAll, x[e], from);
      if (in) {
        const float c = __ldg(cs + i0 + e), s = __ldg(cs + half + i0 + e);
        const float u = __fmul_rn(x[e], c), v = __fmul_rn(o, s);
        x[e] = low ? __fsub_rn(u, v) : __fadd_rn(u, v);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(32 * kRowWarps) rope_append_row_kernel(const RopeParams p) {
  pdl_wait_then_release();
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int hkv = p.num_kv_heads;
  const int per = p.num_q_heads + hkv * p.num_tensors;  // rows of a token: q heads, k, v
  const int64_t gw = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (gw >= int64_t(p.num_tokens) * per) return;
  const int t = int(gw / per), j = int(gw - int64_t(t) * per);
  const bool f16 = p.in_f16 != 0;
  const bool is_q = j < p.num_q_heads;
  const int tensor = is_q || j < p.num_q_heads + hkv ? 0 : 1;
  const int hd = is_q ? j : j - p.num_q_heads - tensor * hkv;
  const bool turned = is_q || tensor == 0;

  int32_t slot = -1, pos = 0;
  if (!is_q) slot = p.slot_mapping[t];
  if (turned) {
    pos = p.positions[t];
    if (pos < 0 || pos >= p.max_pos) {  // the token is skipped and reported
      if (lane == 0) report(p.dev_status, SAW_ERR_DEVICE_INDEX);
      return;
    }
  }
  if (!is_q) {
    if (slot == -1) return;
    if (slot < 0 || int64_t(slot) >= p.num_slots) {
      if (lane == 0) report(p.dev_status, SAW_ERR_DEVICE_INDEX);
      return;
    }
    if (!turned) {  // V of a token whose position is bad is skipped with its K
      const int32_t q = p.positions[t];
      if (q < 0 || q >= p.max_pos) return;
    }
  }
  const uint16_t* src = is_q ? p.q + int64_t(t) * p.q_stride
                             : (tensor ? p.v + int64_t(t) * p.v_stride : p.k + int64_t(t) * p.k_stride);
  float x[E];
  load_row<D>(src + int64_t(hd) * D + E * lane, f16, x);
  if (turned)
    turn_row<D>(x, p.cos_sin + int64_t(pos) * p.rope_dim, p.rope_dim, p.interleaved != 0, lane);

  if (is_q) {
    uint16_t* dst = p.q_out + int64_t(t) * p.q_out_stride + int64_t(hd) * D + E * lane;
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) w[e / 2] = f16 ? pack_half2(x[e], x[e + 1]) : pack_bf162(x[e], x[e + 1]);
    if constexpr (E == 2) *reinterpret_cast<uint32_t*>(dst) = w[0];
    else if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }

  if (tensor ? p.rotate_v : p.rotate_k) {
    const int h = p.block_h;
#pragma unroll
    for (int s = 1; s < E; s <<= 1) {
      if (s < h) {
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (!(i & s)) {
            const float a = x[i], b = x[i + s];
            x[i] = __fadd_rn(a, b);
            x[i + s] = __fsub_rn(a, b);
          }
      }
    }
    for (int s = E; s < h; s <<= 1) {
      const int m = s / E;
      const bool upper = (lane & m) != 0;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float o = __shfl_xor_sync(kAll, x[i], m);
        x[i] = upper ? __fsub_rn(o, x[i]) : __fadd_rn(x[i], o);
      }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = __fmul_rn(x[i], p.c_h);
  }
  float mn = x[0], mx = x[0];
#pragma unroll
  for (int i = 1; i < E; ++i) {
    mn = fminf(mn, x[i]);
    mx = fmaxf(mx, x[i]);
  }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) {
    mn = fminf(mn, __shfl_xor_sync(kAll, mn, m));
    mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, m));
  }
  const RowMeta m = row_meta(mn, mx, p.meta_bf16 != 0);
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    int q = __float2int_rn(__fmul_rn(__fsub_rn(x[i], m.z), m.rcp));
    q = min(max(q, 0), 15);
    codes |= uint32_t(q) << (4 * i);
  }
  const int P = p.page_size;
  const int page = slot >> p.page_shift, off = slot & (P - 1);
  uint8_t* chunk = (tensor ? p.v_cache : p.k_cache) + (int64_t(page) * hkv + hd) * int64_t(P * (D / 2 + 4));
  if constexpr (E == 2) chunk[off * (D / 2) + lane] = uint8_t(codes);
  else if constexpr (E == 4) reinterpret_cast<uint16_t*>(chunk + off * (D / 2))[lane] = uint16_t(codes);
  else reinterpret_cast<uint32_t*>(chunk + off * (D / 2))[lane] = codes;
  if (lane == 0)
    *reinterpret_cast<uint32_t*>(chunk + P * (D / 2) + 4 * off) = uint32_t(m.sb) | (uint32_t(m.zb) << 16);
}

template <int D>
cudaError_t launch_rows(const RopeParams& p, cudaStream_t stream) {
  const int64_t warps = int64_t(p.num_tokens) * (p.num_q_heads + p.num_kv_heads * p.num_tensors);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((warps + kRowWarps - 1) / kRowWarps));
  cfg.blockDim = dim3(32 * kRowWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_append_row_kernel<D>, p);
}

// ------------------------------------------------------------ bulk
//
// Large batches.  Item = (token, part): up to kQPart q-heads, or the token's K
// rows, or its V rows; every warp walks items on its own, so that the q parts
// (pure traffic) and the K and V parts (150 or so instructions a row, which
// alone would be bound by issue) of different warps share an SM.  A lane holds
// two 16-byte chunks (8 dims) of a row, D / 16 lanes share it.  The chunks lie
// r / 2 dims apart where r / 16 is a power of two (else, and interleaved, D / 2
// apart): the (i, i + r/2) pairs sit in one lane, the butterfly's strides 1, 2,
// 4 and that one too, and only the others cross lanes.  The lane's cosines and
// sines serve all heads of the token.
//
// Bound: HBM.  131072 tokens, Hq 32, Hkv 8, D 128: 2.90 GB in 484 us, 6.0 TB/s
// (426 us at the measured copy rate); 2047 tokens, half the head turned (45
// MB), 12.7 us, where a warp has an item or two and latency counts.
constexpr int kBulkWarps = 8;
constexpr int kRounds = 4;  // rounds of q-head loads in flight
// Smaller batches take a warp per row.  That against this kernel, us: 64
// q-heads 96 tokens 3.5 / 3.7, 128 tokens 3.7 / 3.7, 160 tokens 4.6 / 3.7, 256
// tokens 6.1 / 4.4; 32 q-heads, half the head turned, 64 tokens 2.8 / 4.9, 256
// tokens 5.0 / 4.9, 512 tokens 8.2 / 5.6.
constexpr int64_t kBulkMinElems = int64_t(5) << 18;
constexpr int kQPart = 16;  // q-heads per item
enum { kHalfWhole = 0, kHalfPart = 1, kInter = 2, kHalfBit = 3 };  // whole head; any part; -; r / 16 a power of two
// CTAs per SM (85 or 128 registers a thread): 131072 tokens 484 us with three,
// 527 with two; the layout that exchanges partners by shuffles keeps two (2047
// tokens, half the head: 14.4 us, 22.3 with three and spills; by kHalfBit 12.7,
// 8192 tokens 47.2 against 37.9).
constexpr int bulk_ctas(int layout) { return layout == kHalfPart ? 2 : 3; }

template <bool F16IN>
__device__ __forceinline__ void widen8(const uint4& w, float* x) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = in_lo(ws[j], F16IN);
    x[2 * j + 1] = in_hi(ws[j], F16IN);
  }
}
template <bool F16IN>
__device__ __forceinline__ uint4 narrow8(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = F16IN ? pack_half2(x[2 * j], x[2 * j + 1]) : pack_bf162(x[2 * j], x[2 * j + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A lane's cosines and sines: of its pairs (kHalfWhole, kHalfBit: 8), of its
// chunks' 2 x 4 pairs (kInter), or of its chunks' 2 x 8 elements (kHalfPart).
template <int LAYOUT>
struct Angles {
  static constexpr int kN = LAYOUT == kHalfPart ? 16 : 8;
  float c[kN], s[kN];
};

template <int D, int LAYOUT>
__device__ __forceinline__ void load_angles(Angles<LAYOUT>& t, const float* cs, int r, int a) {
  const int half = r >> 1;
  auto run = [&](int at, int i, auto count) {  // c, s [at ..] from pairs i ..
    constexpr int n = decltype(count)::value;
#pragma unroll
    for (int k = 0; k < n; k += 4) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(cs + i + k));
      const float4 y = __ldg(reinterpret_cast<const float4*>(cs + half + i + k));
      t.c[at + k] = x.x; t.c[at + k + 1] = x.y; t.c[at + k + 2] = x.z; t.c[at + k + 3] = x.w;
      t.s[at + k] = y.x; t.s[at + k + 1] = y.y; t.s[at + k + 2] = y.z; t.s[at + k + 3] = y.w;
    }
  };
  using N4 = std::integral_constant<int, 4>;
  using N8 = std::integral_constant<int, 8>;
  if constexpr (LAYOUT == kHalfWhole) {
    run(0, 8 * a, N8{});
  } else if constexpr (LAYOUT == kHalfBit) {  // (a: the lane's first chunk)
    if (8 * a < half) run(0, 8 * a, N8{});
  } else {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int ch = a + u * (D / 16);
      if (8 * ch < r) {
        if constexpr (LAYOUT == kInter) run(4 * u, 4 * ch, N4{});
        else run(8 * u, 8 * (8 * ch < half ? ch : ch - half / 8), N8{});
      }
    }
  }
}

// Turns a lane's 16 values.  Each product and each sum is rounded once
// (scalar sums: packed products and packed sums were fused by the assembler).
template <int D, int LAYOUT>
__device__ __forceinline__ void turn16(float (&x)[16], const Angles<LAYOUT>& t, int r, int a, int lane) {
  if constexpr (LAYOUT == kHalfWhole || LAYOUT == kHalfBit) {
    if (LAYOUT == kHalfBit && 16 * a >= r) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float u = x[e], v = x[8 + e];
      x[e] = __fsub_rn(__fmul_rn(u, t.c[e]), __fmul_rn(v, t.s[e]));
      x[8 + e] = __fadd_rn(__fmul_rn(v, t.c[e]), __fmul_rn(u, t.s[e]));
    }
  } else if constexpr (LAYOUT == kInter) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (8 * (a + u * (D / 16)) < r) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p = x[8 * u + 2 * e], q = x[8 * u + 2 * e + 1];
          x[8 * u + 2 * e] = __fsub_rn(__fmul_rn(p, t.c[4 * u + e]), __fmul_rn(q, t.s[4 * u + e]));
          x[8 * u + 2 * e + 1] = __fadd_rn(__fmul_rn(q, t.c[4 * u + e]), __fmul_rn(p, t.s[4 * u + e]));
        }
      }
  } else {
    // the partner of chunk ch is `half` elements away: chunk pc, in lane pc %
    // (D / 16) of this row as its first or second chunk
    constexpr int LPR = D / 16;
    const int hc = r >> 4;  // chunks of half the turned part
    float o[16];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int ch = a + u * LPR;
      const int pc = ch < hc ? ch + hc : (ch < 2 * hc ? ch - hc : ch);
      const int from = (lane & ~(LPR - 1)) | (pc & (LPR - 1));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f0 = __shfl_sync(kAll, x[e], from), f1 = __shfl_sync(kAll, x[8 + e], from);
        o[8 * u + e] = pc >= LPR ? f1 : f0;
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int ch = a + u * LPR;
      if (ch < 2 * hc) {
        const bool low = ch < hc;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float m = __fmul_rn(x[8 * u + e], t.c[8 * u + e]), n = __fmul_rn(o[8 * u + e], t.s[8 * u + e]);
          x[8 * u + e] = low ? __fsub_rn(m, n) : __fadd_rn(m, n);
        }
      }
    }
  }
}

// The row's butterfly (blocks of h, ascending strides), then the factor.
// Sums with a partner lane as RN(+-x + o), the +-1 product exact.  The lane's
// two chunks are hc chunks apart.
template <int D>
__device__ __forceinline__ void rotate16(float (&x)[16], int h, float c_h, int hc, int lane) {
#pragma unroll
  for (int s = 1; s < 8; s <<= 1) {  // (h >= 16)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!(i & s)) {
        const float a = x[i], b = x[i + s];
        x[i] = __fadd_rn(a, b);
        x[i + s] = __fsub_rn(a, b);
      }
  }
#pragma unroll
  for (int s = 8; s < D; s <<= 1) {
    if (s >= h) continue;
    if (s == 8 * hc) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = x[i], b = x[i + 8];
        x[i] = __fadd_rn(a, b);
        x[i + 8] = __fsub_rn(a, b);
      }
    } else {
      const int m = s < 8 * hc ? s >> 3 : s >> 4;
      const float sign = (lane & m) ? -1.0f : 1.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __fmaf_rn(x[i], sign, __shfl_xor_sync(kAll, x[i], m));
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(x[i], c_h);
}

// Eight codes as a word.  fast (no clamp can bite): (y - z) r 2^-24 converts
// to a binary16 whose bits are the round-half-even code.
__device__ __forceinline__ uint32_t codes8(const float* x, const RowMeta& m) {
  if (m.fast) {
    const float r24 = __fmul_rn(m.rcp, 5.9604644775390625e-08f);
    uint32_t d[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int a = (k & 1) + 4 * (k >> 1);
      d[k] = pack_half2(__fmul_rn(__fsub_rn(x[a], m.z), r24), __fmul_rn(__fsub_rn(x[a + 2], m.z), r24));
    }
    // bytes 0 and 2: (c0 c1), (c2 c3); (c4 c5), (c6 c7); a -0 leaves its sign
    // in a byte that is dropped or masked
    const uint32_t lo = d[0] | ((d[1] << 4) & 0x00F000F0u), hi = d[2] | ((d[3] << 4) & 0x00F000F0u);
    return prmt(lo, hi, 0x6420u);
  }
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    int q = __float2int_rn(__fmul_rn(__fsub_rn(x[k], m.z), m.rcp));
    q = min(max(q, 0), 15);
    w |= uint32_t(q) << (4 * k);
  }
  return w;
}

template <int D, bool F16IN, int LAYOUT>
__global__ void __launch_bounds__(32 * kBulkWarps, bulk_ctas(LAYOUT))
    rope_append_bulk_kernel(const RopeParams p, uint32_t warps) {
  pdl_wait_then_release();
  constexpr int LPR = D / 16, RPW = 32 / LPR;  // lanes per row, rows per warp
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR;
  // the lane's chunks are a and a + hc: its index with a zero put in at hc's bit
  const int hc = LAYOUT == kHalfBit ? p.rope_dim >> 4 : LPR;
  const int a = LAYOUT == kHalfBit ? ((lane & (LPR - 1) & -hc) << 1) | (lane & (hc - 1)) : lane & (LPR - 1);
  const int nq = (p.num_q_heads + kQPart - 1) / kQPart;
  const uint32_t parts = uint32_t(nq + p.num_tensors);
  const uint32_t items = uint32_t(p.num_tokens) * parts;
  const int hkv = p.num_kv_heads;
  uint32_t it = blockIdx.x * kBulkWarps + (threadIdx.x >> 5);
  if (it >= warps) return;
  // the next item's position and slot are under way while one is worked on
  int pos_next = it < items ? p.positions[it / parts] : 0;
  int slot_next = it < items ? p.slot_mapping[it / parts] : 0;
  for (; it < items; it += warps) {
    const int t = int(it / parts), part = int(it - uint32_t(t) * parts);
    const int pos = pos_next, slot = slot_next;
    if (it + warps < items) {
      pos_next = p.positions[(it + warps) / parts];
      slot_next = p.slot_mapping[(it + warps) / parts];
    }
    const bool pos_ok = pos >= 0 && pos < p.max_pos;
    if (part < nq) {
      // ---- q-heads, kRounds rounds of loads in flight
      if (!pos_ok) continue;  // (reported with the K rows)
      const int h0 = part * kQPart, h1 = min(p.num_q_heads, h0 + kQPart);
      const uint16_t* src = p.q + int64_t(t) * p.q_stride + 8 * a;
      uint16_t* dst = p.q_out + int64_t(t) * p.q_out_stride + 8 * a;
      Angles<LAYOUT> ang;
      load_angles<D>(ang, p.cos_sin + int64_t(pos) * p.rope_dim, p.rope_dim, a);
      for (int hb = h0; hb < h1; hb += RPW * kRounds) {
        uint4 w[kRounds][2];
#pragma unroll
        for (int k = 0; k < kRounds; ++k) {
          const int h = hb + k * RPW + sub;
          w[k][0] = w[k][1] = make_uint4(0u, 0u, 0u, 0u);
          if (h < h1) {
            w[k][0] = *reinterpret_cast<const uint4*>(src + h * D);
            w[k][1] = *reinterpret_cast<const uint4*>(src + h * D + 8 * hc);
          }
        }
#pragma unroll
        for (int k = 0; k < kRounds; ++k) {
          if (hb + k * RPW >= h1) break;
          const int h = hb + k * RPW + sub;
          float x[16];
          widen8<F16IN>(w[k][0], x);
          widen8<F16IN>(w[k][1], x + 8);
          turn16<D, LAYOUT>(x, ang, p.rope_dim, a, lane);
          if (h < h1) {
            *reinterpret_cast<uint4*>(dst + h * D) = narrow8<F16IN>(x);
            *reinterpret_cast<uint4*>(dst + h * D + 8 * hc) = narrow8<F16IN>(x + 8);
          }
        }
      }
      continue;
    }
    // ---- K or V rows
    const int tensor = part - nq;
    if (!pos_ok && tensor == 0 && lane == 0) report(p.dev_status, SAW_ERR_DEVICE_INDEX);
    if (slot == -1 || !pos_ok) continue;
    if (slot < 0 || int64_t(slot) >= p.num_slots) {
      if (lane == 0) report(p.dev_status, SAW_ERR_DEVICE_INDEX);
      continue;
    }
    const uint16_t* src = (tensor ? p.v + int64_t(t) * p.v_stride : p.k + int64_t(t) * p.k_stride) + 8 * a;
    const int P = p.page_size;
    const int page = slot >> p.page_shift, off = slot & (P - 1);
    uint8_t* chunk0 = (tensor ? p.v_cache : p.k_cache) + int64_t(page) * hkv * int64_t(P * (D / 2 + 4));
    const bool rot = (tensor ? p.rotate_v : p.rotate_k) != 0;
    uint4 w0 = make_uint4(0u, 0u, 0u, 0u), w1 = w0;
    if (sub < hkv) {
      w0 = *reinterpret_cast<const uint4*>(src + sub * D);
      w1 = *reinterpret_cast<const uint4*>(src + sub * D + 8 * hc);
    }
    Angles<LAYOUT> ang;
    if (tensor == 0) load_angles<D>(ang, p.cos_sin + int64_t(pos) * p.rope_dim, p.rope_dim, a);
    for (int hb = 0; hb < hkv; hb += RPW) {
      const int h = hb + sub;
      float x[16];
      widen8<F16IN>(w0, x);
      widen8<F16IN>(w1, x + 8);
      if (h + RPW < hkv) {  // the next rows, under way while these are worked on
        w0 = *reinterpret_cast<const uint4*>(src + (h + RPW) * D);
        w1 = *reinterpret_cast<const uint4*>(src + (h + RPW) * D + 8 * hc);
      }
      if (tensor == 0) turn16<D, LAYOUT>(x, ang, p.rope_dim, a, lane);
      if (rot) rotate16<D>(x, p.block_h, p.c_h, hc, lane);
      float mn = fminf(x[0], x[1]), mx = fmaxf(x[0], x[1]);
#pragma unroll
      for (int i = 2; i < 16; ++i) {
        mn = fminf(mn, x[i]);
        mx = fmaxf(mx, x[i]);
      }
#pragma unroll
      for (int d = 1; d < LPR; d <<= 1) {
        mn = fminf(mn, __shfl_xor_sync(kAll, mn, d));
        mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, d));
      }
      const RowMeta m = row_meta(mn, mx, p.meta_bf16 != 0);
      const uint32_t c0 = codes8(x, m), c1 = codes8(x + 8, m);
      if (h < hkv) {
        uint8_t* chunk = chunk0 + int64_t(h) * (P * (D / 2 + 4));
        uint32_t* codes = reinterpret_cast<uint32_t*>(chunk + off * (D / 2));
        codes[a] = c0;
        codes[a + hc] = c1;
        if (a == 0)
          *reinterpret_cast<uint32_t*>(chunk + P * (D / 2) + 4 * off) = uint32_t(m.sb) | (uint32_t(m.zb) << 16);
      }
    }
  }
}

template <int D, bool F16IN, int LAYOUT>
cudaError_t launch_bulk_l(const RopeParams& p, int sms, cudaStream_t stream) {
  const int parts = (p.num_q_heads + kQPart - 1) / kQPart + p.num_tensors;
  const int64_t items = int64_t(p.num_tokens) * parts;
  const int64_t want = (items + kBulkWarps - 1) / kBulkWarps;
  cudaLaunchConfig_t cfg = {};
  const int64_t most = int64_t(bulk_ctas(LAYOUT)) * sms;
  cfg.gridDim = dim3(unsigned(want < most ? want : most));
  cfg.blockDim = dim3(32 * kBulkWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // a stride coprime to the parts gives every warp all kinds of them in turn
  // (a common divisor: some warps quantize, some only turn q; 525 -> 690 us)
  uint32_t warps = cfg.gridDim.x * kBulkWarps;
  while (warps > 1 && std::gcd(warps, uint32_t(parts)) != 1) --warps;
  return cudaLaunchKernelEx(&cfg, rope_append_bulk_kernel<D, F16IN, LAYOUT>, p, warps);
}

template <int D>
cudaError_t launch_bulk(const RopeParams& p, int sms, cudaStream_t stream) {
  const int hc = p.rope_dim >> 4;
  const int layout = p.interleaved ? kInter : p.rope_dim == D ? kHalfWhole : hc & (hc - 1) ? kHalfPart : kHalfBit;
  auto with = [&](auto f16) {
    constexpr bool F = decltype(f16)::value;
    switch (layout) {
      case kInter: return launch_bulk_l<D, F, kInter>(p, sms, stream);
      case kHalfWhole: return launch_bulk_l<D, F, kHalfWhole>(p, sms, stream);
      case kHalfBit: return launch_bulk_l<D, F, kHalfBit>(p, sms, stream);
      default: return launch_bulk_l<D, F, kHalfPart>(p, sms, stream);
    }
  };
  return p.in_f16 ? with(std::true_type{}) : with(std::false_type{});
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableParams& p, int sms, cudaStream_t stream) {
  const int64_t items = int64_t(p.max_pos) * (p.pairs / 4);
  const int64_t want = (items + kTableThreads - 1) / kTableThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(want < int64_t(8) * sms ? want : int64_t(8) * sms));
  cfg.blockDim = dim3(kTableThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_table_kernel, p);
}

cudaError_t launch_rope_append(const RopeParams& p, int sms, cudaStream_t stream) {
  const bool bulk = int64_t(p.num_tokens) * (p.num_q_heads + 2 * p.num_kv_heads) * p.head_dim >= kBulkMinElems;
  switch (p.head_dim) {
    case 64: return bulk ? launch_bulk<64>(p, sms, stream) : launch_rows<64>(p, stream);
    case 128: return bulk ? launch_bulk<128>(p, sms, stream) : launch_rows<128>(p, stream);
    case 256: return bulk ? launch_bulk<256>(p, sms, stream) : launch_rows<256>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace saw
