// build_tables.cu -- block tables, slot mapping, positions and lengths of a
// batch, built on the GPU from the requests' lengths and a list of free pages.
//
// For request b with c cached and n new tokens and pages of P tokens:
//   old = ceil(c / P), need = ceil((c + n) / P) - old,
//   off = sum of need over the requests before b,
//   table entry e: the source row's for e < old, free[off + e - old] up to
//   old + need; token i of the n: position c + i, slot
//   entry[(c + i) / P] * P + (c + i) % P.
// A request with off + need beyond the free list gets no page: every later
// request that needs one fails the same test, so the pages taken are always
// a prefix of the list, whatever the order in which CTAs run.
//
// One launch, and no CTA waits for another: every CTA computes the two
// exclusive sums (tokens, pages) over all requests itself -- coalesced loads
// into shared memory, each thread the sum of a run of requests, one scan over
// threads -- and keeps them with the requests' lengths and rows (above kDirect
// requests, 229 KB, the sums of every 32nd only).  That is 12 bytes per request and
// CTA from L2, against a second launch or a look-back between CTAs.  Then the
// grid shares out (request, 512 entries) pieces of table rows and runs of 128
// tokens to warps.  A warp's first and last token, found by bisection, bound
// the search of the others; the four page words of a lane load together.
//
// Bound: 64 requests with tables of up to 16384 tokens (0.3 MB), 4.2 us, are
// a launch and four dependent loads.  4096 requests of up to 32768 cached and
// 256 new tokens, 13.1 us over one batch again and again and 15.3 over three in
// turn, move 42 MB (6.2 us at the measured copy rate); the rest is issue: 17.6 us with 64-bit sums and the group size a variable, 33.9
// with a scan per 32 requests in two CTAs per SM.
#include "saw_device.cuh"
#include "saw_int4.h"
#include "saw_quant_row.cuh"

namespace saw {
namespace {

constexpr int kTabMaxThreads = 1024;
// Up to this many requests: one prefix entry per request, as many as 227 KB of
// shared memory hold.  Above: one per 32, the requests read again where they are
// needed (1000 cached and one new token each, us: 4097 requests 8.6 / 23.6, 6000
// 9.7 / 26.9, 10240 12.6 / 35.2; 16384 only so, 45.7; 65535 of 200 tokens 176).
constexpr int kDirect = 11264;
constexpr int kGroup = 32;
constexpr int kPiece = 512;     // table entries per warp item
constexpr int kAhead = 4;       // requests a thread loads at once
constexpr int kTokPerLane = 4;
constexpr uint32_t kAll = 0xFFFFFFFFu;

struct Req {
  int cached, fresh;  // tokens; both 0 for a refused request
  int tokens;         // rows in the packed batch (fresh, or the refused request's count)
  int old, need;      // pages
  int row;            // row of the source table
  bool ok;
};

struct Raw {
  int c, n, row;
};
__device__ __forceinline__ Raw load_raw(const TablesParams& p, int b) {
  return Raw{p.cached_lens ? p.cached_lens[b] : 0, p.new_lens[b], p.src_rows ? p.src_rows[b] : b};
}
__device__ __forceinline__ Req make_req(const TablesParams& p, const Raw& x) {
  Req r;
  const int c = x.c, n = x.n;
  r.row = x.row;
  r.tokens = max(n, 0);
  // unsigned words hold c + n and c + page_size - 1 of any two counts
  const uint32_t uc = uint32_t(c), total = uc + uint32_t(n), up = uint32_t(p.page_size) - 1;
  const uint32_t old = (uc + up) >> p.page_shift;
  r.ok = c >= 0 && n >= 0 && total <= uint32_t(p.max_blocks) << p.page_shift;
  if (c > 0)
    r.ok = r.ok && p.src_tables != nullptr && uint32_t(r.row) < uint32_t(p.num_src_rows) &&
           old <= uint32_t(p.src_blocks);
  r.cached = r.ok ? c : 0;
  r.fresh = r.ok ? n : 0;
  r.old = r.ok ? int(old) : 0;
  r.need = r.ok ? int(((total + up) >> p.page_shift) - old) : 0;
  return r;
}

__device__ __forceinline__ Req load_req(const TablesParams& p, int b) { return make_req(p, load_raw(p, b)); }

__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(kAll, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

__device__ __forceinline__ int clamp32(int64_t v) { return int(min(v, int64_t(INT32_MAX))); }

// Whether `need` pages after `off` are within the list; off and need <= 2^31 - 1.
__device__ __forceinline__ bool covered(int off, int need, int nfree) {
  return need == 0 || uint32_t(off) + uint32_t(need) <= uint32_t(nfree);
}

// The last entry u in [lo, hi) with pre[u] <= x (pre ascending, pre[lo] <= x).
__device__ __forceinline__ int find_last(const int* pre, int lo, int hi, int x) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Entry b of a shared array, one word skipped per 32: a thread's run of
// consecutive requests starts in a bank of its own.
__device__ __forceinline__ int pad(int b) { return b + (b >> 5); }

// unit: requests per entry of the exclusive sums, 1 or kGroup.
template <int unit>
__global__ void __launch_bounds__(kTabMaxThreads) build_tables_kernel(const TablesParams p) {
  pdl_wait_then_release();
  extern __shared__ int sm[];
  __shared__ int64_t base_tok[kTabMaxThreads / 32], base_page[kTabMaxThreads / 32];
  __shared__ int64_t total_tok;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = blockDim.x, cta_warps = threads >> 5;
  const int B = p.num_seqs;
  const int units = (B + unit - 1) / unit;
  int* pre_tok = sm;                      // [units + 1] tokens before unit u (clamped to int32)
  int* pre_page = pre_tok + units + 1;    // [units + 1] pages before unit u
  int* req_c = pre_page + units + 1;      // with unit 1, by pad(b): cached, new, row as given
  int* req_n = req_c + pad(units) + 1;
  int* req_row = req_n + pad(units) + 1;
  const int nfree_raw = p.num_free ? *p.num_free : p.max_free;

  // ---- exclusive sums: thread t takes the requests [t run, (t + 1) run)
  if (unit == 1) {
    for (int b0 = tid; b0 < B; b0 += kAhead * threads) {
      Raw x[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (b0 + k * threads < B) x[k] = load_raw(p, b0 + k * threads);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int b = b0 + k * threads;
        if (b < B) {
          req_c[pad(b)] = x[k].c;
          req_n[pad(b)] = x[k].n;
          req_row[pad(b)] = x[k].row;
        }
      }
    }
    __syncthreads();
  }
  auto req_of = [&](int b) {
    return make_req(p, unit == 1 ? Raw{req_c[pad(b)], req_n[pad(b)], req_row[pad(b)]} : load_raw(p, b));
  };
  const int run = (units + threads - 1) / threads * unit;
  const int b_lo = int(min(int64_t(B), int64_t(tid) * run)), b_hi = min(B, b_lo + run);
  int64_t ct = 0, cp = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const Req r = req_of(b);
    ct += r.tokens;
    cp += r.need;
  }
  const int64_t ti = warp_scan(ct, lane), gi = warp_scan(cp, lane);
  if (lane == 31) {
    base_tok[warp] = ti;
    base_page[warp] = gi;
  }
  __syncthreads();
  if (warp == 0) {
    const int64_t t = lane < cta_warps ? base_tok[lane] : 0, g = lane < cta_warps ? base_page[lane] : 0;
    const int64_t te = warp_scan(t, lane), ge = warp_scan(g, lane);
    __syncwarp();
    if (lane < cta_warps) {
      base_tok[lane] = te - t;
      base_page[lane] = ge - g;
    }
    if (lane == 31) {
      total_tok = te;
      pre_tok[units] = clamp32(te);
      pre_page[units] = clamp32(ge);
    }
  }
  __syncthreads();
  ct = base_tok[warp] + ti - ct;
  cp = base_page[warp] + gi - cp;
  for (int b = b_lo; b < b_hi; ++b) {
    if (b % unit == 0) {
      pre_tok[b / unit] = clamp32(ct);
      pre_page[b / unit] = clamp32(cp);
      if (unit != 1 && b + unit >= b_hi) break;
    }
    const Req r = req_of(b);
    ct += r.tokens;
    cp += r.need;
  }
  __syncthreads();

  const int nfree = min(max(nfree_raw, 0), p.max_free);
  // warps of the grid, those of one CTA far apart in the order of the work
  const int gw = warp * gridDim.x + blockIdx.x, warps = gridDim.x * cta_warps;

  // ---- per-request words, 32 requests per warp; the pages taken
  for (int b0 = 32 * gw; b0 < B; b0 += 32 * warps) {
    const int b = b0 + lane;
    Req r{};
    if (b < B) r = req_of(b);
    const int64_t t = pre_tok[b0 / unit] + warp_scan(r.tokens, lane);
    const int64_t g = pre_page[b0 / unit] + warp_scan(r.need, lane);
    if (b < B) {
      const bool fits = r.need == 0 || g <= nfree;
      p.cu_q_lens[b + 1] = clamp32(t);
      p.seq_lens[b] = fits ? r.cached + r.fresh : r.cached;
      if (!r.ok) report(p.dev_status, SAW_ERR_DEVICE_INDEX);
      if (!fits) report(p.dev_status, SAW_ERR_DEVICE_PAGES);
    }
  }
  if (blockIdx.x == 0 && warp == cta_warps - 1) {
    if (lane == 0) {
      p.cu_q_lens[0] = 0;
      if (total_tok > p.max_tokens || nfree_raw != nfree) report(p.dev_status, SAW_ERR_DEVICE_INDEX);
    }
    // the largest sum of needs that the list covers lies in the last group
    // of 32 requests that starts within it
    if (p.pages_taken) {
      const int step = kGroup / unit;                 // prefix entries per 32 requests
      const int groups = (B + kGroup - 1) / kGroup;
      int lo = 0, hi = groups;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre_page[mid * step] <= nfree) lo = mid; else hi = mid;
      }
      const int b = lo * kGroup + lane;
      int64_t need = 0;
      if (b < B) need = req_of(b).need;
      const int64_t first = pre_page[lo * step], g = first + warp_scan(need, lane);
      int64_t best = g <= nfree ? g : first;
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) best = max(best, __shfl_xor_sync(kAll, best, d));
      if (lane == 0) *p.pages_taken = int(best);
    }
  }

  // first page of request b in the free list
  auto page_base = [&](int b) -> int {  // whole warp, b uniform
    if constexpr (unit == 1) return pre_page[b];
    const int b0 = b / kGroup * kGroup;
    int64_t n = 0;
    if (b0 + lane < b) n = load_req(p, b0 + lane).need;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) n += __shfl_xor_sync(kAll, n, d);
    return clamp32(pre_page[b / kGroup] + n);
  };
  auto free_page = [&](int i) {  // i < nfree
    const int id = p.free_pages[i];
    if (id >= 0 && id < p.num_pages) return id;
    report(p.dev_status, SAW_ERR_DEVICE_INDEX);
    return -1;
  };

  // ---- table rows, kPiece entries per warp item
  const int pieces = max(1, (p.max_blocks + kPiece - 1) / kPiece);
  const bool in_place = p.block_tables == p.src_tables;
  const int rows_on = warps / pieces, pieces_on = warps % pieces;
  int64_t row = gw / pieces;
  int piece = gw % pieces;
  for (; row < B; row += rows_on, piece += pieces_on) {
    if (piece >= pieces) {
      piece -= pieces;
      if (++row >= B) break;
    }
    const int b = int(row), e0 = piece * kPiece;
    const Req r = req_of(b);
    const int last = r.old + r.need;
    if (e0 >= last || (in_place && e0 + kPiece <= r.old)) continue;
    int off = 0;
    bool fits = true;
    if (r.need > 0 && e0 + kPiece > r.old) {
      off = page_base(b);
      fits = covered(off, r.need, nfree);
    }
    const int32_t* src = p.src_tables + int64_t(r.row) * p.src_blocks;
    int32_t* dst = p.block_tables + int64_t(b) * p.max_blocks;
    int v[kPiece / 32];
    if (!in_place && e0 < r.old) {
#pragma unroll
      for (int k = 0; k < kPiece / 32; ++k)
        if (e0 + 32 * k + lane < r.old) v[k] = src[e0 + 32 * k + lane];
#pragma unroll
      for (int k = 0; k < kPiece / 32; ++k)
        if (e0 + 32 * k + lane < r.old) dst[e0 + 32 * k + lane] = v[k];
    }
    if (fits) {
      const int e1 = min(e0 + kPiece, last);
      for (int e = max(e0, r.old) + lane; e < e1; e += 32) dst[e] = free_page(off + (e - r.old));
    }
  }

  // ---- tokens
  const int total = int(min(total_tok, int64_t(p.max_tokens)));
  const int64_t step = int64_t(warps) * 32 * kTokPerLane;
  // (from the far end of the grid: the near warps have the requests' words)
  for (int64_t t0 = int64_t(warps - 1 - gw) * 32 * kTokPerLane; t0 < p.max_tokens; t0 += step) {
    // the requests of the warp's first and last token bound every lane's search
    const int t_end = int(min(t0 + 32 * kTokPerLane, int64_t(total))) - 1;
    int u_lo = 0, u_hi = 0;
    if (t0 < total) {
      const int u = find_last(pre_tok, 0, units, lane < 16 ? int(t0) : t_end);
      u_lo = __shfl_sync(kAll, u, 0);
      u_hi = __shfl_sync(kAll, u, 31) + 1;
    }
    // each token's place and the word that names its page; then all the words
    const int32_t* word[kTokPerLane];
    int at[kTokPerLane];
#pragma unroll
    for (int k = 0; k < kTokPerLane; ++k) {
      const int64_t t = t0 + 32 * k + lane;
      word[k] = nullptr;
      at[k] = 0;
      if (t >= total) continue;
      int b = find_last(pre_tok, u_lo, u_hi, int(t)) * unit;
      int off = pre_page[b / unit];
      int i = int(t) - pre_tok[b / unit];
      Req r = req_of(b);
      if constexpr (unit != 1) {  // one of 32 holds it
        int64_t pages = off;
        while (i >= r.tokens && b + 1 < B) {
          i -= r.tokens;
          pages += r.need;
          r = load_req(p, ++b);
        }
        off = clamp32(pages);
      }
      if (!r.ok || !covered(off, r.need, nfree)) continue;
      at[k] = r.cached + i;
      const int lp = at[k] >> p.page_shift;
      word[k] = lp < r.old ? p.src_tables + (int64_t(r.row) * p.src_blocks + lp)
                           : p.free_pages + (off + (lp - r.old));
    }
    int id[kTokPerLane];
#pragma unroll
    for (int k = 0; k < kTokPerLane; ++k) id[k] = word[k] ? *word[k] : -1;
#pragma unroll
    for (int k = 0; k < kTokPerLane; ++k) {
      const int64_t t = t0 + 32 * k + lane;
      if (t >= p.max_tokens) break;
      const bool good = id[k] >= 0 && id[k] < p.num_pages;
      if (word[k] && !good) report(p.dev_status, SAW_ERR_DEVICE_INDEX);
      p.slot_mapping[t] = good ? (id[k] << p.page_shift) + (at[k] & (p.page_size - 1)) : -1;
      if (p.positions) p.positions[t] = at[k];
    }
  }
}

}  // namespace

cudaError_t launch_build_tables(const TablesParams& p, int sms, cudaStream_t stream) {
  const int unit = p.num_seqs <= kDirect ? 1 : kGroup;
  const int units = (p.num_seqs + unit - 1) / unit;
  constexpr auto bytes = [](int unit, int units) {
    return (2 * (units + 1) + (unit == 1 ? 3 * (units + units / 32 + 1) : 0)) * int(sizeof(int));
  };
  const int smem = bytes(unit, units);
  // the kernel's static arrays, 520 bytes, count towards the first 48 KB too
  constexpr int kFree = 47 * 1024;
  static_assert(bytes(kGroup, (65535 + kGroup - 1) / kGroup) <= kFree, "no attribute for the grouped form");
  const auto kernel = unit == 1 ? &build_tables_kernel<1> : &build_tables_kernel<kGroup>;
  if (smem > kFree) {
    // (the most any batch takes: the attribute is the process's, and a call of
    // another thread between this line and the launch must not lower it)
    const cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(1, kDirect));
    if (err != cudaSuccess) return err;
  }
  // a warp for every row piece or 128 tokens, at most one full CTA per SM
  const int64_t pieces = int64_t(p.num_seqs) * ((p.max_blocks + kPiece - 1) / kPiece);
  const int64_t tok = (int64_t(p.max_tokens) + 32 * kTokPerLane - 1) / (32 * kTokPerLane);
  const int64_t items = pieces > tok ? pieces : tok;
  // (256 threads start and synchronise sooner, 1024 have more work in flight: 64
  // requests 4.0 / 4.8 us, 300 with 256 new tokens each 5.2 / 6.1, 512 short ones
  // 5.8 / 7.3, 1000 7.9 / 6.9, 4096 26.6 / 12.9)
  const int threads = items > 24 * sms ? kTabMaxThreads : 256;
  const int64_t want = (items + threads / 32 - 1) / (threads / 32);
  const int grid = int(want < 1 ? 1 : want > sms ? sms : want);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace saw
