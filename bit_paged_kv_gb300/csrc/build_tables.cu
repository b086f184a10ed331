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
// exclusive sums (tokens, pages) over all requests itself -- each warp a
// contiguous run of requests with coalesced loads, then one scan over the 16
// warps' totals -- and keeps them in shared memory, one entry per request (per
// 32 requests above kDirect).  That is 8 bytes per request and CTA from L2,
// against a second launch or a look-back between CTAs.  Then the grid shares
// out (request, 256 entries) pieces of table rows to warps and the tokens to
// threads, each token finding its request by bisection in shared memory.
#include "saw_device.cuh"
#include "saw_int4.h"
#include "saw_quant_row.cuh"

namespace saw {
namespace {

constexpr int kTabThreads = 512;
constexpr int kTabWarps = kTabThreads / 32;
constexpr int kDirect = 4096;   // up to this many requests: one prefix entry per request
constexpr int kGroup = 32;      // above: one per 32
constexpr int kPiece = 256;     // table entries per warp item
constexpr int kTokPerLane = 4;
constexpr uint32_t kAll = 0xFFFFFFFFu;

struct Req {
  int cached, fresh;  // tokens; both 0 for a refused request
  int tokens;         // rows in the packed batch (fresh, or the refused request's count)
  int old, need;      // pages
  int row;            // row of the source table
  bool ok;
};

__device__ __forceinline__ Req load_req(const TablesParams& p, int b) {
  Req r;
  const int c = p.cached_lens ? p.cached_lens[b] : 0;
  const int n = p.new_lens[b];
  r.row = p.src_rows ? p.src_rows[b] : b;
  r.tokens = max(n, 0);
  const int64_t total = int64_t(c) + n;
  r.ok = c >= 0 && n >= 0 && total <= (int64_t(p.max_blocks) << p.page_shift);
  if (r.ok && c > 0)
    r.ok = p.src_tables != nullptr && r.row >= 0 && r.row < p.num_src_rows &&
           ((int64_t(c) + p.page_size - 1) >> p.page_shift) <= p.src_blocks;
  r.cached = r.ok ? c : 0;
  r.fresh = r.ok ? n : 0;
  r.old = int((int64_t(r.cached) + p.page_size - 1) >> p.page_shift);
  r.need = int((int64_t(r.cached) + r.fresh + p.page_size - 1) >> p.page_shift) - r.old;
  return r;
}

__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(kAll, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

__device__ __forceinline__ int clamp32(int64_t v) { return int(min(v, int64_t(INT32_MAX))); }

// The last entry u in [0, n) with pre[u] <= x (pre ascending, pre[0] = 0).
__device__ __forceinline__ int find_last(const int* pre, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTabThreads) build_tables_kernel(const TablesParams p) {
  pdl_wait_then_release();
  extern __shared__ int sm[];
  __shared__ int64_t base_tok[kTabWarps], base_page[kTabWarps];
  __shared__ int64_t total_tok;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.num_seqs;
  const int unit = B <= kDirect ? 1 : kGroup;
  const int units = (B + unit - 1) / unit;
  int* pre_tok = sm;            // [units + 1] tokens before unit u (clamped to int32)
  int* pre_page = sm + units + 1;

  // ---- exclusive sums: warp w takes requests [w run, (w + 1) run)
  const int run = ((B + kTabWarps - 1) / kTabWarps + 31) / 32 * 32;
  const int b_lo = min(B, warp * run), b_hi = min(B, b_lo + run);
  int64_t ct = 0, cp = 0;
  for (int b0 = b_lo; b0 < b_hi; b0 += 32) {
    const int b = b0 + lane;
    int64_t t = 0, g = 0;
    if (b < b_hi) {
      const Req r = load_req(p, b);
      t = r.tokens;
      g = r.need;
    }
    const int64_t ti = warp_scan(t, lane), gi = warp_scan(g, lane);
    if (b < b_hi && b % unit == 0) {
      pre_tok[b / unit] = clamp32(ct + ti - t);
      pre_page[b / unit] = clamp32(cp + gi - g);
    }
    ct += __shfl_sync(kAll, ti, 31);
    cp += __shfl_sync(kAll, gi, 31);
  }
  if (lane == 0) {
    base_tok[warp] = ct;
    base_page[warp] = cp;
  }
  __syncthreads();
  if (warp == 0) {
    const int64_t t = lane < kTabWarps ? base_tok[lane] : 0, g = lane < kTabWarps ? base_page[lane] : 0;
    const int64_t ti = warp_scan(t, lane), gi = warp_scan(g, lane);
    __syncwarp();
    if (lane < kTabWarps) {
      base_tok[lane] = ti - t;
      base_page[lane] = gi - g;
    }
    if (lane == kTabWarps - 1) {
      total_tok = ti;
      pre_tok[units] = clamp32(ti);
      pre_page[units] = clamp32(gi);
    }
  }
  __syncthreads();
  for (int u = tid; u < units; u += kTabThreads) {
    const int w = u * unit / run;
    pre_tok[u] = clamp32(pre_tok[u] + base_tok[w]);
    pre_page[u] = clamp32(pre_page[u] + base_page[w]);
  }
  __syncthreads();

  const int nfree_raw = p.num_free ? *p.num_free : p.max_free;
  const int nfree = min(max(nfree_raw, 0), p.max_free);
  const int gw = blockIdx.x * kTabWarps + warp, warps = gridDim.x * kTabWarps;

  // ---- per-request words, 32 requests per warp; the pages taken
  for (int b0 = 32 * gw; b0 < B; b0 += 32 * warps) {
    const int b = b0 + lane;
    Req r{};
    if (b < B) r = load_req(p, b);
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
  if (blockIdx.x == 0 && warp == 0) {
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
      if (b < B) need = load_req(p, b).need;
      const int64_t first = pre_page[lo * step], g = first + warp_scan(need, lane);
      int64_t best = g <= nfree ? g : first;
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) best = max(best, __shfl_xor_sync(kAll, best, d));
      if (lane == 0) *p.pages_taken = int(best);
    }
  }

  // first page of request b in the free list
  auto page_base = [&](int b) -> int64_t {  // whole warp, b uniform
    if (unit == 1) return pre_page[b];
    const int b0 = b / kGroup * kGroup;
    int64_t n = 0;
    if (b0 + lane < b) n = load_req(p, b0 + lane).need;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) n += __shfl_xor_sync(kAll, n, d);
    return pre_page[b / kGroup] + n;
  };
  auto free_page = [&](int64_t i) {  // i < nfree
    const int id = p.free_pages[i];
    if (id >= 0 && id < p.num_pages) return id;
    report(p.dev_status, SAW_ERR_DEVICE_INDEX);
    return -1;
  };

  // ---- table rows, kPiece entries per warp item
  const int pieces = (p.max_blocks + kPiece - 1) / kPiece;
  const bool in_place = p.block_tables == p.src_tables;
  for (int64_t it = gw; it < int64_t(B) * pieces; it += warps) {
    const int b = int(it / pieces), e0 = int(it % pieces) * kPiece;
    const Req r = load_req(p, b);
    const int last = r.old + r.need;
    if (e0 >= last || (in_place && e0 + kPiece <= r.old)) continue;
    int64_t off = 0;
    bool fits = true;
    if (r.need > 0 && e0 + kPiece > r.old) {
      off = page_base(b);
      fits = off + r.need <= nfree;
    }
    const int32_t* src = p.src_tables + int64_t(r.row) * p.src_blocks;
    int32_t* dst = p.block_tables + int64_t(b) * p.max_blocks;
    int v[kPiece / 32];
#pragma unroll
    for (int k = 0; k < kPiece / 32; ++k) {
      const int e = e0 + 32 * k + lane;
      if (e < r.old) {
        v[k] = in_place ? 0 : src[e];
      } else if (e < last && fits) {
        v[k] = free_page(off + e - r.old);
      }
    }
#pragma unroll
    for (int k = 0; k < kPiece / 32; ++k) {
      const int e = e0 + 32 * k + lane;
      if (e < r.old ? !in_place : (e < last && fits)) dst[e] = v[k];
    }
  }

  // ---- tokens
  const int total = int(min(total_tok, int64_t(p.max_tokens)));
  const int64_t step = int64_t(warps) * 32 * kTokPerLane;
  for (int64_t t0 = int64_t(gw) * 32 * kTokPerLane; t0 < p.max_tokens; t0 += step) {
#pragma unroll
    for (int k = 0; k < kTokPerLane; ++k) {
      const int64_t t64 = t0 + 32 * k + lane;
      if (t64 >= p.max_tokens) break;
      const int t = int(t64);
      int slot = -1, pos = 0;
      if (t < total) {
        int b = find_last(pre_tok, units, t) * unit;
        int64_t off = pre_page[b / unit];
        Req r;
        int i = t - pre_tok[b / unit];
        if (unit == 1) {
          r = load_req(p, b);
        } else {
          for (;; ++b) {  // within 32 requests (t < total: one of them holds it)
            r = load_req(p, b);
            if (i < r.tokens || b + 1 >= B) break;
            i -= r.tokens;
            off += r.need;
          }
        }
        if (r.ok && (r.need == 0 || off + r.need <= nfree)) {
          const int at = r.cached + i, lp = at >> p.page_shift;
          int id;
          if (lp < r.old) {
            id = p.src_tables[int64_t(r.row) * p.src_blocks + lp];
            if (id < 0 || id >= p.num_pages) {
              report(p.dev_status, SAW_ERR_DEVICE_INDEX);
              id = -1;
            }
          } else {
            id = free_page(off + lp - r.old);
          }
          if (id >= 0) slot = (id << p.page_shift) + (at & (p.page_size - 1));
          pos = at;
        }
      }
      p.slot_mapping[t] = slot;
      if (p.positions) p.positions[t] = pos;
    }
  }
}

}  // namespace

cudaError_t launch_build_tables(const TablesParams& p, int sms, cudaStream_t stream) {
  const int unit = p.num_seqs <= kDirect ? 1 : kGroup;
  const int units = (p.num_seqs + unit - 1) / unit;
  const size_t smem = size_t(2) * (units + 1) * sizeof(int);
  // warps for every row piece and token, at most two CTAs per SM
  const int64_t pieces = int64_t(p.num_seqs) * ((p.max_blocks + kPiece - 1) / kPiece);
  const int64_t tok = (int64_t(p.max_tokens) + 32 * kTokPerLane - 1) / (32 * kTokPerLane);
  const int64_t want = ((pieces > tok ? pieces : tok) + kTabWarps - 1) / kTabWarps;
  const int grid = int(want < 1 ? 1 : want > 2 * sms ? 2 * sms : want);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kTabThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, build_tables_kernel, p);
}

}  // namespace saw
