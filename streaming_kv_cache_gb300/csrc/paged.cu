// The paged cache's bookkeeping and writes: block tables, slot maps and free
// pages of a step from the requests' lengths (kv_paged_plan), and a step's
// keys and values into their pages with the rotary embedding of q and k
// (kv_paged_write).
#include <atomic>

#include "common.cuh"
#include "ragged.h"
#include "skv.h"
#include "tc.cuh"

namespace skv {

namespace {

// ---------------------------------------------------------------------------
// Plan.  Three running sums over the requests (new tokens, pages needed,
// pages given back) decide everything; what is left is one independent item
// per token, per new page and per page given back.  A grid-wide scan would
// need a second launch or a barrier, so every CTA repeats the scan over all
// requests (a few loads per thread, all CTAs at once out of L2) into its own
// shared memory and then takes its part of the items, each of which finds its
// request by bisection there.  Bound by latency: launch, one load round trip
// for the lengths, one for the state of an item (8 requests 4.3 us, 2,048
// requests with 64 chunks of 1,024 tokens 8.2 us).  Sums saturate (lengths are
// caller data): a sum past its cap already means "does not fit".

constexpr int PT = 512;                      // threads per CTA

// exclusive sums of K arrays v[k][0 .. n) in shared memory, in place, with the
// totals in v[k][n]; sums saturate at cap
template <int K>
__device__ void block_scan(int* const (&v)[K], int n, int cap, int (*warp_sum)[PT / 32]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + PT - 1) / PT;
  const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
  auto add = [&](int a, int b) { return a > cap - b ? cap : a + b; };
  int incl[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    int s = 0;
    for (int i = i0; i < i1; ++i) s = add(s, v[k][i]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s = add(s, t);
    }
    incl[k] = s;
    if (lane == 31) warp_sum[k][warp] = s;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    // every warp adds up the warps' sums for itself, a lane each
    static_assert(PT / 32 <= 32, "a lane per warp");
    int s = lane < PT / 32 ? warp_sum[k][lane] : 0;
#pragma unroll
    for (int o = 1; o < PT / 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s = add(s, t);
    }
    const int total = __shfl_sync(0xffffffffu, s, PT / 32 - 1);
    const int base = warp ? __shfl_sync(0xffffffffu, s, warp - 1) : 0;
    // sums before this thread's items: those of its warp's earlier lanes too
    int excl = __shfl_up_sync(0xffffffffu, incl[k], 1);
    if (lane == 0) excl = 0;
    int run = add(base, excl);
    for (int i = i0; i < i1; ++i) {
      const int x = v[k][i];
      v[k][i] = run;
      run = add(run, x);
    }
    if (tid == 0) v[k][n] = total;
  }
  __syncthreads();
}

// the request whose span of the running sums holds x (sums[0] <= x < sums[n])
__device__ __forceinline__ int find_request(const int* sums, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sums[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(PT) paged_plan_kernel(const PlanArgs a) {
  extern __shared__ int sm[];
  const int n = a.n_req;
  int* s_tok = sm;                 // running sums of the new tokens
  int* s_need = s_tok + n + 1;     // of the pages needed
  int* s_back = s_need + n + 1;    // of the pages given back
  int* s_ctx = s_back + n + 1;     // tokens held (-1: left out altogether)
  int* s_new = s_ctx + n;          // new_len
  __shared__ int warp_sum[2][PT / 32];
  const int tid = threadIdx.x;
  const uint32_t ps = (uint32_t)a.page_size;
  const int row_tokens = (int)min((long long)a.max_block * ps, (long long)kMaxKeys);   // what a request may hold
  // 32-bit quotients by multiply-high throughout: x and page_size are below 2^31
  auto pages = [&](int x) {
    int rem;
    const int q = fastdiv(x, (int)ps, a.ps_m, rem);
    return q + (rem > 0);
  };
  const bool reporter = blockIdx.x == 0;
  tc::grid_dep_wait();

  int head = a.state[n], count = a.state[n + 1];
  for (int b = tid; b < n; b += PT) {
    const int c = a.state[b], w = a.new_len[b];
    const bool bad = c < 0 || c > row_tokens || w < -1;
    if (bad && reporter) set_status(a.status, SKV_DEV_BAD_LEN);
    s_ctx[b] = bad ? -1 : c;
    s_new[b] = w;
    s_tok[b] = bad ? 0 : max(w, 0);
    s_back[b] = !bad && w == -1 ? pages(c) : 0;
  }
  if (head < 0 || head >= a.n_page || count < 0 || count > a.n_page) {
    head = 0;
    count = 0;
    if (reporter && tid == 0) set_status(a.status, SKV_DEV_BAD_LEN);
  }
  __syncthreads();
  {
    // token sums go one past the rows there are; a span that ends there does not fit
    int* const v[1] = {s_tok};
    block_scan<1>(v, n, a.n_tok + 1, warp_sum);
  }
  for (int b = tid; b < n; b += PT) {
    const int c = s_ctx[b], w = s_new[b];
    int need = 0;
    if (c >= 0 && w > 0) {
      const bool fits = s_tok[b + 1] <= a.n_tok && (long long)c + w <= row_tokens;
      if (!fits && reporter) set_status(a.status, SKV_DEV_TABLE_FULL);
      need = fits ? pages(c + w) - pages(c) : 0;
    }
    s_need[b] = need;
  }
  __syncthreads();
  {
    int* const v[2] = {s_need, s_back};
    block_scan<2>(v, n, 0x7FFFFFFF, warp_sum);
  }

  // A request is planned if its rows, its table and the free pages hold it.
  // The sums of the needs only grow, so the requests that get pages are those
  // before the first that does not fit, and the pages given out are [0, given).
  auto planned = [&](int b, int c, int w) {
    return c >= 0 && (w == 0 || (w > 0 && s_tok[b + 1] <= a.n_tok && (long long)c + w <= row_tokens &&
                                 (s_need[b + 1] == s_need[b] || s_need[b + 1] <= count)));
  };
  int given = s_need[n];   // the largest running sum of the needs that the queue covers
  if (given > count) {
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_need[mid] <= count) lo = mid;
      else hi = mid - 1;
    }
    given = s_need[lo];
  }
  const int room = a.n_page - count;               // a consistent state gives back at most this
  const int back = min(s_back[n], room);
  // entry i of the queue, i < 2 n_page - head
  auto ring = [&](uint32_t i) {
    i += (uint32_t)head;
    return i >= (uint32_t)a.n_page ? i - (uint32_t)a.n_page : i;
  };
  if (reporter && tid == 0) {
    if (s_need[n] > count) set_status(a.status, SKV_DEV_NO_PAGE);
    if (s_back[n] > room) set_status(a.status, SKV_DEV_BAD_LEN);
    a.q_start[n] = min(s_tok[n], a.n_tok);
    a.next_state[n] = (int)ring((uint32_t)given);
    a.next_state[n + 1] = count - given + back;
  }
  const int stride = gridDim.x * PT, first = blockIdx.x * PT + tid;
  for (int t = first; t < a.n_tok; t += stride) {
    int pos = 0, slot = -1;
    if (t < s_tok[n]) {
      const int b = find_request(s_tok, n, t), c = s_ctx[b], w = s_tok[b + 1] - s_tok[b];
      const long long p = (long long)c + (t - s_tok[b]);
      pos = (int)min(p, 0x7FFFFFFFLL);
      if (planned(b, c, w)) {
        int r;
        const int j = fastdiv(pos, (int)ps, a.ps_m, r), old = pages(c);
        // a new page comes straight from the queue: its table entry may be
        // another CTA's to write
        const int page = j < old ? a.table[(size_t)b * a.max_block + j] : a.queue[ring((uint32_t)(s_need[b] + j - old))];
        if (page >= 0 && page < a.n_page) slot = page * (int)ps + r;
        else set_status(a.status, SKV_DEV_BAD_PAGE);
      }
    }
    a.position[t] = pos;
    a.slot[t] = slot;
  }
  for (int b = first; b < n; b += stride) {
    const int c = s_ctx[b], w = s_new[b];
    a.q_start[b] = min(s_tok[b], a.n_tok);
    const bool ok = planned(b, c, w);
    a.kv_len[b] = ok ? c + w : 0;
    a.next_state[b] = c >= 0 && w == -1 ? 0 : ok ? c + w : c >= 0 ? c : a.state[b];
  }
  for (int i = first; i < given; i += stride) {
    const int b = find_request(s_need, n, i);
    a.table[(size_t)b * a.max_block + pages(s_ctx[b]) + (i - s_need[b])] = a.queue[ring((uint32_t)i)];
  }
  // The tail's entries are none of the count that the loops above read.
  for (int i = first; i < back; i += stride) {
    const int b = find_request(s_back, n, i);
    a.queue[ring((uint32_t)(count + i))] = a.table[(size_t)b * a.max_block + (i - s_back[b])];
  }
}

// ---------------------------------------------------------------------------
// Write.  One thread takes 16-byte chunk c of the first half of a head and
// its partner in the second half, for RPT rows (heads) of one token: the
// chunk's eight angles are loaded once for all of them, and a token's rows are
// spread over threads so that a decode step of a few tokens still fills more
// than one warp.  All 2 RPT loads are out before the first store.  Bound by
// HBM: every value is read and written once (16,384 tokens of 32 query and 8 kv
// heads of 128: 66 us, 6.2 TB/s).

constexpr int WT = 256;
constexpr int RPT = 4;      // rows per thread

__device__ __forceinline__ float f16_lo(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu))); }
__device__ __forceinline__ float f16_hi(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }

// x' = x cos - y sin, y' = y cos + x sin for 8 pairs, in fp32, rounded once
template <bool F16>
__device__ __forceinline__ void rotate_chunk(uint4& a, uint4& b, const float4 (&t)[4]) {
  uint32_t* pa = reinterpret_cast<uint32_t*>(&a);
  uint32_t* pb = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float x0 = F16 ? f16_lo(pa[w]) : bf16_lo(pa[w]), x1 = F16 ? f16_hi(pa[w]) : bf16_hi(pa[w]);
    const float y0 = F16 ? f16_lo(pb[w]) : bf16_lo(pb[w]), y1 = F16 ? f16_hi(pb[w]) : bf16_hi(pb[w]);
    const float r0 = x0 * t[w].x - y0 * t[w].y, r1 = x1 * t[w].z - y1 * t[w].w;
    const float s0 = y0 * t[w].x + x0 * t[w].y, s1 = y1 * t[w].z + x1 * t[w].w;
    if constexpr (F16) {
      const __half2 r = __floats2half2_rn(r0, r1), s = __floats2half2_rn(s0, s1);
      pa[w] = *reinterpret_cast<const uint32_t*>(&r);
      pb[w] = *reinterpret_cast<const uint32_t*>(&s);
    } else {
      pa[w] = pack_bf16x2(r0, r1);
      pb[w] = pack_bf16x2(s0, s1);
    }
  }
}

template <int D, bool F16>
__global__ void __launch_bounds__(WT) paged_write_kernel(const WriteArgs a) {
  constexpr int NCH = D / 16;                       // chunks of half a head
  const int hq = a.q ? a.Hq : 0;                    // rows of a token: q heads, k heads, v heads
  const int rows = hq + 2 * a.Hkv, groups = (rows + RPT - 1) / RPT;
  const long long item = blockIdx.x * (long long)WT + threadIdx.x;
  const int c = (int)(item % NCH);
  const long long rest = item / NCH;
  const int grp = (int)(rest % groups);
  const long long tok = rest / groups;
  tc::grid_dep_wait();
  if (tok >= a.n_tok) return;
  const int slot = a.slot[tok];
  if (slot < 0) return;
  int row_in;
  const int page = fastdiv(slot, a.page_size, a.ps_m, row_in);
  const bool first = grp == 0 && c == 0;
  if (page >= a.n_page) {
    if (first) set_status(a.status, SKV_DEV_BAD_PAGE);
    return;
  }
  float4 t[4];
  if (a.rope) {
    const int pos = a.position[tok];
    if (pos < 0 || pos >= a.rope_len) {
      if (first) set_status(a.status, SKV_DEV_BAD_POS);
      return;
    }
    const float4* r4 = reinterpret_cast<const float4*>(a.rope) + ((size_t)pos * (D / 2) + c * 8) / 2;
#pragma unroll
    for (int w = 0; w < 4; ++w) t[w] = r4[w];
  }
  uint4 x[RPT], y[RPT];
  uint16_t* dst[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = grp * RPT + i;
    const uint16_t* src = nullptr;
    dst[i] = nullptr;
    if (r < hq) {
      src = a.q + tok * a.q_stride + (size_t)r * D;
      dst[i] = a.q_out + ((size_t)tok * a.Hq + r) * D;
    } else if (r < rows) {
      const bool is_k = r < hq + a.Hkv;
      const int h = is_k ? r - hq : r - hq - a.Hkv;
      src = (is_k ? a.k + tok * a.k_stride : a.v + tok * a.v_stride) + (size_t)h * D;
      dst[i] = (is_k ? a.k_pages : a.v_pages) + (((size_t)page * a.Hkv + h) * a.page_size + row_in) * D;
    }
    if (src) {
      x[i] = *reinterpret_cast<const uint4*>(src + c * 8);
      y[i] = *reinterpret_cast<const uint4*>(src + D / 2 + c * 8);
    }
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    if (!dst[i]) continue;
    if (a.rope && grp * RPT + i < hq + a.Hkv) rotate_chunk<F16>(x[i], y[i], t);
    *reinterpret_cast<uint4*>(dst[i] + c * 8) = x[i];
    *reinterpret_cast<uint4*>(dst[i] + D / 2 + c * 8) = y[i];
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t st) {
  // A thread per token, request and page that finished requests may give back
  // (which the host does not know: all that they can hold).  CTAs without items
  // cost nothing to speak of (64 single tokens over a pool of 100,000 pages 3.8
  // us with one CTA, 3.9 with 152); too few made a step in which 8 requests of
  // 131,072 tokens finish 43 us, 3.5 so.
  const long long pages = min((long long)a.n_page, (long long)a.n_req * a.max_block);
  const long long items = max(max((long long)a.n_tok, (long long)a.n_req), pages);
  const long long want = (items + PT - 1) / PT;
  const int grid = (int)min(want > 0 ? want : 1LL, 152LL);
  const int smem = (5 * a.n_req + 3) * (int)sizeof(int);
  static std::atomic<int> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (smem > 48 * 1024 && !(dev >= 0 && dev < 64 && done[dev].load(std::memory_order_relaxed))) {
    e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (5 * SKV_PAGED_MAX_REQUESTS + 3) * (int)sizeof(int));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev].store(1, std::memory_order_relaxed);
  }
  return launch_dependent(paged_plan_kernel, dim3(grid), PT, smem, st, a);
}

cudaError_t launch_paged_write(const WriteArgs& a, int d, bool f16, cudaStream_t st) {
  const int rows = (a.q ? a.Hq : 0) + 2 * a.Hkv;
  const long long items = (long long)a.n_tok * ((rows + RPT - 1) / RPT) * (d / 16);
  const long long blocks = (items + WT - 1) / WT;
  if (blocks <= 0) return cudaSuccess;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  auto launch = [&](auto kernel) { return launch_dependent(kernel, dim3((unsigned)blocks), WT, 0, st, a); };
  if (d == 128) return f16 ? launch(paged_write_kernel<128, true>) : launch(paged_write_kernel<128, false>);
  return f16 ? launch(paged_write_kernel<64, true>) : launch(paged_write_kernel<64, false>);
}

}  // namespace skv
