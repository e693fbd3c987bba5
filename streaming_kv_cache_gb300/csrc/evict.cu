// Eviction from the paged cache: which tokens of every (layer, request, kv
// head) over its budget stay (kv_evict_plan), and the rows of those that lie
// behind the budget into the places that become free (kv_evict_move).
//
// Keys are rotated when they are written and the attention does not look at
// the order of cached keys, so what stays need not move together: only the
// kept tokens behind the first `keep` places move, into places of tokens that
// go.  Sources and destinations are apart, every move is independent, and a
// request that is one token over its budget moves one row of each kv head.
#include "common.cuh"
#include "evict.h"
#include "skv.h"
#include "tc.cuh"

namespace skv {

namespace {

// Where token j of a request lies in a layer's pool of [page][kv head][row].
struct Place {
  const int32_t* row;     // the request's block table row
  int page_size, Hkv, h, n_page;
  uint32_t ps_m;
  // index of the token's entry, -1 with its page outside the pool
  __device__ __forceinline__ long long operator()(int j) const {
    int r;
    const int page = row[fastdiv(j, page_size, ps_m, r)];
    return page >= 0 && page < n_page ? ((long long)page * Hkv + h) * page_size + r : -1;
  }
};

__device__ __forceinline__ Place place_of(const EvictArgs& a, int b, int h) {
  return Place{a.table + (size_t)b * a.max_block, a.page_size, a.Hkv, h, a.n_page, a.ps_m};
}

// tokens that a request holds: 0 with a length out of range
__device__ __forceinline__ int held_tokens(const EvictArgs& a, int b, bool& bad) {
  const int m = a.kv_len[b];
  bad = m < 0 || m > min((long long)a.max_block * a.page_size, (long long)kMaxKeys);
  return bad ? 0 : m;
}

// ---------------------------------------------------------------------------
// Plan.  A token's key orders what stays: protected tokens (the first and the
// most recent positions) above all others, then by score; equal keys go to
// the lowest index.  The keep-th largest key is found digit by digit, 8 bits
// at a time, from histograms; then one pass in index order tells kept tokens
// from the others and numbers the free places and the tokens that move.

constexpr int ET = 512;

// order of floats as unsigned numbers; -0 as 0, NaN below all
__device__ __forceinline__ uint32_t order_of(float s) {
  if (s != s) return 0;
  const uint32_t u = __float_as_uint(s + 0.f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(ET) evict_plan_kernel(const EvictArgs a) {
  __shared__ int s_hist[256];
  __shared__ int s_sum[3][ET / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_rank;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % a.Hkv, b = blockIdx.x / a.Hkv % a.n_req, layer = blockIdx.x / a.Hkv / a.n_req;
  tc::grid_dep_wait();
  bool bad;
  const int m = held_tokens(a, b, bad), keep = a.keep[b];
  const int gone = a.evicted ? a.evicted[b] : 0;
  if ((bad || keep < 0 || gone < 0) && tid == 0 && h == 0 && layer == 0) set_status(a.status, SKV_DEV_BAD_LEN);
  int32_t* n_move = a.n_move + ((size_t)layer * a.n_req + b) * a.Hkv + h;
  if (keep <= 0 || m <= keep) {          // all stay, or none
    if (tid == 0) *n_move = 0;
    return;
  }
  const Place place = place_of(a, b, h);
  const size_t pool = (size_t)layer * a.n_page * a.Hkv * a.page_size;
  const float* score = a.score + pool;
  const int32_t* pos = a.pos + pool;
  int32_t* move = a.move + pool;
  const long long next = (long long)max(gone, 0) + m;      // the next token's position
  auto key = [&](int j) -> uint32_t {
    const long long at = place(j);
    if (at < 0) return 0;
    const int p = pos[at];
    return p < a.n_sink || (p >= next - a.n_recent && p < next) ? 0xFFFFFFFFu : order_of(score[at]);
  };
  // the keep-th largest key: `prefix` its digits so far, `rank` its rank among
  // the keys that share them
  uint32_t prefix = 0;
  int rank = keep;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += ET) s_hist[i] = 0;
    __syncthreads();
    for (int j = tid; j < m; j += ET) {
      const uint32_t k = key(j);
      if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&s_hist[k >> shift & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // digits from the top, 8 to a lane
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += c[i] = s_hist[255 - (lane * 8 + i)];
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      int above = incl - sum;
      if (above < rank && incl >= rank) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (above < rank && above + c[i] >= rank) {
            s_prefix = prefix << 8 | (255 - (lane * 8 + i));
            s_rank = rank - above;
          }
          above += c[i];
        }
      }
    }
    __syncthreads();
    prefix = s_prefix;
    rank = s_rank;
  }
  // in index order: of the keys equal to the keep-th largest the first `rank`
  // stay; free places and moving tokens in ascending order
  int eq0 = 0, hole0 = 0, come0 = 0;     // before this round's tokens
  bool lost = false;                     // a page outside the pool
  for (int j0 = 0; j0 < m; j0 += ET) {
    const int j = j0 + tid;
    const bool in = j < m;
    const uint32_t k = in ? key(j) : 0;
    const bool eq = in && k == prefix;
    const uint32_t me = __ballot_sync(0xffffffffu, eq);
    const uint32_t before = (1u << lane) - 1;
    if (lane == 0) s_sum[0][warp] = __popc(me);
    __syncthreads();
    int eq_at = eq0 + __popc(me & before), eq_all = 0;
    for (int w = 0; w < ET / 32; ++w) {
      if (w < warp) eq_at += s_sum[0][w];
      eq_all += s_sum[0][w];
    }
    const bool kept = in && (k > prefix || (eq && eq_at < rank));
    const bool hole = in && j < keep && !kept, come = in && j >= keep && kept;
    const uint32_t mh = __ballot_sync(0xffffffffu, hole), mc = __ballot_sync(0xffffffffu, come);
    if (lane == 0) {
      s_sum[1][warp] = __popc(mh);
      s_sum[2][warp] = __popc(mc);
    }
    __syncthreads();
    int hole_at = hole0 + __popc(mh & before), come_at = come0 + __popc(mc & before);
    for (int w = 0; w < ET / 32; ++w) {
      if (w < warp) {
        hole_at += s_sum[1][w];
        come_at += s_sum[2][w];
      }
      hole0 += s_sum[1][w];
      come0 += s_sum[2][w];
    }
    eq0 += eq_all;
    if (hole || come) {
      const long long at = place(hole ? 2 * hole_at : 2 * come_at + 1);
      if (at >= 0) move[at] = j;
    }
    lost |= in && place(j) < 0;
    __syncthreads();
  }
  if (__syncthreads_or(lost) && tid == 0) set_status(a.status, SKV_DEV_BAD_PAGE);
  if (tid == 0) *n_move = come0;
}

// ---------------------------------------------------------------------------
// Move.  D / 8 lanes take 16 bytes of a row each, of its key and its value;
// bound by HBM.

constexpr int MT = 256;

template <int D>
__global__ void __launch_bounds__(MT) evict_move_kernel(const EvictArgs a) {
  constexpr int LANES = D / 8, PER = MT / LANES;     // moves that a CTA has in flight
  const int unit = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
  const int h = unit % a.Hkv, b = unit / a.Hkv % a.n_req, layer = unit / a.Hkv / a.n_req;
  const int c = threadIdx.x % LANES, sub = threadIdx.x / LANES;
  tc::grid_dep_wait();
  bool bad;
  const int m = held_tokens(a, b, bad);
  int n = a.n_move[((size_t)layer * a.n_req + b) * a.Hkv + h];
  bad |= n < 0 || n > m / 2;
  if (bad) {
    if (part == 0 && threadIdx.x == 0) set_status(a.status, SKV_DEV_BAD_LEN);
    return;
  }
  const Place place = place_of(a, b, h);
  const size_t pool = (size_t)layer * a.n_page * a.Hkv * a.page_size;
  const int32_t* move = a.move + pool;
  uint4* k = reinterpret_cast<uint4*>(a.k) + pool * LANES;
  uint4* v = reinterpret_cast<uint4*>(a.v) + pool * LANES;
  for (int i = part * PER + sub; i < n; i += a.parts * PER) {
    const long long at = place(2 * i);
    int2 p = make_int2(0, 0);
    if (at >= 0) p = *reinterpret_cast<const int2*>(move + at);
    if (p.x < 0 || p.x >= m || p.y < 0 || p.y >= m) {
      if (c == 0) set_status(a.status, SKV_DEV_BAD_LEN);
      continue;
    }
    const long long to = place(p.x), from = place(p.y);
    if (at < 0 || to < 0 || from < 0) {
      if (c == 0) set_status(a.status, SKV_DEV_BAD_PAGE);
      continue;
    }
    k[to * LANES + c] = k[from * LANES + c];
    v[to * LANES + c] = v[from * LANES + c];
    if (c == 0) {
      a.score[pool + to] = a.score[pool + from];
      a.pos[pool + to] = a.pos[pool + from];
    }
  }
}

}  // namespace

cudaError_t launch_evict_plan(const EvictArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)a.n_layer * a.n_req * a.Hkv;
  return launch_dependent(evict_plan_kernel, dim3(grid), ET, 0, st, a);
}

cudaError_t launch_evict_move(const EvictArgs& a, int d, cudaStream_t st) {
  EvictArgs p = a;
  p.parts = 8;
  const unsigned grid = (unsigned)a.n_layer * a.n_req * a.Hkv * p.parts;
  auto launch = [&](auto kernel) { return launch_dependent(kernel, dim3(grid), MT, 0, st, p); };
  return d == 128 ? launch(evict_move_kernel<128>) : launch(evict_move_kernel<64>);
}

}  // namespace skv
