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
// the lowest index.  The keep-th largest key is found digit by digit, 11, 11
// and 10 bits, from histograms in shared memory; then scans in index order tell
// kept tokens from the others and number the free places and the tokens that
// move.
//
// A cluster per (layer, request, kv head).  A thread takes a run of up to KEYS
// consecutive tokens and keeps their keys in registers, so that scores and
// positions are read once; a CTA takes SLICE tokens at a time.  How many CTAs
// of the cluster take part goes by the request's own length, which the host
// does not know: the others leave at once.  Longer requests than the cluster
// holds go over their tokens again for every digit.
//
// Bound by instructions and by the barriers of a CTA's chain, not by the 8 bytes
// a token: 64 requests one token over 2,048, 4 layers and 8 kv heads, 28 us with table
// rows of up to 4,096 tokens (more with longer ones: launch_evict_plan); four
// prompts of 6 to 12.8 k tokens, 36 layers, 86 us (HBM would take 16).

constexpr int KEYS = 32;
constexpr int BINS = 2048;
constexpr int EVICT_CLUSTER = 8;

// order of floats as unsigned numbers; -0 as 0, NaN below all
__device__ __forceinline__ uint32_t order_of(float s) {
  if (s != s) return 0;
  const uint32_t u = __float_as_uint(s + 0.f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// sum over the threads before this one, and over all
template <int ET>
__device__ __forceinline__ int block_prefix(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int before = incl - v;
  total = 0;
#pragma unroll
  for (int w = 0; w < ET / 32; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  return before;
}

template <int ET>
__global__ void __launch_bounds__(ET, 1024 / ET) evict_plan_kernel(const EvictArgs a) {
  constexpr int SLICE = ET * KEYS;
  __shared__ int s_hist[BINS];
  __shared__ int s_warp[ET / 32];
  __shared__ uint16_t s_list[SLICE];           // tokens of a round, by their offset
  __shared__ int s_cta[2][EVICT_CLUSTER][2];   // of the cluster's CTAs: equal keys; free places and moving tokens
  __shared__ uint32_t s_digit;
  __shared__ int s_rank;
  const int tid = threadIdx.x;
  const int unit = blockIdx.x / a.parts;
  int rank_cta = a.parts > 1 ? (int)tc::cluster_ctarank() : 0;
  const int h = unit % a.Hkv, b = unit / a.Hkv % a.n_req, layer = unit / a.Hkv / a.n_req;
  tc::grid_dep_wait();
  bool bad;
  const int m = held_tokens(a, b, bad), keep = a.keep[b];
  const int gone = a.evicted ? a.evicted[b] : 0;
  if ((bad || keep < 0 || gone < 0) && tid == 0 && rank_cta == 0 && h == 0 && layer == 0) set_status(a.status, SKV_DEV_BAD_LEN);
  int32_t* n_move = a.n_move + ((size_t)layer * a.n_req + b) * a.Hkv + h;
  if (keep <= 0 || m <= keep) {              // all stay, or none
    if (tid == 0 && rank_cta == 0) *n_move = 0;
    return;
  }
  // CTAs that take part: as many as hold the tokens in registers
  const int ctas = min(a.parts, (m + a.per_cta - 1) / a.per_cta);
  if (rank_cta >= ctas) return;
  const Place place = place_of(a, b, h);
  const size_t pool = (size_t)layer * a.n_page * a.Hkv * a.page_size;
  const float* score = a.score + pool;
  const int32_t* pos = a.pos + pool;
  int32_t* move = a.move + pool;
  const long long next = (long long)max(gone, 0) + m;      // the next token's position
  const int safe_lo = (int)min(max(next - a.n_recent, 0LL), 0x7FFFFFFFLL);
  const int safe_hi = (int)min(next, 0x7FFFFFFFLL);
  // this CTA's tokens, and a thread's run of them: a multiple of 4, so that a
  // group of 4 lies in one page
  const int per = (m + ctas - 1) / ctas + 3 & ~3;
  const int t_lo = min((long long)m, (long long)rank_cta * per), t_hi = min(m, t_lo + per);
  const int rounds = max(1, (t_hi - t_lo + SLICE - 1) / SLICE);
  const int run = rounds > 1 ? KEYS : (t_hi - t_lo + ET - 1) / ET + 3 & ~3;
  bool lost = false;                         // a page outside the pool
  uint32_t key[KEYS];
  int j0 = 0;                                // the run's first token
  auto load_keys = [&](int round) {
    j0 = t_lo + round * SLICE + tid * run;
#pragma unroll
    for (int g = 0; g < KEYS / 4; ++g) {
      const int j = j0 + 4 * g;
#pragma unroll
      for (int k = 0; k < 4; ++k) key[4 * g + k] = 0;
      if (4 * g >= run || j >= t_hi) continue;
      const long long at = place(j);
      if (at < 0) {
        lost = true;
        continue;
      }
      const float4 s = *reinterpret_cast<const float4*>(score + at);
      const int4 p = *reinterpret_cast<const int4*>(pos + at);
      const float sv[4] = {s.x, s.y, s.z, s.w};
      const int pv[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool safe = pv[k] < a.n_sink || (pv[k] >= safe_lo && pv[k] < safe_hi);
        key[4 * g + k] = j + k >= t_hi ? 0 : safe ? 0xFFFFFFFFu : order_of(sv[k]);
      }
    }
  };
  // tokens of the run that there are
  auto count = [&]() { return max(0, min(run, t_hi - j0)); };

  // The keep-th largest key: `prefix` its digits so far, `rank` its rank among
  // the keys that share them.  Protected tokens (many of one key, the top bin's
  // only one: the largest score is +inf) are counted without atomics; keys of
  // 0, the lowest, by no bin.
  uint32_t prefix = 0;
  int rank = keep;
  load_keys(0);
#pragma unroll 1
  for (int digit = 0; digit < 3; ++digit) {
    const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0, bits = digit == 2 ? 10 : 11;
    // keys from lo on, span of them: those with the prefix
    const uint32_t lo = digit ? max(prefix << (shift + bits), 1u) : 1u;
    const uint32_t span = digit ? (prefix << (shift + bits)) + (1u << (shift + bits)) - lo : 0xFFFFFFFEu;
    const uint32_t mask = ((1u << bits) - 1) << 2;
    for (int i = tid; i < BINS; i += ET) s_hist[i] = 0;
    __syncthreads();
    const uint32_t hist = tc::smem_u32(s_hist);
    int top = 0;
    for (int round = 0; round < rounds; ++round) {
      if (rounds > 1) load_keys(round);
#pragma unroll
      for (int g = 0; g < KEYS; g += 4) {
        if (g >= run) break;
#pragma unroll
        for (int i = g; i < g + 4; ++i) {
          const uint32_t k = key[i];
          const uint32_t bin = hist + ((digit == 2 ? k << 2 : k >> (shift - 2)) & mask);
          asm volatile("{\n .reg .pred p;\n setp.lt.u32 p, %1, %2;\n @p red.shared.add.u32 [%0], 1;\n}\n"
                       ::"r"(bin), "r"(k - lo), "r"(span) : "memory");
          if (digit == 0) top += k == 0xFFFFFFFFu;
        }
      }
    }
    if (digit == 0) {
      top = __reduce_add_sync(0xffffffffu, top);
      if ((tid & 31) == 0 && top) atomicAdd(&s_hist[BINS - 1], top);
    }
    __syncthreads();
    // bins from the top, 8 to a thread; all of the cluster's CTAs
    int c[BINS / ET], sum = 0;
#pragma unroll
    for (int i = 0; i < BINS / ET; ++i) c[i] = s_hist[BINS - 1 - (tid * (BINS / ET) + i)];
    if (ctas > 1) {
      tc::cluster_sync();
      for (int o = 1; o < ctas; ++o) {
        const int other = rank_cta + o < ctas ? rank_cta + o : rank_cta + o - ctas;
        const uint32_t from = tc::map_to_cta(tc::smem_u32(&s_hist[BINS - (tid + 1) * (BINS / ET)]), (uint32_t)other);
#pragma unroll
        for (int i = 0; i < BINS / ET; ++i) {
          int x;
          asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(x) : "r"(from + 4 * (BINS / ET - 1 - i)));
          c[i] += x;
        }
      }
      tc::cluster_sync();
    }
#pragma unroll
    for (int i = 0; i < BINS / ET; ++i) sum += c[i];
    int total;
    const int rank_before = rank;
    int above = block_prefix<ET>(sum, s_warp, total);
    if (above < rank && above + sum >= rank) {
#pragma unroll
      for (int i = 0; i < BINS / ET; ++i) {
        if (above < rank && above + c[i] >= rank) {
          s_digit = BINS - 1 - (tid * (BINS / ET) + i);
          s_rank = rank - above;
        }
        above += c[i];
      }
    }
    if (tid == 0 && total < rank) {          // the rest of the rank falls to keys of 0, which no bin counts
      s_digit = 0;
      s_rank = rank - total;
    }
    __syncthreads();
    prefix = prefix << bits | s_digit;
    rank = s_rank;
    if (total < rank_before) break;
    if (prefix == BINS - 1 && digit == 0) {
      prefix = 0xFFFFFFFFu;
      break;
    }
  }

  // In index order: of the keys equal to the keep-th largest the first `rank`
  // stay; free places and moving tokens are numbered in ascending order.  The
  // CTAs of a cluster count first what lies before each of them.
  int eq0 = 0, hole0 = 0, come0 = 0;
  // pass 0: equal keys of the CTA; 1: its free places and moving tokens; 2: the moves
#pragma unroll 1
  for (int pass = ctas > 1 ? 0 : 2; pass < 3; ++pass) {
    int eq_run = eq0, hole_run = hole0, come_run = come0;
    for (int round = 0; round < rounds; ++round) {
      if (rounds > 1) load_keys(round);
      const int n = count();
      const uint32_t in = n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1;   // a bit per token of the run
      uint32_t kept = 0, same = 0;
#pragma unroll
      for (int g = 0; g < KEYS; g += 4) {
        if (g >= run) break;
#pragma unroll
        for (int i = g; i < g + 4; ++i) {
          if (key[i] > prefix) kept |= 1u << i;
          if (key[i] == prefix) same |= 1u << i;
        }
      }
      same &= in;
      int all;
      int eq_at = eq_run + block_prefix<ET>(__popc(same), s_warp, all);
      eq_run += all;
      if (pass == 0) continue;
      for (; same && eq_at < rank; same &= same - 1, ++eq_at) kept |= same & -same;
      const int below = max(0, min(keep - j0, 32));           // tokens of the run in the first keep places
      const uint32_t low = below >= 32 ? 0xFFFFFFFFu : (1u << below) - 1;
      uint32_t hole = in & low & ~kept, come = in & ~low & kept;
      const int at = block_prefix<ET>(__popc(hole) << 16 | __popc(come), s_warp, all);
      const int holes = all >> 16, comes = all & 0xFFFF;
      if (pass == 2) {
        // into shared memory in their order, then out, a thread per entry
        int to = at >> 16;
        for (; hole; hole &= hole - 1) s_list[to++] = (uint16_t)(tid * run + __ffs(hole) - 1);
        to = holes + (at & 0xFFFF);
        for (; come; come &= come - 1) s_list[to++] = (uint16_t)(tid * run + __ffs(come) - 1);
        __syncthreads();
        const int base = t_lo + round * SLICE;
        for (int i = tid; i < holes + comes; i += ET) {
          const long long entry = place(i < holes ? 2 * (hole_run + i) : 2 * (come_run + i - holes) + 1);
          if (entry >= 0) move[entry] = base + s_list[i];
        }
      }
      hole_run += holes;
      come_run += comes;
    }
    if (pass == 2) {
      if (tid == 0 && rank_cta == ctas - 1) *n_move = come_run;
      break;
    }
    // to every CTA of the cluster
    if (tid < ctas) {
      const uint32_t to = tc::map_to_cta(tc::smem_u32(&s_cta[pass][rank_cta][0]), (uint32_t)tid);
      asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(to), "r"(pass ? hole_run : eq_run), "r"(come_run) : "memory");
    }
    tc::cluster_sync();
    for (int c = 0; c < rank_cta; ++c) {
      if (pass == 0) {
        eq0 += s_cta[0][c][0];
      } else {
        hole0 += s_cta[1][c][0];
        come0 += s_cta[1][c][1];
      }
    }
  }
  if (__syncthreads_or(lost) && tid == 0) set_status(a.status, SKV_DEV_BAD_PAGE);
}

// ---------------------------------------------------------------------------
// Move.  D / 8 lanes take 16 bytes of a row each, of its key and its value; a
// warp takes every parts-th batch of moves of one (layer, request, kv head),
// and all loads of a batch are out before its first store.  Few moves are bound
// by four dependent loads (64 requests with a move of each of 8 kv heads and 4
// layers: 4.9 us), many by HBM (four prompts of 6 to 12.8 k tokens cut to 4,096,
// 8 layers: 115 us, 5.0 TB/s).

constexpr int MT = 256;
constexpr int MU = 2;           // moves in flight per D / 8 lanes (4: 64 requests with one each 4.6 -> 6.9 us, prompts 114 -> 110)

template <int D>
__global__ void __launch_bounds__(MT) evict_move_kernel(const EvictArgs a) {
  constexpr int LANES = D / 8, PER = 32 / LANES;     // moves that a warp takes side by side
  const int worker = blockIdx.x * (MT / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int unit = worker / a.parts, part = worker % a.parts;
  if (unit >= a.n_layer * a.n_req * a.Hkv) return;
  const int h = unit % a.Hkv, b = unit / a.Hkv % a.n_req, layer = unit / a.Hkv / a.n_req;
  const int c = lane % LANES, sub = lane / LANES;
  tc::grid_dep_wait();
  bool bad;
  const int m = held_tokens(a, b, bad);
  const int n = a.n_move[unit];
  bad |= n < 0 || n > m / 2;
  if (bad) {
    if (part == 0 && lane == 0) set_status(a.status, SKV_DEV_BAD_LEN);
    return;
  }
  const Place place = place_of(a, b, h);
  const size_t pool = (size_t)layer * a.n_page * a.Hkv * a.page_size;
  const int32_t* move = a.move + pool;
  uint4* k = reinterpret_cast<uint4*>(a.k) + pool * LANES;
  uint4* v = reinterpret_cast<uint4*>(a.v) + pool * LANES;
  for (int i0 = part * PER * MU + sub; i0 < n; i0 += a.parts * PER * MU) {
    int2 pair[MU];
    int fault[MU];                           // status bits of a move that is left out
    long long at[MU];
#pragma unroll
    for (int u = 0; u < MU; ++u) {
      const int i = i0 + u * PER;
      pair[u] = make_int2(0, 0);
      at[u] = i < n ? place(2 * i) : -1;
      fault[u] = at[u] >= 0 ? 0 : SKV_DEV_BAD_PAGE;
      if (at[u] >= 0) pair[u] = *reinterpret_cast<const int2*>(move + at[u]);
    }
    long long to[MU], from[MU];
#pragma unroll
    for (int u = 0; u < MU; ++u) {
      if (pair[u].x < 0 || pair[u].x >= m || pair[u].y < 0 || pair[u].y >= m) {
        fault[u] = SKV_DEV_BAD_LEN;
        pair[u] = make_int2(0, 0);
      }
      to[u] = from[u] = -1;
      if (i0 + u * PER < n) {
        to[u] = place(pair[u].x);
        from[u] = place(pair[u].y);
        if (to[u] < 0 || from[u] < 0) fault[u] |= SKV_DEV_BAD_PAGE;
        if (fault[u]) {
          if (c == 0) set_status(a.status, fault[u]);
          to[u] = -1;
        }
      }
    }
    uint4 kv[MU], vv[MU];
    float sc[MU];
    int ps[MU];
#pragma unroll
    for (int u = 0; u < MU; ++u)
      if (to[u] >= 0) {
        kv[u] = k[from[u] * LANES + c];
        vv[u] = v[from[u] * LANES + c];
        if (c == 0) {
          sc[u] = a.score[pool + from[u]];
          ps[u] = a.pos[pool + from[u]];
        }
      }
#pragma unroll
    for (int u = 0; u < MU; ++u)
      if (to[u] >= 0) {
        k[to[u] * LANES + c] = kv[u];
        v[to[u] * LANES + c] = vv[u];
        if (c == 0) {
          a.score[pool + to[u]] = sc[u];
          a.pos[pool + to[u]] = ps[u];
        }
      }
  }
}

}  // namespace

cudaError_t launch_evict_plan(const EvictArgs& in, cudaStream_t st) {
  EvictArgs a = in;
  const long long units = (long long)a.n_layer * a.n_req * a.Hkv;
  const long long room = min((long long)a.max_block * a.page_size, (long long)kMaxKeys);   // tokens that a request may hold
  // As many threads as hold a full table row in registers: with 256 where 128
  // do, 64 requests at a budget of 2,048 take 41 us instead of 31; a cluster of
  // two CTAs of 256 instead of 512 threads 174 us for prompts instead of 98.
  // A cluster has as many CTAs as hold the row, and no more where that leaves SMs
  // idle: its barriers cost more than shorter slices save (one request of 3,000
  // tokens, 8 kv heads, over four CTAs 23.8 us, in one 9.5; of 60,000 tokens and 4
  // layers over eight 91 us, over four 38).
  // The host knows the rows, not what the requests hold: the 64 requests of 2,049
  // tokens take 28 us with rows of up to 4,096 tokens, 37 of 8,192, 71 of 12,864 and of
  // 16,384, 135 of 32,768, 207 of 131,072.
  const int threads = room > 256 * KEYS ? 512 : room > 128 * KEYS ? 256 : 128;
  a.per_cta = threads * KEYS;
  a.parts = 1;
  while (a.parts < EVICT_CLUSTER && (long long)a.parts * a.per_cta < room) a.parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(units * a.parts));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = a.parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, threads == 512   ? evict_plan_kernel<512>
                                  : threads == 256 ? evict_plan_kernel<256>
                                                   : evict_plan_kernel<128>, a);
}

cudaError_t launch_evict_move(const EvictArgs& a, int d, cudaStream_t st) {
  EvictArgs p = a;
  const long long units = (long long)a.n_layer * a.n_req * a.Hkv;
  // some 8,000 warps: one wave (32,000: prompts 114 -> 103 us, 64 requests with a move each 4.6 -> 8.3)
  p.parts = (int)max(1LL, 8192 / units);
  const unsigned grid = (unsigned)((units * p.parts + MT / 32 - 1) / (MT / 32));
  auto launch = [&](auto kernel) { return launch_dependent(kernel, dim3(grid), MT, 0, st, p); };
  return d == 128 ? launch(evict_move_kernel<128>) : launch(evict_move_kernel<64>);
}

}  // namespace skv
