// paged_attn_weight on the 5th-generation tensor cores (tcgen05 + TMEM): the
// attention weight that each cached key has got from a step's rows, added to
// what it had.
//
//   w[h][j] = sum over rows i that see key j and query heads g of kv head h of
//             exp(scale q_ig . k_j - lse_ig)
//
// Keys are the rows of the MMA (M = 128) and queries its columns, so a TMEM
// lane and the thread that reads it belong to one key: the sum over the
// queries stays in a register, and threads meet at a unit's end at most.  A
// unit is 256 keys (two tiles) of one (request, kv head) against the query
// tiles that see them; a query tile packs TQ tokens x the G query heads that
// share the kv head.  K is read once; with many rows the two key tiles stay in
// shared memory while the query tiles pass, with few (decode) the key tiles
// pass and a query tile is a few rows.
//
// With many rows either pipe is idle half the time.  A step has 1024 cycles of MMAs
// and as many of exponentials, and the two lines of steps (below) run in phase:
// the odd line's MMAs start some 500 cycles after the even line's, both score
// buffers are full 1850 cycles after their MMAs' start, then both lines take
// exponentials, and 3700 cycles after the first start comes the next (time stamps
// of one CTA).  Nothing but the release of its own buffer orders an issuer (four
// chunks of 2,048 tokens over 6 to 13 k keys, 32 query and 8 kv heads of 128:
// 515 us, 1220 TFLOP/s).  With few rows it streams K (64 requests of 0.4 to 8 k
// keys in pages of 16 tokens: 105 us, 5.4 TB/s).  Between them lie mixed calls: a tile
// that some of the keys do not see costs half as much again, and a unit against one
// row what its one K producer takes for its copies (pages of 48 tokens: 16 of them,
// 4800 cycles).
//
// Units form one sequence, ordered by request, kv head and key block, each as
// long as its query tiles and unit_cost more; CTA c of a persistent grid takes
// positions [c W, (c + 1) W) of it.  In calls of many rows a unit that several
// CTAs share leaves its sums in the workspace, and a second kernel adds them up
// in order, so that results do not depend on timing; else units stay whole.
//
// A step is a query tile against the unit's two key tiles.  Steps run in two
// lines, each with an MMA issuer, a score buffer, a pair of warpgroups and its
// own query stages: with many rows the even and the odd steps, with few the
// even and the odd pieces.  A wait names the parity of a phase only.  So whoever
// waits on a barrier waits for each of its phases, and no phase ends without
// those that wait for the one before: a line's barriers serve that line alone,
// a K ring its own producers.
//
//   warps 0 .. 15  four warpgroups, a thread per key: exponentials, sums, scores
//   then           scheduler (with many rows K producer too), Q producer (TMA),
//                  two MMA issuers; with few rows four K producers (TMA)
#include <math.h>

#include "common.cuh"
#include "evict.h"
#include "launch.cuh"
#include "skv.h"
#include "tc.cuh"

namespace skv {

namespace {

constexpr int BM = 128;       // keys of a key tile
constexpr int UK = 2 * BM;    // and of a unit
constexpr int BN = 128;       // rows of a query tile, at most
constexpr int EPI_WARPS = 16, WARP_K = 16, WARP_Q = 17, WARP_MMA = 18;   // two MMA warps
constexpr int WARP_MORE = 20;     // in the narrow form, four K producers
constexpr int NP = 4;         // pieces in flight between the scheduler and the other warps
constexpr int LL = 2;         // query tiles of a line whose logarithms are in shared memory
constexpr int WC = BN / 2;    // columns of a warpgroup in the wide form
constexpr int LIST = 512;     // requests with rows that a CTA knows ahead

template <int D, bool WIDE>
struct WCfg {
  static constexpr int NT = WIDE ? 640 : 768;
  // K producers of a key tile.  A copy of a small page's 16 rows takes the
  // issuing warp some 150 cycles, a key tile of them 2500, in which HBM would
  // bring two: with few rows each half of each tile has a warp of its own (64 requests, pages of
  // 16 tokens: 135 us with one warp per tile, 112 with the scheduler as one of four,
  // 105 so).
  static constexpr int PARTS = WIDE ? 1 : 2;
  // K and Q stages.  Many rows: the key tiles stay, the query tiles pass.  Few
  // (64 columns at most): the key tiles pass, and the bytes in flight hide
  // HBM's latency.
  static constexpr int QR = WIDE ? BN : 64;    // rows of a query stage
  static constexpr int KST = WIDE ? (D == 128 ? 3 : 6) : (D == 128 ? 4 : 10);
  static constexpr int QST = WIDE ? (D == 128 ? 2 : 6) : 4;
  // either key tile of a piece has a ring of its own where it has producers of its own
  static constexpr int KR = WIDE ? KST : KST / 2;
  static_assert(WIDE || KST % 2 == 0, "a ring for either key tile");
  static_assert(QST % 2 == 0, "a half for either line of steps");
  static constexpr int KT = BM * D * 2;        // bytes of a key tile
  static constexpr int HALF = BM * 128;        // one 64-dimension half of it
  static constexpr int QT = QR * D * 2;        // and of a query stage
  static constexpr int QHALF = QR * 128;
  static constexpr int K_OFF = 0;
  static constexpr int Q_OFF = KST * KT;
  static constexpr int L_OFF = Q_OFF + QST * QT;             // logarithms of query tiles' columns, [2 LL][BN]
  static constexpr int X_OFF = L_OFF + 2 * LL * BN * 4;         // sums of the upper warpgroups' columns, [3][2][BM]
  static constexpr int BAR_OFF = X_OFF + 3 * 2 * BM * 4;
  static constexpr int MISC_OFF = BAR_OFF + 72 * 8;
  static constexpr int PIECE_OFF = MISC_OFF + 64;
  static constexpr int LIST_OFF = PIECE_OFF + NP * 64;
  static constexpr int SCAN_OFF = LIST_OFF + LIST * 2;
  static constexpr int BYTES = SCAN_OFF + NT / 32 * 16;
  static constexpr int ALLOC = BYTES + 1024;                 // slack for 1024-byte alignment
  static_assert(ALLOC <= 232448, "shared memory");
};

template <int KST, int QST, int PARTS>
struct WBars {
  enum : int {
    KFULL = 0,                 // a part of a K tile landed
    KEMPTY = KFULL + PARTS * KST,   // MMA commit: the piece is done with it
    QFULL = KEMPTY + KST,      // Q tile landed
    QEMPTY = QFULL + QST,      // MMA commit
    SFULL = QEMPTY + QST,      // MMA commit: a step's scores, of both key tiles, in its line's buffer
    SFREE = SFULL + 2,         // its warps have read them
    LFULL = SFREE + 2,         // Q producer: logarithms of a query tile written
    LEMPTY = LFULL + 2 * LL,      // its warps are done with them
    XFULL = LEMPTY + 2 * LL,      // WIDE: the upper warpgroups' sums of a lane group's keys
    XEMPTY = XFULL + 4,        // they have been added
    PCFULL = XEMPTY + 4,       // scheduler: piece published
    PCEMPTY = PCFULL + NP,     // every other warp has read it
    DRAIN = PCEMPTY + NP,      // MMA commit: everything issued is complete
    COUNT
  };
  static_assert(COUNT <= 72, "barrier slots");
};

struct WParams {
  WeightArgs w;
  int G, TQ;              // query heads per kv head, tokens per query tile
  int N;                  // columns of an MMA: TQ G, up to a multiple of 16 (wide: 32)
  int BR, boxes;          // rows per TMA box, boxes per key tile (8 at most)
  uint32_t ps_m;          // fastdiv multiplier of the page size
  bool shared;            // WIDE: CTAs share units
  int unit_cost;          // positions that a unit takes before its query tiles
  float scale_log2;
  bool wait_poll;         // LIMITED: the limit is shorter than a try of a wait may sleep
  uint64_t wait_cycles;   // and the limit of a wait
  int4* ws_unit;          // [CTAs] the shared unit that starts in a CTA: pieces (0: none), request, kv head, key block
  float* ws_sum;          // [2 * CTAs][UK]
};

// Query tiles [qa, qa + nt) of a unit.
struct Piece {
  int nt;          // 0: no more pieces
  int qa;
  int b, h, k0;    // request, kv head, first key
  int q0, L, kv;   // the request's span
  int slot;        // -1: the whole unit; else the workspace slot of its sums
};
static_assert(sizeof(Piece) <= 64, "piece slot");

// A request's units, for one kv head.
struct Units {
  int L, old, nq, nkb;    // rows, keys before the step, query tiles, key blocks
  __device__ __forceinline__ Units(const Span& s, int TQ) {
    L = s.L;
    old = s.kv - s.L;
    nq = (s.L + TQ - 1) / TQ;
    nkb = (s.kv + UK - 1) / UK;
  }
  // the first query tile that sees a key of block kb
  __device__ __forceinline__ int first(int kb, int TQ) const { return max(0, kb * UK - old) / TQ; }
  // blocks that every query tile sees
  __device__ __forceinline__ int full(int TQ) const { return min(nkb, (old + TQ - 1) / UK + 1); }
  __device__ __forceinline__ long long positions(int TQ, int cost) const {
    const int f = full(TQ);
    long long p = (long long)f * (cost + nq);
    for (int kb = f; kb < nkb; ++kb) p += cost + nq - first(kb, TQ);
    return p;
  }
};

// Where key j of request b lies in the pools, -1 with a page outside the pool.
__device__ __forceinline__ long long key_place(const RaggedArgs& r, int b, int h, int j) {
  const int page = __ldcg(r.table + (size_t)b * r.max_block + j / r.page_size);
  return page >= 0 && page < r.n_page ? ((long long)page * r.Hkv + h) * r.page_size + j % r.page_size : -1;
}

template <int D, bool F16, bool WIDE, bool LIMITED>
__global__ void __launch_bounds__(WCfg<D, WIDE>::NT, 1)
attn_weight_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ WParams p) {
  using C = WCfg<D, WIDE>;
  using B = WBars<C::KST, C::QST, C::PARTS>;
  constexpr int KST = C::KST, QST = C::QST, QL = QST / 2, KR = C::KR, PARTS = C::PARTS, NT = C::NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = tc::smem_u32(smem);
  auto bar = [&](int i) { return sbase + C::BAR_OFF + 8u * i; };
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  int* s_rank = reinterpret_cast<int*>(smem + C::MISC_OFF + 8);      // the share's first request among those with rows
  long long* s_off = reinterpret_cast<long long*>(smem + C::MISC_OFF + 16);
  int* s_odd = reinterpret_cast<int*>(smem + C::MISC_OFF + 24);      // [2 LL] beside the logarithms: some row gives nothing
  static_assert(24 + 2 * LL * sizeof(int) <= 64, "misc slots");
  Piece* s_piece = reinterpret_cast<Piece*>(smem + C::PIECE_OFF);
  uint16_t* s_list = reinterpret_cast<uint16_t*>(smem + C::LIST_OFF);
  struct Sums {
    long long positions;
    int active, pad;
  };
  Sums* s_scan = reinterpret_cast<Sums*>(smem + C::SCAN_OFF);

  const RaggedArgs& r = p.w.r;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int TQ = p.TQ;

  if (tid < B::COUNT) {
    const int i = tid;
    int count = 1;
    if (i >= B::SFREE && i < B::SFREE + 2) count = 8;
    if (i >= B::LEMPTY && i < B::LEMPTY + 2 * LL) count = 8;
    if ((i >= B::KEMPTY && i < B::KEMPTY + KST) || i == B::DRAIN) count = 2;
    if (i >= B::XFULL && i < B::XFULL + 4) count = 3;
    if (i >= B::PCEMPTY && i < B::PCEMPTY + NP) count = (WIDE ? 3 : 7) + EPI_WARPS;
    tc::mbar_init(bar(i), count);
    tc::fence_barrier_init();
    tc::fence_proxy_async_smem();
  }
  if (WIDE) {
    // Rows of the query stages that no copy writes, where a tile holds fewer than
    // N: their columns then have scores of 0 and, with logarithms of -inf, weigh
    // nothing without a mask (seven heads per kv head leave two of 128).
    const int q0 = TQ * p.G, idle = p.N - q0;
    for (int i = tid; i < idle * QST * (D / 64) * 8; i += NT) {
      const int c = i & 7, hf = i / 8 % (D / 64), row = i / 8 / (D / 64);
      *reinterpret_cast<uint4*>(smem + C::Q_OFF + row / idle * C::QT + hf * C::QHALF + (q0 + row % idle) * 128 + c * 16) =
          make_uint4(0u, 0u, 0u, 0u);
    }
    tc::fence_proxy_async_smem();
  }
  if (warp == WARP_K) {
    tc::tmem_alloc(tc::smem_u32(s_tmem), 512);
    tc::tmem_relinquish();
  }
  if (lane == 0) {
    if (warp == WARP_K) tc::prefetch_tmap(&tmap_k);
    if (warp == WARP_Q) tc::prefetch_tmap(&tmap_q);
  }
  tc::grid_dep_wait();

  // ------------------------------------------------------------ this CTA's share
  long long total = 0, share, g0;
  {
    constexpr int PER = (SKV_PAGED_MAX_REQUESTS + NT - 1) / NT;
    static_assert(PER <= 32, "a bit per request");
    const int per = (r.n_req + NT - 1) / NT;
    const int i0 = min(r.n_req, tid * per), i1 = min(r.n_req, i0 + per);
    uint32_t rows = 0;                       // this thread's requests with rows
    Sums sum{0, 0, 0};
    auto cost = [&](const Span& s) { return s.L == 0 || s.kv == 0 ? 0ll : r.Hkv * Units(s, TQ).positions(TQ, p.unit_cost); };
    for (int b = i0; b < i1; ++b) {
      const Span s = request_span(r, b);
      if (s.bad && blockIdx.x == 0) set_status(r.status, SKV_DEV_BAD_LEN);
      const long long c = cost(s);
      sum.positions += c;
      if (c) {
        ++sum.active;
        rows |= 1u << (b - i0);
      }
    }
    Sums incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, incl.positions, o);
      const int v = __shfl_up_sync(0xffffffffu, incl.active, o);
      if (lane >= o) {
        incl.positions += t;
        incl.active += v;
      }
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    long long at = incl.positions - sum.positions;
    int rank = incl.active - sum.active, active = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      const Sums x = s_scan[w];
      if (w == warp) {
        at += total;
        rank += active;
      }
      total += x.positions;
      active += x.active;
    }
    share = max(1LL, (total + gridDim.x - 1) / gridDim.x);
    g0 = blockIdx.x * share;
    if (g0 >= total) {                       // nothing left for this CTA
      if (p.shared && tid == 0) p.ws_unit[blockIdx.x] = make_int4(0, 0, 0, 0);
      if (warp == WARP_K) tc::tmem_dealloc(*s_tmem, 512);
      return;
    }
    if (g0 >= at && g0 < at + sum.positions) {
      int k = rank;
      for (int b = i0;; ++b) {
        const long long c = rows >> (b - i0) & 1 ? cost(request_span(r, b)) : 0;
        if (g0 < at + c) break;
        at += c;
        k += c > 0;
      }
      *s_rank = k;
      *s_off = g0 - at;
    }
    __syncthreads();
    const int k0 = *s_rank;
    for (int b = i0; b < i1; ++b)
      if (rows >> (b - i0) & 1) {
        if (rank >= k0 && rank < k0 + LIST) s_list[rank - k0] = (uint16_t)b;
        ++rank;
      }
  }
  const long long g1 = min(g0 + share, total);

  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *s_tmem;
  auto wait = [&](int b, uint32_t phase) {
    if constexpr (LIMITED) {
      if (p.wait_poll) return tc::mbar_poll(bar(b), phase & 1, p.wait_cycles);
      return tc::mbar_sleep(bar(b), phase & 1, p.wait_cycles);
    } else {
      return tc::mbar_sleep(bar(b), phase & 1);
    }
  };
  // all lanes go on or none
  auto wait_all = [&](int b, uint32_t phase) { return (bool)__all_sync(0xffffffffu, wait(b, phase)); };
  // for what a warp has started itself and must not leave behind: however short
  // the caller's limit is
  auto drain = [&](int b, uint32_t phase) { return tc::mbar_sleep(bar(b), phase & 1); };
  auto take_piece = [&](int pi, Piece& pc) {
    const int s = pi % NP;
    if (!wait_all(B::PCFULL + s, pi / NP)) return false;
    pc = s_piece[s];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar(B::PCEMPTY + s));
    return true;
  };
  auto tiles_of = [&](const Piece& pc) { return pc.kv - pc.k0 > BM ? 2 : 1; };   // key tiles with keys

  // The page of box `lane & 7` of key tile kt of a piece; nothing is done with
  // the number before it is needed, so that the load does not stop the warp.
  auto page_of = [&](const Piece& pc, int kt) {
    const int x = lane & 7, j = pc.k0 + kt * BM + x * p.BR;
    int in_page, id = -1;
    const int at = fastdiv(j, r.page_size, p.ps_m, in_page);
    if (x < p.boxes && j < pc.kv) id = __ldcg(r.table + (size_t)pc.b * r.max_block + at);
    return id;
  };
  // The stage of key tile kt of a piece, its ring's nth.
  auto k_stage = [&](int kt, int n) { return (WIDE ? 0 : kt * KR) + n % KR; };
  // Part `part` of key tile kt of a piece, its ring's nth, into its stage: a half
  // of the dimensions (d = 64: every second box), a box at a time by one lane.
  auto load_keys = [&](const Piece& pc, int kt, int part, int n, int id) {
    const int j0 = pc.k0 + kt * BM, st = k_stage(kt, n);
    const int n_box = (min(BM, pc.kv - j0) + p.BR - 1) / p.BR;
    int in_page;
    fastdiv(j0 + (lane & 7) * p.BR, r.page_size, p.ps_m, in_page);
    // a page outside the pool reads as the zeros outside the map
    const bool in = id >= 0 && id < r.n_page;
    if (!in && lane < n_box) set_status(r.status, SKV_DEV_BAD_PAGE);
    const int z = in ? id * r.Hkv + pc.h : -1;
    if (n >= KR && !wait_all(B::KEMPTY + st, n / KR - 1)) return false;
    constexpr bool BOXES = PARTS == 2 && D == 64;
    const int first = BOXES ? part : 0, step = BOXES ? 2 : 1;
    constexpr int HALVES = PARTS == 2 ? 1 : D / 64;     // of this part's boxes
    const int h0 = PARTS == 2 && D == 128 ? part : 0;
    const uint32_t full = bar(B::KFULL + part * KST + st);
    if (lane == 0) tc::mbar_arrive_expect_tx(full, max(0, (n_box - first + step - 1) / step) * p.BR * 128 * HALVES);
    const uint32_t dst = sbase + C::K_OFF + st * C::KT;
    for (int x = first; x < n_box; x += step) {
      const int yx = __shfl_sync(0xffffffffu, in_page, x), zx = __shfl_sync(0xffffffffu, z, x);
      if (lane == 0) {
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf)
          tc::tma_load_3d(dst + (h0 + hf) * C::HALF + x * p.BR * 128, &tmap_k, full, (h0 + hf) * 64, yx, zx);
      }
    }
    __syncwarp();
    return true;
  };
  // the last of the n copies that a warp has started into a ring land before the CTA exits
  auto drain_keys = [&](int kt, int part, int n) {
    for (int j = max(0, n - KR); j < n && tc::mbar_sleep(bar(B::KFULL + part * KST + k_stage(kt, j)), (j / KR) & 1); ++j) {
    }
  };

  bool ok = true;
  if (warp >= EPI_WARPS) {
    // 512 x 104 + 128 x 64 = the 640 x 96 registers of the launch; with few rows
    // 512 x 88 + 256 x 64 = 768 x 80
    tc::setmaxnreg_dec<64>();
    if (warp == WARP_K) {
      // --------------------------- scheduler, and in the wide form K producer, one warp
      int n = 0, pi = 0;                         // key tiles of this warp so far, pieces published
      auto publish = [&](const Piece& pc) {
        const int slot = pi % NP;
        if (pi >= NP && !wait_all(B::PCEMPTY + slot, pi / NP - 1)) return false;
        if (lane == 0) {
          s_piece[slot] = pc;
          tc::mbar_arrive(bar(B::PCFULL + slot));
        }
        __syncwarp();
        ++pi;
        return true;
      };
      int at = 0;                                // place in the list of requests with rows
      int b = s_list[0];
      Span s = request_span(r, b);
      Units u(s, TQ);
      int h, kb;
      long long pos;                             // of the unit's start
      {
        long long off = *s_off;
        const long long per_head = u.positions(TQ, p.unit_cost);
        h = (int)(off / per_head);
        off -= h * per_head;
        const int whole = p.unit_cost + u.nq;    // positions of a block that every query tile sees
        kb = (int)min((long long)u.full(TQ), off / whole);
        off -= (long long)kb * whole;
        for (;; ++kb) {
          const int len = whole - u.first(kb, TQ);
          if (off < len) break;
          off -= len;
        }
        pos = g0 - off;
      }
      int4 shared_unit = make_int4(0, 0, 0, 0);  // the unit that starts here and goes on in the next CTA
      // the next piece of the share; nt 0: none
      auto next_piece = [&]() {
        Piece pc{};
        while (pos < g1 && !pc.nt) {
          pc.qa = u.first(kb, TQ);
          const int tiles = u.nq - pc.qa;
          const long long u0 = pos + p.unit_cost, u1 = u0 + tiles;
          pc.nt = tiles;
          pc.slot = -1;
          if (p.shared) {
            const long long lo = max(u0, g0), hi = min(u1, g1);
            pc.nt = (int)max(0LL, hi - lo);
            if (u0 < g0 || u1 > g1) pc.slot = 2 * (int)blockIdx.x + (u0 < g0 ? 0 : 1);
            if (u0 >= g0 && u0 < g1 && u1 > g1)
              shared_unit = make_int4((int)((u1 - 1) / share) - (int)blockIdx.x + 1, b, h, kb);
            pc.qa += (int)(lo - u0);
          } else if (pos < g0) {
            pc.nt = 0;                           // it started in the CTA before
          }
          pc.b = b;
          pc.h = h;
          pc.k0 = kb * UK;
          pc.q0 = s.q0;
          pc.L = s.L;
          pc.kv = s.kv;
          pos = u1;
          if (++kb == u.nkb) {
            kb = 0;
            if (++h == r.Hkv) {
              h = 0;
              if (pos < g1) {                    // the share goes on: some later request has rows
                if (++at < LIST) b = s_list[at];
                else ++b;
                s = request_span(r, b);
                while (s.L == 0 || s.kv == 0) s = request_span(r, ++b);
                u = Units(s, TQ);
              }
            }
          }
        }
        return pc;
      };
      // a piece ahead, so that its pages' numbers come while the one before loads
      Piece pc = next_piece();
      int id0 = WIDE ? page_of(pc, 0) : 0, id1 = WIDE ? page_of(pc, 1) : 0;
      while (pc.nt) {
        const Piece next = next_piece();
        const int next0 = WIDE ? page_of(next, 0) : 0, next1 = WIDE ? page_of(next, 1) : 0;
        if (!(ok = publish(pc))) break;
        if (WIDE) {
          for (int kt = 0; kt < tiles_of(pc) && ok; ++kt) {
            if ((ok = load_keys(pc, kt, 0, n, kt ? id1 : id0))) ++n;
          }
          if (!ok) break;
        }
        pc = next;
        id0 = next0;
        id1 = next1;
      }
      if (ok) ok = publish(Piece{});
      // always written: the second kernel reads it
      if (p.shared && lane == 0) p.ws_unit[blockIdx.x] = ok ? shared_unit : make_int4(0, 0, 0, 0);
      if (WIDE) drain_keys(0, 0, n);
    } else if (warp == WARP_Q) {
      // ------------------------------------------------------------ Q producer
      // With a query tile come the logarithms of its columns, four to a lane,
      // loaded a tile ahead: -lse log2 e, and -inf for a row that gives nothing.
      // Such a row's scores are most often not finite either, and a NaN or +inf
      // outlasts -inf: a tile that has one says so, and its scores are looked
      // through (all others pay for the word with 1.6% of a mixed batch at d = 64, and
      // less than 1% of decode steps and chunks).
      int steps = 0, line[2] = {};             // steps so far, and of either line
      int col_tok[4], col_off[4];              // token of a column, and its offset in lse
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = lane * 4 + q;
        col_tok[q] = c / p.G < TQ ? c / p.G : 1 << 30;
        col_off[q] = c % p.G * r.n_tok + c / p.G;
      }
      Piece pc;
      for (int pi = 0; (ok = take_piece(pi, pc)) && pc.nt; ++pi) {
        const float* lse = p.w.lse + (size_t)pc.h * p.G * r.n_tok + pc.q0;
        float lg[4];
        auto load_log = [&](int t0) {
#pragma unroll
          for (int q = 0; q < 4; ++q) lg[q] = col_tok[q] < pc.L - t0 ? lse[col_off[q] + t0] : INFINITY;
        };
        load_log(pc.qa * TQ);
        for (int i = 0; i < pc.nt; ++i, ++steps) {
          const int x = WIDE ? steps & 1 : pi & 1, m = line[x];
          const int st = x * QL + m % QL, ls = x * LL + m % LL;
          if (m >= QL && !(ok = wait_all(B::QEMPTY + st, m / QL - 1))) break;
          if (lane == 0) {
            tc::mbar_arrive_expect_tx(bar(B::QFULL + st), TQ * p.G * 128 * (D / 64));
#pragma unroll
            for (int hf = 0; hf < D / 64; ++hf)
              tc::tma_load_3d(sbase + C::Q_OFF + st * C::QT + hf * C::QHALF, &tmap_q, bar(B::QFULL + st), hf * 64, pc.h * p.G,
                              pc.q0 + (pc.qa + i) * TQ);
          }
          __syncwarp();
          ++line[x];
          if (m >= LL && !(ok = wait_all(B::LEMPTY + ls, m / LL - 1))) break;
          bool odd = false;                    // of the columns with rows
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const bool fin = isfinite(lg[q]);
            odd |= !fin && col_tok[q] < pc.L - (pc.qa + i) * TQ;
            lg[q] = fin ? lg[q] * -kLog2e : -INFINITY;
          }
          *reinterpret_cast<float4*>(smem + C::L_OFF + (ls * BN + lane * 4) * 4) = make_float4(lg[0], lg[1], lg[2], lg[3]);
          if (i + 1 < pc.nt) load_log((pc.qa + i + 1) * TQ);
          odd = __any_sync(0xffffffffu, odd);
          if (lane == 0) s_odd[ls] = odd;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(B::LFULL + ls));
        }
        if (!ok) break;
      }
      for (int x = 0; x < 2; ++x)
        for (int j = max(0, line[x] - QL); j < line[x] && drain(B::QFULL + x * QL + j % QL, j / QL); ++j) {
        }
    } else if (!WIDE && warp >= WARP_MORE) {
      // ------------------------------------- K producers: either tile, either part
      const int kt = (warp - WARP_MORE) >> 1, part = (warp - WARP_MORE) & 1;
      int n = 0;                               // tiles of the ring so far
      Piece pc;
      for (int pi = 0; (ok = take_piece(pi, pc)) && pc.nt; ++pi) {
        if (kt == 1 && tiles_of(pc) == 1) continue;
        if (!(ok = load_keys(pc, kt, part, n, page_of(pc, kt)))) break;
        ++n;
      }
      drain_keys(kt, part, n);
    } else if (warp == WARP_MMA || warp == WARP_MMA + 1) {
      // ----------------------------------------------------------- MMA issuers
      // One for either line: the tensor pipe takes only a few MMAs ahead, so that
      // one warp's waits and commits, about 650 cycles a step, would leave it
      // idle; here the other's MMAs run under them.
      const uint32_t idesc = F16 ? tc::idesc_f16(BM, p.N) : tc::idesc_bf16(BM, p.N);
      const uint64_t dk0 = tc::sdesc_sw128(sbase + C::K_OFF), dq0 = tc::sdesc_sw128(sbase + C::Q_OFF);
      const bool lead = tc::elect_one();
      const int x = warp - WARP_MMA;           // its line
      int k0 = 0, k1 = WIDE ? 1 : 0;           // either key tile's number in its ring
      int n0 = 0, m = 0;                       // steps before the piece, steps of the line so far
      for (int pi = 0; ok; ++pi) {
        const int slot = pi % NP;
        if (!(ok = wait_all(B::PCFULL + slot, pi / NP))) break;
        const int nt = s_piece[slot].nt, two = nt && tiles_of(s_piece[slot]) == 2;
        __syncwarp();
        if (lead) tc::mbar_arrive(bar(B::PCEMPTY + slot));
        if (!nt) break;
        // in a piece without steps for this warp too: its word that it is done
        // with a K stage must not come before the one on the stage's last use
        ok = true;
        for (int kt = 0; kt <= two && ok; ++kt)
          for (int part = 0; part < PARTS && ok; ++part)
            ok = wait_all(B::KFULL + part * KST + k_stage(kt, kt ? k1 : k0), (kt ? k1 : k0) / KR);
        if (!ok) break;
        const int mine = WIDE ? (nt + ((n0 ^ x) & 1 ? 0 : 1)) >> 1 : (pi & 1) == x ? nt : 0;   // steps of the piece
        for (int i = 0; i < mine; ++i, ++m) {
          const int qs = x * QL + m % QL;
          ok = wait_all(B::QFULL + qs, m / QL);
          if (m >= 1) ok = ok && wait_all(B::SFREE + x, m - 1);
          if (!ok) break;
          tc::tc_fence_after();
          if (lead) {
            for (int kt = 0; kt <= two; ++kt) {
              const uint64_t dk = tc::opaque(dk0 + ((uint32_t)(k_stage(kt, kt ? k1 : k0) * C::KT) >> 4));
              const uint64_t dq = tc::opaque(dq0 + ((uint32_t)(qs * C::QT) >> 4));
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t in = (kk & 3) * 32;
                tc::mma_ss(tmem + (2 * x + kt) * BN, dk + (((kk >> 2) * C::HALF + in) >> 4),
                           dq + (((kk >> 2) * C::QHALF + in) >> 4), idesc, kk > 0);
              }
            }
            tc::mma_commit(bar(B::SFULL + x));
            tc::mma_commit(bar(B::QEMPTY + qs));
          }
        }
        if (!ok) break;
        if (lead)
          for (int kt = 0; kt <= two; ++kt) tc::mma_commit(bar(B::KEMPTY + k_stage(kt, kt ? k1 : k0)));
        k0 += WIDE ? 1 + two : 1;
        k1 += WIDE ? 1 + two : two;
        n0 += nt;
      }
      if (lead) tc::mma_commit(bar(B::DRAIN));   // every MMA issued completes before TMEM is released
      drain(B::DRAIN, 0);
    }
  } else {
    tc::setmaxnreg_inc<WIDE ? 104 : 88>();
    // ---------------------------------------------- exponentials and scores
    // Two pairs of warpgroups.  WIDE: a pair takes every second step, so that
    // one's waits and reads run under the other's exponentials; a warpgroup
    // takes half the columns of both key tiles, so that a logarithm that it
    // reads from shared memory serves two scores.  Else a pair takes every
    // second piece, a warpgroup per key tile.
    const int wg = warp >> 2, lg = warp & 3;         // warpgroup, TMEM lane group
    const int row = lg * 32 + lane, tile = WIDE ? 0 : wg & 1;   // key, and key tile or the first of two
    const int pair = wg >> 1, col0 = WIDE ? (wg & 1) * WC : 0;
    constexpr int TILES = WIDE ? 2 : 1;              // key tiles of a thread
    constexpr int CH = 32;                           // scores of one that it takes from TMEM at a time
    const uint32_t t_lane = tmem + ((uint32_t)(lg * 32) << 16);
    const uint32_t s_log = sbase + C::L_OFF;
    float* s_x = reinterpret_cast<float*>(smem + C::X_OFF) + row;
    const float sl = p.scale_log2;
    const uint64_t sl2 = f2_pack(sl, sl);
    int n = 0, m = 0;                                // steps of the CTA and of the line so far
    Piece pc;
    for (int pi = 0; (ok = take_piece(pi, pc)) && pc.nt; ++pi) {
      const bool two = tiles_of(pc) == 2;
      if (!WIDE && (pi & 1) != pair) {               // the other pair's
        n += pc.nt;
        continue;
      }
      const int j0 = pc.k0 + tile * BM + row, old = pc.kv - pc.L;   // the thread's key, or its first
      const int jw = pc.k0 + tile * BM + lg * 32;                   // the warp's first
      const bool store = !WIDE || wg == 0;           // this thread writes the scores
      // of a whole unit: where the scores lie and what the weights are added to;
      // looked up ahead where a piece is short
      long long at = -1;
      float w0 = 0.f;
      if (!WIDE && j0 < pc.kv) {
        at = key_place(r, pc.b, pc.h, j0);
        if (at >= 0 && j0 < old && p.w.add) w0 = p.w.add[at];
      }
      uint64_t acc[TILES][2] = {};
      for (int i = 0; i < pc.nt; ++i, ++n) {
        if (WIDE && (n & 1) != pair) continue;       // the other pair's
        const int t0 = (pc.qa + i) * TQ, ls = pair * LL + m % LL;
        const int nv = min(TQ, pc.L - t0) * p.G;     // columns with rows
        const int end = WIDE ? min(nv, col0 + WC) : tile && !two ? 0 : nv;
        // every key of the warp is seen by every row of the tile, which is full
        bool all = jw + (TILES - 1) * BM + 31 - old <= t0 &&
                   (WIDE ? two && t0 + TQ <= pc.L : nv >= (end + CH - 1) / CH * CH);
        const uint32_t tS = t_lane + (2 * pair + tile) * BN;
        ok = wait_all(B::LFULL + ls, m / LL) && wait_all(B::SFULL + pair, m);
        if (!ok) break;
        const bool odd = tc::ld_shared_s32(sbase + C::MISC_OFF + 24 + ls * 4) != 0;
        all &= !odd;
        tc::tc_fence_after();
        auto release = [&]() {                       // the scores have been read
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(B::SFREE + pair));
        };
        if (end <= col0) release();
#pragma unroll 1
        for (int c0 = col0; c0 < end; c0 += CH) {
          uint32_t v[TILES][CH];
#pragma unroll
          for (int t = 0; t < TILES; ++t) tc::tmem_ld32(tS + t * BN + c0, v[t]);
          tc::tmem_wait_ld();
          if (c0 + CH >= end) release();
          if (!all) {
            // some of the scores are of rows that do not see the key, or of none
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
              const int lo = t && !two ? CH : min(max(j0 + t * BM - old - t0, 0), TQ) * p.G - c0;
#pragma unroll
              for (int k = 0; k < CH; ++k)
                if (k < lo || k >= nv - c0) v[t][k] = __float_as_uint(-INFINITY);
            }
            if (odd) {
              // nor those of a row that gives nothing, whatever they are
#pragma unroll
              for (int k = 0; k < CH; ++k) {
                const bool none = tc::ld_shared_s32(s_log + (ls * BN + c0 + k) * 4) == __float_as_int(-INFINITY);
#pragma unroll
                for (int t = 0; t < TILES; ++t)
                  if (none) v[t][k] = __float_as_uint(-INFINITY);
              }
            }
          }
#pragma unroll
          for (int k = 0; k < CH; k += 4) {
            uint64_t l0, l1;
            tc::ld_shared_pairs(s_log + (ls * BN + c0 + k) * 4, l0, l1);
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
              float a0, a1, a2, a3;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(v[t][k]), __uint_as_float(v[t][k + 1])), sl2, l0), a0, a1);
              f2_unpack(f2_fma(f2_pack(__uint_as_float(v[t][k + 2]), __uint_as_float(v[t][k + 3])), sl2, l1), a2, a3);
              acc[t][0] = f2_add(acc[t][0], f2_pack(tc::ex2(a0), tc::ex2(a1)));
              acc[t][1] = f2_add(acc[t][1], f2_pack(tc::ex2(a2), tc::ex2(a3)));
            }
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(B::LEMPTY + ls));
        ++m;
      }
      if (!ok) break;
      float sum[TILES];
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        float e0, e1;
        f2_unpack(f2_add(acc[t][0], acc[t][1]), e0, e1);
        sum[t] = e0 + e1;
      }
      if constexpr (WIDE) {
        // the columns' sums meet in the first warpgroup, in their order
        if (wg) {
          if (pi && !(ok = wait_all(B::XEMPTY + lg, pi - 1))) break;
          s_x[(wg - 1) * 2 * BM] = sum[0];
          s_x[(wg - 1) * 2 * BM + BM] = sum[1];
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(B::XFULL + lg));
        } else {
          if (!(ok = wait_all(B::XFULL + lg, pi))) break;
#pragma unroll
          for (int w = 0; w < 3; ++w) {
            sum[0] += s_x[w * 2 * BM];
            sum[1] += s_x[w * 2 * BM + BM];
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(B::XEMPTY + lg));
        }
      }
      if (!store) continue;
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        const int j = j0 + t * BM;
        if (WIDE && pc.slot >= 0) {
          p.ws_sum[(size_t)pc.slot * UK + t * BM + row] = sum[t];
          continue;
        }
        if (WIDE && j < pc.kv) {
          at = key_place(r, pc.b, pc.h, j);
          w0 = at >= 0 && j < old && p.w.add ? p.w.add[at] : 0.f;
        }
        if (at >= 0 && j < pc.kv) {
          p.w.score[at] = w0 + sum[t];
          if (j >= old) p.w.pos[at] = p.w.position[pc.q0 + j - old];
        }
      }
    }
  }
  if (!ok && lane == 0) set_status(r.status, SKV_DEV_TIMEOUT);

  tc::tc_fence_before();
  __syncthreads();
  if (warp == WARP_K) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// The units that several CTAs share: their pieces' sums in order, and the scores.
__global__ void __launch_bounds__(UK) weight_merge_kernel(const WParams p) {
  tc::grid_dep_wait();
  const RaggedArgs& r = p.w.r;
  const int4 u = __ldcg(p.ws_unit + blockIdx.x);
  if (u.x == 0) return;
  const Span s = request_span(r, u.y);
  const int j = u.w * UK + threadIdx.x, old = s.kv - s.L;
  if (j >= s.kv) return;
  const long long at = key_place(r, u.y, u.z, j);
  float sum = j < old && p.w.add && at >= 0 ? p.w.add[at] : 0.f;
  float w = 0.f;
  for (int k = 0; k < u.x; ++k)       // piece 0 is the last of its CTA's share, every other the first
    w += __ldcg(p.ws_sum + (size_t)(2 * (blockIdx.x + k) + (k == 0 ? 1 : 0)) * UK + threadIdx.x);
  if (at < 0) return;
  p.w.score[at] = sum + w;
  if (j >= old) p.w.pos[at] = p.w.position[s.q0 + j - old];
}

}  // namespace

cudaError_t launch_attn_weight(const WeightArgs& a, int d, bool f16, cudaStream_t st) {
  const RaggedArgs& r = a.r;
  WParams p;
  p.w = a;
  p.G = r.Hq / r.Hkv;
  // The form goes by the call's rows and slots, which is all that the host knows:
  // a tile holds the tokens that a slot has on average, and units are shared where
  // that is more than a tile.  Idle slots, and single tokens beside a chunk, make the
  // chunk's tiles small and leave its units whole.  32 query and 8 kv heads of 128: a
  // chunk of 2,048 tokens over 8,192 keys takes 121 us in up to 16 slots, 163 in
  // 64, 423 in 256, 1850 in 1,024, 3690 in 4,096; one of 512 tokens over 4,096 keys 32
  // in 4 slots, 315 in 256.  One decoding request of 3,136 keys takes 9.5 us, in 4,096
  // slots 13, beside 63 padding rows 12.
  const int most = BN / p.G;                 // tokens that a query tile may hold
  const int mean = (r.n_tok + r.n_req - 1) / r.n_req;
  p.TQ = 1;
  while (p.TQ < most && p.TQ < mean) p.TQ *= 2;
  p.TQ = min(p.TQ, most);
  p.shared = r.n_tok > (long long)r.n_req * most;
  const bool wide = p.TQ * p.G > 64;
  p.N = wide ? (p.TQ * p.G + 31) / 32 * 32 : (p.TQ * p.G + 15) / 16 * 16;   // wide: whole reads of 32 columns
  p.unit_cost = 2;
  p.BR = BM;
  while (r.page_size % p.BR) p.BR /= 2;
  p.boxes = BM / p.BR;
  p.ps_m = fastdiv_m((uint32_t)r.page_size);
  p.scale_log2 = r.sm_scale * kLog2e;
  // in cycles at the 2.07 GHz maximum clock: a slower one only lengthens it
  p.wait_cycles = (uint64_t)(min(r.wait_ns, (uint64_t)1 << 62) * 2.07);
  p.wait_poll = r.wait_ns < tc::kSuspendHintNs;
  constexpr int MAX_CTAS = 512;
  const int grid = min(sm_count(), MAX_CTAS);
  p.ws_unit = static_cast<int4*>(r.ws);
  p.ws_sum = reinterpret_cast<float*>(static_cast<char*>(r.ws) + MAX_CTAS * sizeof(int4));
  if (ragged_ws_bytes() < MAX_CTAS * sizeof(int4) + (size_t)2 * grid * UK * sizeof(float)) return cudaErrorInvalidValue;

  CUtensorMap tq, tk;
  const cuuint64_t dd = (cuuint64_t)d;
  if (!encode_3d(&tq, f16, r.q, {dd, (cuuint64_t)r.Hq, (cuuint64_t)r.n_tok}, {dd * 2, (cuuint64_t)r.q_stride * 2},
                 {64, (cuuint32_t)p.G, (cuuint32_t)p.TQ}) ||
      !encode_3d(&tk, f16, r.k, {dd, (cuuint64_t)r.page_size, (cuuint64_t)r.n_page * r.Hkv}, {dd * 2, dd * 2 * r.page_size},
                 {64, (cuuint32_t)p.BR, 1}))
    return cudaErrorInvalidValue;
  auto launch = [&](auto kernel, int threads, int smem, int variant) -> cudaError_t {
    cudaError_t e = set_smem_once(kernel, smem, variant);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kernel, dim3(grid), threads, smem, st, tq, tk, p);
    if (e != cudaSuccess || !p.shared) return e;
    return launch_dependent(weight_merge_kernel, dim3(grid), UK, 0, st, p);
  };
#define SKV_WEIGHT(DD, FF, SS, VAR)                                                                                 \
  (r.wait_ns ? launch(attn_weight_kernel<DD, FF, SS, true>, WCfg<DD, SS>::NT, WCfg<DD, SS>::ALLOC, 8 + (VAR))      \
             : launch(attn_weight_kernel<DD, FF, SS, false>, WCfg<DD, SS>::NT, WCfg<DD, SS>::ALLOC, VAR))
#define SKV_WEIGHT_FORMS(DD, FF, VAR) (wide ? SKV_WEIGHT(DD, FF, true, VAR) : SKV_WEIGHT(DD, FF, false, VAR + 1))
  if (d == 128) return f16 ? SKV_WEIGHT_FORMS(128, true, 0) : SKV_WEIGHT_FORMS(128, false, 2);
  return f16 ? SKV_WEIGHT_FORMS(64, true, 4) : SKV_WEIGHT_FORMS(64, false, 6);
#undef SKV_WEIGHT_FORMS
#undef SKV_WEIGHT
}

}  // namespace skv
