// paged_attn and cross_attn on the 5th-generation tensor cores (tcgen05 +
// TMEM): attention of packed queries over each request's pages or packed
// states.
//
//   S = Q K^T,  P = exp(scale S - m),  O = P V / sum P,  lse = m + log sum P
//
// in one pass over the keys: the maximum m is taken on a row's first key tile
// and kept until a later tile's probability sum passes LAG_LIMIT, then O and
// the sum are scaled down to the new one (see p_pass).
//
// A unit is NQ query tiles of one (request, kv head): a tile packs TQ =
// floor(128 / G) tokens x the G query heads that share the kv head into the
// 128 rows of an MMA.  The units' key tiles (128 keys each; a causal unit ends
// at its last token's key) form one sequence, ordered by request, kv head and
// query block, and CTA b of a persistent grid takes tiles [b W, (b + 1) W) of
// it: every SM streams the same number of tiles whatever the lengths, which
// the host never sees.  Each CTA finds its place by a scan over the requests'
// tile counts (closed forms, see unit_prefix).  A unit that several CTAs
// share leaves fp32 partials (O, m, sum) in the workspace, which a second
// kernel merges in the pieces' order, so results do not depend on timing (see
// merge_kernel).
//
// Two forms.  NQ = 2, for calls with more than TQ tokens per request: two
// query tiles share every key tile, and one tile's softmax runs under the
// other's MMAs.  At d = 128 it is bound by the tensor pipe and the waits of the
// warp that feeds it (four chunks of 2,048 tokens over 6 to 13 k keys, 32 query
// and 8 kv heads: 0.81 to 0.93 ms on several GPUs, 1360 to 1550 TFLOP/s); at d = 64,
// with half the MMA work per score, by the chain from scores over probabilities
// to the next scores, 2540 cycles a key tile for 1060 of MMAs (six requests of
// 1,536 tokens over up to 12,800 states: 203 to 220 us, 860 to 940 TFLOP/s).
// NQ = 1, for decode: one query tile, two score buffers, so that Q K^T of the
// next key tile runs under the softmax.  It is bound by streaming K and V from
// HBM (64 requests of 0.4 to 8 k keys: 172 to 177 us, 6.2 to 6.4 TB/s); most MMA
// rows are idle.
//
//   warps 0 .. 4 NQ - 1  softmax and epilogue: a warpgroup per query tile, a
//                        thread per row
//   then one warp each   K producer (TMA), V producer (TMA), MMA issuer,
//                        scheduler (splits the CTA's share into pieces of
//                        units, loads the pieces' queries by TMA)
//
// Keys and values are read as they lie: K rows are the K-major B operand of
// Q K^T, token-major V rows the MN-major B operand of P V.  A TMA box is 64
// dimensions x BR rows, BR the largest power of two (at most 128) that
// divides the page size, so that a key tile is 128 / BR boxes from any pages.
// Value rows past the request's length are set to zero in shared memory: a
// probability of 0 does not cancel a NaN there.
#include <cudaTypedefs.h>
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "ragged.h"
#include "skv.h"
#include "tc.cuh"

namespace skv {

PFN_cuTensorMapEncodeTiled_v12000 tmap_encode_fn();

namespace {

constexpr int BM = 128;   // rows of a query tile
constexpr int BN = 128;   // keys of a key tile
constexpr int NP = 4;     // pieces in flight between the scheduler and the other warps

template <int D, int NQ>
struct RCfg {
  static constexpr int SM_WARPS = 4 * NQ;
  static constexpr int WARP_K = SM_WARPS, WARP_V = SM_WARPS + 1, WARP_MMA = SM_WARPS + 2, WARP_SCHED = SM_WARPS + 3;
  static constexpr int NT = 32 * SM_WARPS + 128;
  // K and V stages: what the 227 KB hold beside the queries (for d = 64 as
  // many bytes in flight as for 128)
  static constexpr int KST = D == 128 ? 3 : (NQ == 2 ? 4 : 6);
  static constexpr int VST = D == 128 ? (NQ == 2 ? 2 : 3) : (NQ == 2 ? 4 : 6);
  static_assert(VST <= KST, "V stages are freed with the K stages (see the producers)");
  // 16-bit terms of a probability in P V.  One: each p is rounded once, which
  // moves the output by about as much as its own rounding.  Decode has the
  // tensor pipe and the softmax warps idle most of the time (HBM-bound: 64
  // requests of 4 k keys take 176 us with two terms, 175 with one), so it adds
  // what the first rounding left as a second term: the output's own rounding
  // is all there is.
  static constexpr int P_TERMS = NQ == 1 ? 2 : 1;
  // Key tiles that one accumulation in tensor memory takes.  The tensor cores
  // cut the low bits of every sum off, so a long sum of values of one sign
  // drifts towards zero, by about 2^-24 of itself per MMA of 16 keys: the mean
  // of positive values over 320,000 keys in one CTA was 1.1e-3 too small, over 4
  // million 1.8e-2.  Longer runs are cut into parts of 32,768 keys, a drift of a
  // quarter of fp16's half step (with P in two terms up to half), whose sums are
  // added in fp32 arithmetic that rounds to nearest.  An addition takes some 4
  // us of a part's 300 to 400 (152 requests of 65,536 keys in L2 563 -> 572 us,
  // 16 of 131,072 from HBM 1183 -> 1192); twice as many parts twice that.
  static constexpr int FOLD = 256;
  static constexpr int QT = BM * D * 2;        // bytes of a query tile
  static constexpr int KT = BN * D * 2;        // of a key or value tile
  static constexpr int HALF = BM * 128;        // one 64-dimension half of either
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = Q_OFF + NQ * QT;
  static constexpr int V_OFF = K_OFF + KST * KT;
  static constexpr int BAR_OFF = V_OFF + VST * KT;
  static constexpr int MISC_OFF = BAR_OFF + 44 * 8;
  static constexpr int PIECE_OFF = MISC_OFF + 64;
  static constexpr int SCAN_OFF = PIECE_OFF + NP * 64;       // sums of the prologue, one of each per warp
  static constexpr int BYTES = SCAN_OFF + NT / 32 * 16;
  static constexpr int ALLOC = BYTES + 1024;                 // slack for 1024-byte alignment
  static_assert(ALLOC <= 232448, "shared memory");
};

template <int KST, int VST, int NQ>
struct RBars {
  enum : int {
    QFULL = 0,                 // the piece's queries landed (TMA)
    QEMPTY,                    // MMA commit: the piece's Q K^T are done with them
    KFULL,                     // K tile landed
    EMPTY = KFULL + KST,       // MMA commit: K stage free, and the V stage of the tile before
    VFULL = EMPTY + KST,       // V tile landed
    SFULL = VFULL + VST,       // MMA commit: scores in buffer x
    PFULL = SFULL + 2,         // softmax warps: probabilities in buffer x
    PVDONE = PFULL + 2,        // MMA commit: the P V from buffer x landed in O
    OFREE = PVDONE + 2,        // softmax warps: O of query tile i read out
    PCFULL = OFREE + NQ,       // scheduler: piece published
    PCEMPTY = PCFULL + NP,     // every other warp has read it
    DRAIN = PCEMPTY + NP,      // MMA commit: everything issued is complete
    COUNT
  };
  static_assert(COUNT <= 44, "barrier slots");
};

struct RParams {
  RaggedArgs a;
  int G, TQ, TB;          // query heads per kv head, tokens per query tile and per unit
  int BR, boxes;          // rows per TMA box, boxes per key tile
  int whole_slack;        // positions that the longest unit may have over an equal share to keep units whole: what the partials and their merge take
  int unit_cost;          // positions that a unit takes before its tiles, for what it costs beside them
  float scale_log2;
  bool wait_poll;         // LIMITED: the limit is shorter than a try of a wait may sleep
  uint64_t wait_cycles;   // and the limit of a wait
  int4* ws_unit;          // [CTAs] the shared unit that starts in a CTA: pieces (0: none), first token row, kv head, tokens
  float* ws_ml;           // [2 * CTAs][NQ][BM][2]
  float* ws_o;            // [2 * CTAs][NQ][D / 4][BM][4], see ws_index
};

// One piece of a CTA's share, or a part of one: key tiles [ta, ta + nt) of a unit.
struct Piece {
  int nt;          // 0: no more pieces
  int ta;
  int b, h;
  int row0;        // the unit's first token row
  int ntok;        // its tokens
  int kv;          // keys of the request
  int pos0;        // keys that the unit's first token sees, less one
  int step;        // 1: each later token sees one more (causal), 0: all see the same
  int krow;        // first state of the request (cross attention)
  int sums;        // 4 times the workspace slot of its sums, | ADDS | LEAVES
};
static_assert(sizeof(Piece) <= 64, "piece slot");
constexpr int ADDS = 1;     // a part that adds the sums of the one before to its own
constexpr int LEAVES = 2;   // it leaves its sums in the workspace: more parts or other CTAs' pieces of the unit follow

// sum over i < n of floor((a i + b) / BN), by the Euclid-like reduction of
// counting lattice points under a line: O(log) steps.  a n + b < 2^32.
__device__ __forceinline__ unsigned long long floor_sum(uint32_t n, uint32_t a, uint32_t b) {
  unsigned long long ans = 0;
  uint32_t m = BN;
  while (n) {
    if (a >= m) {
      const uint32_t q = a / m;
      ans += (unsigned long long)n * (n - 1) / 2 * q;
      a -= q * m;
    }
    if (b >= m) {
      const uint32_t q = b / m;
      ans += (unsigned long long)n * q;
      b -= q * m;
    }
    const uint32_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y - n * m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return ans;
}

// x / y for x, y >= 0; most values fit 32 bits, whose division is short
__device__ __forceinline__ long long udiv(long long x, long long y) {
  if (((x | y) >> 32) == 0) return (uint32_t)x / (uint32_t)y;
  return x / y;
}

// Key tiles of query block qb of a request (at least one, so that a block
// without keys is visited and gets its zeros), and of the blocks before qb.
__device__ __forceinline__ int unit_tiles(const Span& s, bool causal, int TB, int qb) {
  if (s.kv == 0) return 1;
  const long long seen = causal ? (long long)(s.kv - s.L) + min((long long)(qb + 1) * TB, (long long)s.L) : s.kv;
  return (int)((seen + BN - 1) / BN);
}
__device__ __forceinline__ long long unit_prefix(const Span& s, bool causal, int TB, int nqb, int qb) {
  if (qb == 0) return 0;
  if (s.kv == 0 || !causal) return (long long)qb * unit_tiles(s, causal, TB, 0);
  const int full = min(qb, nqb - 1);       // blocks that end at a multiple of TB
  long long t = (long long)floor_sum(full, TB, (uint32_t)(s.kv - s.L) + TB + BN - 1);
  if (qb > full) t += unit_tiles(s, causal, TB, nqb - 1);
  return t;
}

// Token-major V as the MN-major B operand: 64 dimensions (128 bytes) by 8
// keys per 1024-byte swizzle group; the next 8 keys follow it, the next 64
// dimensions lie HALF bytes on.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t half) {
  return (tc::sdesc_sw128(saddr) & ~(uint64_t(0x3FFF) << 16)) | ((uint64_t)(half >> 4) << 16);
}

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (F16) return pack_f16x2_sat(lo, hi);
  else return pack_bf16x2(lo, hi);
}

template <bool F16>
__device__ __forceinline__ void unpack16(uint32_t w, float& lo, float& hi) {
  if constexpr (F16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
  } else {
    lo = bf16_lo(w);
    hi = bf16_hi(w);
  }
}

// Workspace offset (floats) of columns [4 c, 4 c + 4) of row r of a slot's
// query tile i: a column group of all rows is contiguous, so that a warp whose
// lanes hold consecutive rows reads and writes whole lines.
template <int D, int NQ>
__device__ __forceinline__ size_t ws_index(int slot, int i, int c, int r) {
  return ((((size_t)slot * NQ + i) * (D / 4) + c) * BM + r) * 4;
}

// Merge of the units that several CTAs share: O = sum_k w_k O_k / sum_k w_k l_k
// with w_k = 2^(m_k - M), over the n pieces' partials (O_k, m_k, l_k) in their
// order.  One CTA after the last piece would have to read all of a unit's
// partials by itself (36 rows x 13 pieces took it 15 us); here a unit's rows
// and columns are spread over blocks, which start as the attention's CTAs
// leave their SMs.  Block (c, i, x) takes part x of query tile i of the unit
// that starts in CTA c (if one does); a thread takes CU groups of 4 columns of
// a row, with KU pieces in flight, M following as it grows: bound by one or
// two round trips to L2 (2.6 us of a decode call's 13, launch and all).  Wide
// units have two or three pieces: few in flight and eight blocks an SM, so
// that the many blocks without work pass in two rounds; decode units have a
// dozen: as many in flight as registers allow.
constexpr int MT = 128;         // threads per block
constexpr int MERGE_PARTS = 8;  // blocks per query tile: 128 rows x 8 threads, or 32 rows x 32

template <int D, bool F16, int NQ, int CU, int KU>
__device__ __forceinline__ void merge_part(const RParams& p, const int4& u, int c0, int i, int rows, int t) {
  const RaggedArgs& a = p.a;
  const int r = t % rows, c = t / rows * CU;     // row, first column group
  if (c >= D / 4) return;
  // piece 0 is the last of its CTA's share, every other the first
  auto slot = [&](int k) { return 2 * (c0 + k) + (k == 0 ? 1 : 0); };
  float4 acc[CU];
#pragma unroll
  for (int q = 0; q < CU; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, den = 0.f;
  for (int k0 = 0; k0 < u.x; k0 += KU) {
    float4 v[KU][CU];
    float2 ml[KU];
#pragma unroll
    for (int x = 0; x < KU; ++x) {
      const bool on = k0 + x < u.x;
      ml[x] = on ? __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + ((size_t)slot(k0 + x) * NQ + i) * BM + r)
                 : make_float2(0.f, 0.f);
#pragma unroll
      for (int q = 0; q < CU; ++q)
        v[x][q] = on ? __ldcg(reinterpret_cast<const float4*>(p.ws_o + ws_index<D, NQ>(slot(k0 + x), i, c + q, r)))
                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float mx = M;
#pragma unroll
    for (int x = 0; x < KU; ++x)
      if (ml[x].y != 0.f) mx = fmaxf(mx, ml[x].x);   // a piece without a visible key left l = 0
    const float al = M == -INFINITY ? 0.f : exp2f(M - mx);
    den *= al;
#pragma unroll
    for (int q = 0; q < CU; ++q) {
      acc[q].x *= al;
      acc[q].y *= al;
      acc[q].z *= al;
      acc[q].w *= al;
    }
#pragma unroll
    for (int x = 0; x < KU; ++x) {
      if (ml[x].y == 0.f) continue;
      const float w = exp2f(ml[x].x - mx);
      den += w * ml[x].y;
#pragma unroll
      for (int q = 0; q < CU; ++q) {
        acc[q].x += w * v[x][q].x;
        acc[q].y += w * v[x][q].y;
        acc[q].z += w * v[x][q].z;
        acc[q].w += w * v[x][q].w;
      }
    }
    M = mx;
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  const int tok = u.y + i * p.TQ + r / p.G, hq = u.z * p.G + r % p.G;
  uint2* dst = reinterpret_cast<uint2*>(a.out + ((size_t)tok * a.Hq + hq) * D + c * 4);
#pragma unroll
  for (int q = 0; q < CU; ++q)
    dst[q] = make_uint2(pack16<F16>(acc[q].x * inv, acc[q].y * inv), pack16<F16>(acc[q].z * inv, acc[q].w * inv));
  if (a.lse && c == 0)
    a.lse[(size_t)hq * a.n_tok + tok] = den == 0.f ? -INFINITY : (M + __log2f(den)) * 0.69314718055994531f;
}

template <int D, bool F16, int NQ>
__global__ void __launch_bounds__(MT, NQ == 2 ? 8 : 4) merge_kernel(const RParams p) {
  tc::grid_dep_wait();
  const int c0 = blockIdx.x, i = blockIdx.y, t = blockIdx.z * MT + threadIdx.x;
  const int4 u = __ldcg(p.ws_unit + c0);
  const int rows = min(p.TQ, u.w - i * p.TQ) * p.G;
  if (u.x == 0 || rows <= 0) return;
  // few rows (decode): a thread per row and 4 columns, many pieces in flight;
  // else whole 32-byte sectors of the output a thread
  if (rows <= MERGE_PARTS * MT / 32) merge_part<D, F16, NQ, 1, NQ == 2 ? 8 : 16>(p, u, c0, i, rows, t);
  else merge_part<D, F16, NQ, 4, NQ == 2 ? 2 : 4>(p, u, c0, i, rows, t);
}

// LIMITED: compiled for a caller's wait limit.  The limit as an operand of every
// wait cost the normal calls 1 to 5% (152 requests of 65,536 keys 464 -> 487 us).
template <int D, bool F16, int NQ, bool PAGED, bool LIMITED>
__global__ void __launch_bounds__(RCfg<D, NQ>::NT, 1)
ragged_attn_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ RParams p) {
  using C = RCfg<D, NQ>;
  using B = RBars<C::KST, C::VST, NQ>;
  constexpr int KST = C::KST, VST = C::VST;
  // Largest probability sum of a tile that keeps the old maximum.  P is
  // rounded to the values' type relative to its own size, so it may exceed 1;
  // fp16 ends at 65504.
  constexpr float LAG_LIMIT = F16 ? 16384.0f : 1048576.0f;
  // log2 of P at a row's maximum.  fp16 also starts at 2^-24: with P = 64 there
  // a probability is lost below 2^-31 of the largest, so that a million keys far
  // below one do not vanish (a tile's sum stays at 64 x 128, under the limit).
  constexpr float P_SHIFT = F16 ? 6.0f : 0.0f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = tc::smem_u32(smem);
  auto bar = [&](int i) { return sbase + C::BAR_OFF + 8u * i; };
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile long long* s_off = reinterpret_cast<volatile long long*>(smem + C::MISC_OFF + 16);
  int* s_first = reinterpret_cast<int*>(smem + C::MISC_OFF + 24);   // the share's first request and its span
  Piece* s_piece = reinterpret_cast<Piece*>(smem + C::PIECE_OFF);
  struct Sums {
    long long positions;
    int units, longest;
  };
  static_assert(sizeof(Sums) == 16, "sums of a warp");
  Sums* s_scan = reinterpret_cast<Sums*>(smem + C::SCAN_OFF);

  const RaggedArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int TB = p.TB;

  // what needs none of the call's inputs runs while the kernel before this
  // one on the stream ends
  if (tid == 0) {
    for (int i = 0; i < B::COUNT; ++i) {
      int count = 1;
      if (i >= B::PFULL && i < B::PFULL + 2) count = 4;
      if (i >= B::OFREE && i < B::OFREE + NQ) count = 4;
      if (i >= B::PCEMPTY && i < B::PCEMPTY + NP) count = 3 + C::SM_WARPS;
      tc::mbar_init(bar(i), count);
    }
    tc::fence_barrier_init();
    tc::fence_proxy_async_smem();
  }
  if (warp == C::WARP_K) {
    tc::tmem_alloc(tc::smem_u32(s_tmem), 512);
    tc::tmem_relinquish();
  }
  if (lane == 0) {
    if (warp == C::WARP_K) tc::prefetch_tmap(&tmap_k);
    if (warp == C::WARP_V) tc::prefetch_tmap(&tmap_v);
    if (warp == C::WARP_SCHED) tc::prefetch_tmap(&tmap_q);
  }
  tc::grid_dep_wait();

  // ------------------------------------------------------------ this CTA's share
  // Sums over the requests: positions of the sequence, units (as far as they
  // are fewer than a million), and the longest unit.
  long long total, share, g0;
  bool whole;                              // a unit per CTA, none of them shared
  {
    const int per = (a.n_req + C::NT - 1) / C::NT;
    const int i0 = min(a.n_req, tid * per), i1 = min(a.n_req, i0 + per);
    constexpr int MANY = 1 << 20;
    Sums sum{0, 0, 0};
    Span sp{};                             // the thread's last request (most have one)
    auto count = [&](int b, Sums& s) {
      sp = request_span(a, b);
      if (sp.L == 0) return;
      const int nqb = (sp.L + TB - 1) / TB;
      s.positions += a.Hkv * (unit_prefix(sp, PAGED, TB, nqb, nqb) + (long long)p.unit_cost * nqb);
      s.units = (int)min((long long)MANY, s.units + (long long)a.Hkv * nqb);
      s.longest = max(s.longest, unit_tiles(sp, PAGED, TB, nqb - 1));
    };
    for (int b = i0; b < i1; ++b) {
      count(b, sum);
      if (sp.bad && blockIdx.x == 0) set_status(a.status, SKV_DEV_BAD_LEN);
    }
    Sums incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, incl.positions, o);
      const int v = __shfl_up_sync(0xffffffffu, incl.units, o);
      if (lane >= o) {
        incl.positions += t;
        incl.units = min(MANY, incl.units + v);
      }
    }
    incl.longest = __reduce_max_sync(0xffffffffu, sum.longest);
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    long long at = incl.positions - sum.positions;   // positions and units before this thread's requests
    int at_unit = incl.units - sum.units, units = 0, longest = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < C::NT / 32; ++w) {
      const Sums x = s_scan[w];
      if (w == warp) {
        at += total;
        at_unit += units;
      }
      total += x.positions;
      units = min(MANY, units + x.units);
      longest = max(longest, x.longest);
    }
    // Equal shares, but of a few keys each they would cost more to merge than
    // to read: a tile takes about seven times as long as a piece's part of a
    // merge, so with T tiles per unit the sum of both is least at sqrt(T / 7)
    // tiles a piece (decode of one request of 30,000 keys and one kv head:
    // 22.6 us at equal shares of two tiles, 19.4 so).  With more units than the
    // sums count, equal shares are the longer ones anyway.
    share = max(1LL, udiv(total + gridDim.x - 1, gridDim.x));
    share = max(share, (long long)ceilf(sqrtf((float)total / (7.f * max(units, 1)))));
    // With a CTA for every unit and the longest not much over an equal share,
    // units stay whole: what the shares save is less than the partials cost (16
    // requests of 20 tokens and 4 k keys, 8 kv heads: 51.4 us whole, 56.3 in
    // shares; single tokens over 2 k keys: 32.1 and 32.5).
    whole = units <= (int)gridDim.x && longest + p.unit_cost <= share + p.whole_slack;
    if (whole) {
      share = 1;
      total = units;
      at = at_unit;
    }
    g0 = blockIdx.x * share;
    if (g0 >= total) {                     // no tiles left for this CTA
      if (tid == 0) p.ws_unit[blockIdx.x] = make_int4(0, 0, 0, 0);
      if (warp == C::WARP_K) tc::tmem_dealloc(*s_tmem, 512);
      return;
    }
    const long long mine = whole ? sum.units : sum.positions;
    if (g0 >= at && g0 < at + mine) {
      int b = i0;
      for (; b < i1 - 1; ++b) {
        Sums s{0, 0, 0};
        count(b, s);
        const long long c = whole ? s.units : s.positions;
        if (g0 < at + c) break;
        at += c;
      }
      if (b == i1 - 1) sp = request_span(a, b);
      s_first[0] = b;
      s_first[1] = sp.q0;
      s_first[2] = sp.L;
      s_first[3] = sp.kv;
      *s_off = g0 - at;
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
  // for what a warp has started itself and must not leave behind: however short
  // the caller's limit is
  auto drain = [&](int b, uint32_t phase) { return tc::mbar_sleep(bar(b), phase & 1); };
  // piece number pi into registers, its slot given back (whole warps)
  auto take_piece = [&](int pi, Piece& pc) {
    const int s = pi % NP;
    if (!__all_sync(0xffffffffu, wait(B::PCFULL + s, pi / NP))) return false;
    pc = s_piece[s];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar(B::PCEMPTY + s));
    return true;
  };
  auto tiles_of = [&](const Piece& pc) { return NQ == 1 || pc.ntok <= p.TQ ? 1 : 2; };   // query tiles with rows

  if (warp >= C::SM_WARPS) {
    // 256 x 208 + 128 x 88 = the 384 x 168 registers of the launch
    if constexpr (NQ == 2) tc::setmaxnreg_dec<88>();
    if (warp == C::WARP_K || warp == C::WARP_V) {
      // ---------------------------------------------------------- producers
      const bool is_k = warp == C::WARP_K;
      const CUtensorMap* map = is_k ? &tmap_k : &tmap_v;
      const int nst = is_k ? KST : VST, full = is_k ? B::KFULL : B::VFULL;
      const uint32_t base = sbase + (is_k ? C::K_OFF : C::V_OFF);
      // Step n of the MMA issuer (Q K^T of tile n, P V of tile n - 1) ends with
      // a commit on EMPTY[n mod KST].  It frees the K stage of tile n and the V
      // stage of tile n - 1: K tile n waits for step n - KST, V tile n for step
      // n - VST + 1, whose barriers cannot be a phase further by then.
      int st = 0, n = 0;                // stage, tiles issued
      int es = 0;                       // EMPTY barrier and phase of the next wait
      uint32_t eph = 0;
      if (!is_k) es = 1;                // V tile VST waits for step 1
      Piece pc;
      bool ok = true;
      for (int pi = 0; (ok = take_piece(pi, pc)) && pc.nt; ++pi) {
        // lane x issues box x of a tile: the page of its first row
        const int32_t* row = PAGED ? a.table + (size_t)pc.b * a.max_block : nullptr;
        auto page_of = [&](int j) {
          const int r = (pc.ta + j) * BN + lane * p.BR;
          return PAGED && j < pc.nt && lane < p.boxes && r < pc.kv ? __ldcg(row + r / a.page_size) : -1;
        };
        int id = page_of(0);
        for (int j = 0; j < pc.nt; ++j, ++n) {
          const int r0 = (pc.ta + j) * BN;
          const int n_box = (max(0, min(BN, pc.kv - r0)) + p.BR - 1) / p.BR;
          if (n >= nst) {
            ok = __all_sync(0xffffffffu, wait(B::EMPTY + es, eph));
            if (!ok) break;
            if (++es == KST) {
              es = 0;
              eph ^= 1;
            }
          }
          if (lane == 0) tc::mbar_arrive_expect_tx(bar(full + st), n_box * p.BR * 128 * (D / 64));
          __syncwarp();
          if (lane < n_box) {
            const int r = r0 + lane * p.BR;
            int y = pc.h, z = pc.krow + r;
            if constexpr (PAGED) {
              // a page outside the pool reads as the zeros outside the map
              const bool in = id >= 0 && id < a.n_page;
              if (!in) set_status(a.status, SKV_DEV_BAD_PAGE);
              y = r % a.page_size;
              z = in ? id * a.Hkv + pc.h : -1;
            }
#pragma unroll
            for (int hf = 0; hf < D / 64; ++hf)
              tc::tma_load_3d(base + st * C::KT + hf * C::HALF + lane * p.BR * 128, map, bar(full + st), hf * 64, y, z);
          }
          id = page_of(j + 1);
          if (++st == nst) st = 0;
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) set_status(a.status, SKV_DEV_TIMEOUT);
      // the copies this warp started land before the CTA exits
      for (int j = max(0, n - nst); j < n && drain(full + j % nst, j / nst); ++j) {
      }
    } else if (warp == C::WARP_MMA) {
      // --------------------------------------------------------- MMA issuer
      // all lanes go on or none: they meet again at the next warp-wide step
      auto wait_all = [&](int b, uint32_t phase) { return (bool)__all_sync(0xffffffffu, wait(b, phase)); };
      constexpr uint32_t idesc_qk = F16 ? tc::idesc_f16(BM, BN) : tc::idesc_bf16(BM, BN);
      constexpr uint32_t idesc_pv = (F16 ? tc::idesc_f16(BM, D) : tc::idesc_bf16(BM, D)) | (1u << 16);
      const uint64_t dq0 = tc::sdesc_sw128(sbase + C::Q_OFF);
      const uint64_t dk0 = tc::sdesc_sw128(sbase + C::K_OFF);
      const uint64_t dv0 = sdesc_mn(sbase + C::V_OFF, C::HALF);
      auto issue_qk = [&](int i, int ks, int buf) {
        const uint64_t dq = tc::opaque(dq0 + ((uint32_t)(i * C::QT) >> 4));
        const uint64_t dk = tc::opaque(dk0 + ((uint32_t)(ks * C::KT) >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4;
          tc::mma_ss(tmem + buf * BN, dq + off, dk + off, idesc_qk, kk > 0);
        }
      };
      auto issue_pv = [&](int i, int vs, int buf, bool fresh) {
        const uint64_t dv = tc::opaque(dv0 + ((uint32_t)(vs * C::KT) >> 4));
#pragma unroll
        for (int t = 0; t < C::P_TERMS; ++t)
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            tc::mma_ts(tmem + 256 + i * 128, tmem + buf * BN + (kk >> 2) * 64 + t * 32 + (kk & 3) * 8,
                       dv + ((kk * 2048) >> 4), idesc_pv, (!fresh || t + kk > 0) ? 1u : 0u);
      };
      // The tensor pipe takes only a few MMAs ahead, so what this warp does
      // between two MMAs may leave it idle: the state is a few scalars (stage
      // numbers and barrier phases), no struct and no division, and one step
      // (Q K^T of a tile, P V of the tile before) has four waits and three
      // commits.  The warp stays converged and one elected lane issues: 17
      // cycles an MMA, 45 under a branch on the lane.
      const bool lead = tc::elect_one();
      bool ok = true;
      int ks = 0, vs = 0, buf = 0;                  // K and V stage; NQ = 1: score buffer of the next tile
      uint32_t kph = 0, vph = 0, qph = 0;           // their phases, and the queries'
      uint32_t pph0 = 0, pph1 = 0;                  // phases of PFULL 0 and 1
      uint32_t oph0 = 1, oph1 = 1;                  // of OFREE: nothing to wait for the first time
      bool prev = false, prev2 = false, fresh = false;   // the tile before: its P V is to come, two query tiles, first of its piece
      bool last = false;                            // it is its piece's last
      // P V of query tile i of the tile before, from score buffer x
      auto pv = [&](int i, int x, uint32_t& pph, uint32_t& oph) {
        ok = wait_all(B::PFULL + x, pph);
        pph ^= 1;
        if (fresh) {
          // the piece before has been read out of O
          ok = wait_all(B::OFREE + i, oph) && ok;
          oph ^= 1;
        }
        if (!ok) return;
        tc::tc_fence_after();
        if (lead) {
          issue_pv(i, vs, x, fresh);
          // two query tiles: the next scores' commit covers this P V
          if (NQ == 1 || last) tc::mma_commit(bar(B::PVDONE + x));
        }
      };
      auto pv_prev1 = [&]() {                       // NQ = 1: the P V before, from the other score buffer
        ok = wait_all(B::VFULL + vs, vph);
        if (!ok) return;
        if (buf) pv(0, 0, pph0, oph0);
        else pv(0, 1, pph1, oph0);
      };
      auto v_done = [&]() {
        if (++vs == VST) {
          vs = 0;
          vph ^= 1;
        }
        prev = false;
      };
      for (int pi = 0; ok; ++pi) {
        const int slot = pi % NP;
        if (!(ok = wait_all(B::PCFULL + slot, pi / NP))) break;
        const int nt = s_piece[slot].nt;
        const bool two = NQ == 2 && s_piece[slot].ntok > p.TQ;
        __syncwarp();
        if (lead) tc::mbar_arrive(bar(B::PCEMPTY + slot));
        for (int j = 0; j < max(nt, 1); ++j) {
          // at a piece's start (and at the end) the P V before do not wait
          // for queries to come
          if (NQ == 2) {
            // the tiles are waited for first, under the MMAs still in the
            // pipe: from the probabilities' arrival on, P V and Q K^T go out
            // back to back
            if (prev) ok = wait_all(B::VFULL + vs, vph);
            if (nt) ok = wait_all(B::KFULL + ks, kph) && ok;
            if (!ok) break;
            if (prev) pv(0, 0, pph0, oph0);
            if (!ok) break;
          } else if (prev && j == 0) {
            pv_prev1();
            if (!ok) break;
            v_done();
          }
          if (nt) {
            if (j == 0) {
              if (!(ok = wait_all(B::QFULL, qph))) break;
              qph ^= 1;
            }
            if (NQ == 1 && !(ok = wait_all(B::KFULL + ks, kph))) break;
            const int x = NQ == 2 ? 0 : buf;
            if (lead) {
              issue_qk(0, ks, x);
              tc::mma_commit(bar(B::SFULL + x));
            }
          }
          if (prev) {
            if (NQ == 1) pv_prev1();
            else if (prev2) pv(1, 1, pph1, oph1);
            if (!ok) break;
            v_done();
          }
          if (nt) {
            if (lead) {
              if (two) {
                issue_qk(1, ks, 1);
                tc::mma_commit(bar(B::SFULL + 1));
              }
              tc::mma_commit(bar(B::EMPTY + ks));
              if (j == nt - 1) tc::mma_commit(bar(B::QEMPTY));
            }
            if (++ks == KST) {
              ks = 0;
              kph ^= 1;
            }
            if (NQ == 1) buf ^= 1;
            prev = true;
            prev2 = two;
            fresh = j == 0;
            last = j == nt - 1;
          }
        }
        if (!nt) break;
      }
      if (lead) {
        if (!ok) set_status(a.status, SKV_DEV_TIMEOUT);
        // every MMA issued completes before TMEM is released
        tc::mma_commit(bar(B::DRAIN));
      }
      drain(B::DRAIN, 0);
    } else if (warp == C::WARP_SCHED) {
      // ---------------------------------------------------------- scheduler
      // A unit takes unit_cost + its tiles positions of the sequence, the tiles
      // last; the CTA has the tiles at positions [g0, g1).
      int b = s_first[0], h, qb = 0, t;              // t: positions of the unit before g0
      Span s{s_first[1], s_first[2], s_first[3], false};
      int nqb = (s.L + TB - 1) / TB;
      {
        long long off = *s_off;
        if (whole) {
          h = (int)off / nqb;
          qb = (int)off - h * nqb;
          t = 0;
        } else if (nqb == 1) {
          const int per_head = unit_tiles(s, PAGED, TB, 0) + p.unit_cost;
          h = (int)udiv(off, per_head);
          t = (int)(off - (long long)h * per_head);
        } else {
          const long long per_head = unit_prefix(s, PAGED, TB, nqb, nqb) + (long long)p.unit_cost * nqb;
          h = (int)udiv(off, per_head);
          off -= h * per_head;
          // the block that holds off: a running sum over the blocks, 32 at a time
          for (;; qb += 32) {
            const int n = qb + lane < nqb ? unit_tiles(s, PAGED, TB, qb + lane) + p.unit_cost : 0;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int x = __shfl_up_sync(0xffffffffu, incl, o);
              if (lane >= o) incl += x;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, incl > off);   // blocks that end past off
            if (past) {
              const int l = __ffs(past) - 1;
              qb += l;
              t = (int)off - __shfl_sync(0xffffffffu, incl - n, l);
              break;
            }
            off -= __shfl_sync(0xffffffffu, incl, 31);
          }
        }
      }
      // The next request after b that has rows, 16 spans at a time: a cache
      // may have hundreds of idle slots between two requests (one by one 70 ns
      // each).
      auto next_request = [&](int& b) {
        Span s{0, 0, 0, false};
        while (s.L == 0 && b < a.n_req - 1) {
          constexpr int AHEAD = 16;
          int at[AHEAD + 1];                // ends of request b and of the ones after it
#pragma unroll
          for (int x = 0; x <= AHEAD; ++x) at[x] = a.q_start[min(b + 1 + x, a.n_req)];
          int x = 0;                        // first that does not end where the one before it does
#pragma unroll
          for (int y = AHEAD; y > 0; --y)
            if (at[y] != at[y - 1]) x = y;
          b = min(b + (x ? x : AHEAD), a.n_req - 1);
          if (x) s = request_span(a, b);
        }
        return s;
      };
      if (lane == 0) {
        long long g = g0;
        bool ok = true;
        int4 shared_unit = make_int4(0, 0, 0, 0);   // the unit that starts here and goes on in the next CTA
        int part = 0;                     // ADDS: the next piece is a part that goes on
        int loaded = 0;                   // pieces whose queries are on their way
        for (int pi = 0; ok; ++pi) {
          Piece pc{};
          const int nt_unit = g < g1 ? unit_tiles(s, PAGED, TB, qb) : 0;
          // positions of the unit's tiles; a whole unit takes the one of its CTA
          const long long u0 = whole ? g : g - t + p.unit_cost, u1 = whole ? g + 1 : u0 + nt_unit;
          if (g < g1 && u0 < g1) {
            pc.ta = whole ? t : max(0, t - p.unit_cost);
            pc.nt = (whole ? nt_unit : (int)(min(u1, g1) - u0)) - pc.ta;
            pc.b = b;
            pc.h = h;
            pc.row0 = s.q0 + qb * TB;
            pc.ntok = min(TB, s.L - qb * TB);
            pc.kv = s.kv;
            pc.step = PAGED && s.kv ? 1 : 0;
            pc.pos0 = pc.step ? s.kv - s.L + qb * TB : s.kv - 1;
            pc.krow = PAGED ? 0 : a.k_start[b];
            // a whole unit's parts are added up where the CTA's last piece will
            // leave its sums
            pc.sums = 4 * (2 * (int)blockIdx.x + (u0 < g0 ? 0 : 1)) | (u0 < g0 || u1 > g1 ? LEAVES : 0) | part;
            // (u0 lies in this CTA's share)
            if (u0 >= g0 && u1 > g1)
              shared_unit = make_int4((int)udiv(u1 - 1, share) - (int)blockIdx.x + 1, pc.row0, h, pc.ntok);
            part = 0;
            if (pc.nt > C::FOLD) {          // a long piece in parts
              pc.nt = C::FOLD;
              pc.sums |= LEAVES;
              part = ADDS;
              t = pc.ta + pc.nt + (whole ? 0 : p.unit_cost);
              if (!whole) g = u0 + pc.ta + pc.nt;
            } else {
              g = u1;
              // the next unit
              t = 0;
              if (++qb == nqb) {
                qb = 0;
                if (++h == a.Hkv) {
                  h = 0;
                  if (g < g1) {             // the share goes on: some later request has rows
                    s = next_request(b);
                    nqb = (s.L + TB - 1) / TB;
                  }
                }
              }
            }
          }
          const int slot = pi % NP;
          if (pi >= NP && !(ok = wait(B::PCEMPTY + slot, pi / NP - 1))) break;
          s_piece[slot] = pc;
          tc::mbar_arrive(bar(B::PCFULL + slot));
          if (!pc.nt) break;
          // its queries, once the piece before is done with the buffer
          if (pi > 0 && !(ok = wait(B::QEMPTY, pi - 1))) break;
          const int nq = tiles_of(pc);
          tc::mbar_arrive_expect_tx(bar(B::QFULL), nq * p.TQ * p.G * 128 * (D / 64));
          for (int i = 0; i < nq; ++i)
#pragma unroll
            for (int hf = 0; hf < D / 64; ++hf)
              tc::tma_load_3d(sbase + C::Q_OFF + i * C::QT + hf * C::HALF, &tmap_q, bar(B::QFULL), hf * 64, pc.h * p.G,
                              pc.row0 + i * p.TQ);
          loaded = pi + 1;
        }
        if (!ok) set_status(a.status, SKV_DEV_TIMEOUT);
        p.ws_unit[blockIdx.x] = ok ? shared_unit : make_int4(0, 0, 0, 0);   // always written: the merge reads it
        if (loaded) drain(B::QFULL, loaded - 1);
      }
    }
  } else {
    // ------------------------------------------------- softmax and epilogue
    if constexpr (NQ == 2) tc::setmaxnreg_inc<208>();
    const int i = warp >> 2, lg = warp & 3;          // query tile, TMEM lane group
    const int row = lg * 32 + lane;
    const uint32_t t_lane = (uint32_t)(lg * 32) << 16;
    const uint32_t tO = tmem + t_lane + 256 + i * 128;
    const int tok = row / p.G, gq = row - tok * p.G;
    const float sl = p.scale_log2;
    int gt = 0, cnt = 0, pcs = 0;                  // key tiles of the CTA and of this query tile, its pieces so far
    Piece pc;
    bool ok = true;
    for (int pi = 0; (ok = take_piece(pi, pc)) && pc.nt; ++pi) {
      if (i >= tiles_of(pc)) {
        gt += pc.nt;
        continue;
      }
      const int ntok = min(p.TQ, pc.ntok - i * p.TQ);   // tokens in this query tile
      const bool valid = tok < ntok;
      const bool active = lg * 32 < ntok * p.G;         // some row of the lane group is valid
      const int n_row = pc.pos0 + pc.step * (i * p.TQ + tok) + 1;   // keys that this row sees
      const int n_all = __reduce_min_sync(0xffffffffu, n_row);   // keys that every row of the warp sees
      float m_used = 0.f, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < pc.nt; ++j, ++gt, ++cnt) {
        const int x = NQ == 2 ? i : cnt & 1, ph = NQ == 2 ? cnt : cnt >> 1;
        const int r0 = (pc.ta + j) * BN;
        const uint32_t tS = tmem + t_lane + x * BN;
        // tcgen05.ld/st are warp-collective: every branch around them is warp-uniform
        ok = __all_sync(0xffffffffu, wait(B::SFULL + x, ph));
        if (!ok) break;
        if (active) {
          tc::tc_fence_after();
          uint32_t v[BN];
#pragma unroll
          for (int cb = 0; cb < BN / 32; ++cb)
            tc::tmem_ld32(tS + cb * 32, *reinterpret_cast<uint32_t(*)[32]>(v + cb * 32));
          tc::tmem_wait_ld();
          if (n_all - r0 < BN) {
            const int n_see = n_row - r0;          // of the tile's keys
#pragma unroll
            for (int k = 0; k < BN; ++k)
              if (k >= n_see) v[k] = __float_as_uint(-INFINITY);
          }
          auto row_max = [&]() {
            float m4[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) m4[q] = fmaxf(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1]));
#pragma unroll
            for (int k = 8; k < BN; k += 2)
              m4[(k >> 1) & 3] = fmax3(m4[(k >> 1) & 3], __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
            return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl;
          };
          // P = 2^(s scale - m) in the values' type over the first half of
          // either 64 scores (the products of P V take 16-bit operands), its
          // second term, if there is one, over the other half; the sum is
          // taken in fp32 before the rounding
          auto p_pass = [&]() {
            const uint64_t sl2 = f2_pack(sl, sl), nm2 = f2_pack(-m_used, -m_used);
            uint64_t l2[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) l2[q] = 0ull;
#pragma unroll
            for (int cb = 0; cb < BN / 32; ++cb) {
              uint32_t pk[16], pl[16];
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                float x0, x1;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(v[cb * 32 + k]), __uint_as_float(v[cb * 32 + k + 1])), sl2, nm2),
                          x0, x1);
                const float p0 = tc::ex2(x0), p1 = tc::ex2(x1);
                l2[(k >> 1) & 3] = f2_add(l2[(k >> 1) & 3], f2_pack(p0, p1));
                pk[k >> 1] = pack16<F16>(p0, p1);
                if constexpr (C::P_TERMS == 2) {
                  float h0, h1;
                  unpack16<F16>(pk[k >> 1], h0, h1);
                  pl[k >> 1] = pack16<F16>(p0 - h0, p1 - h1);
                }
              }
              tc::tmem_st16(tS + (cb >> 1) * 64 + (cb & 1) * 16, pk);
              if constexpr (C::P_TERMS == 2) tc::tmem_st16(tS + (cb >> 1) * 64 + 32 + (cb & 1) * 16, pl);
            }
            const uint64_t s2 = f2_add(f2_add(l2[0], l2[1]), f2_add(l2[2], l2[3]));
            float s0, s1;
            f2_unpack(s2, s0, s1);
            return s0 + s1;
          };
          if (j == 0) {
            const float mx = row_max();
            m_used = mx == -INFINITY ? 0.f : mx - P_SHIFT;
          }
          float ts;
          for (bool again = false;; again = true) {
            ts = p_pass();
            if (again || !__any_sync(0xffffffffu, valid && !(ts <= LAG_LIMIT))) break;
            tc::tmem_wait_st();
            if (NQ == 1 && j > 0) {
              // two query tiles: these scores were issued after the P V before
              // them; one: that P V may still be running
              ok = __all_sync(0xffffffffu, wait(B::PVDONE + ((cnt - 1) & 1), (cnt - 1) >> 1));
              if (!ok) break;
              tc::tc_fence_after();
            }
            const float mx = row_max() - P_SHIFT;
            const float m_new = mx > m_used ? mx : m_used;
            const float alpha = tc::ex2(m_used - m_new);
            l *= alpha;
            if (j > 0) {
#pragma unroll 1
              for (int cb = 0; cb < D / 16; ++cb) {   // 16 columns at a time: the scores stay live
                uint32_t o[16];
                tc::tmem_ld16(tO + cb * 16, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                tc::tmem_st16(tO + cb * 16, o);
              }
            }
            m_used = m_new;
          }
          if (!ok) break;
          l += ts;
        }
        if (r0 + BN > pc.kv) {
          // value rows past the keys (the rest of a page, another request's
          // states, or whatever the stage held before); with two query tiles
          // each sees to it before its own P V, both write the same zeros
          ok = __all_sync(0xffffffffu, wait(B::VFULL + gt % VST, gt / VST));
          if (r0 + row >= pc.kv) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              *reinterpret_cast<uint4*>(smem + C::V_OFF + (gt % VST) * C::KT + (c >> 3) * C::HALF + row * 128 +
                                        (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          tc::fence_proxy_async_smem();
        }
        if (active) {
          tc::tmem_wait_st();
          tc::tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(B::PFULL + x));
      }
      {
        // (two query tiles: one commit per piece, one: one per tile)
        const int c = cnt - 1, x = NQ == 2 ? i : c & 1, ph = NQ == 2 ? pcs++ : c >> 1;
        if (ok) ok = __all_sync(0xffffffffu, wait(B::PVDONE + x, ph));
        if (!ok) break;
      }
      tc::tc_fence_after();
      const int hq = pc.h * p.G + gq, trow = pc.row0 + i * p.TQ + tok;
      uint16_t* orow = a.out + ((size_t)(valid ? trow : 0) * a.Hq + hq) * D;
      const int slot = pc.sums >> 2;
      float2* ml = reinterpret_cast<float2*>(p.ws_ml) + ((size_t)slot * NQ + i) * BM + row;
      if (active && (pc.sums & ADDS)) {
        // add the sums of the part before, which this thread left there (a row
        // sum of 0: no visible key); rows of no token take whatever is there
        const float2 old = *ml;
        const float m = old.y == 0.f ? m_used : l == 0.f ? old.x : fmaxf(old.x, m_used);
        const float w_new = l == 0.f ? 0.f : exp2f(m_used - m), w_old = old.y == 0.f ? 0.f : exp2f(old.x - m);
        l = w_new * l + w_old * old.y;
        m_used = m;
#pragma unroll 1
        for (int cb = 0; cb < D / 32; ++cb) {
          float4 x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            x[k] = *reinterpret_cast<const float4*>(p.ws_o + ws_index<D, NQ>(slot, i, cb * 8 + k, row));
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t o[16];
            tc::tmem_ld16(tO + cb * 32 + hf * 16, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 y = x[hf * 4 + k];
              o[4 * k] = __float_as_uint(w_new * __uint_as_float(o[4 * k]) + w_old * y.x);
              o[4 * k + 1] = __float_as_uint(w_new * __uint_as_float(o[4 * k + 1]) + w_old * y.y);
              o[4 * k + 2] = __float_as_uint(w_new * __uint_as_float(o[4 * k + 2]) + w_old * y.z);
              o[4 * k + 3] = __float_as_uint(w_new * __uint_as_float(o[4 * k + 3]) + w_old * y.w);
            }
            tc::tmem_st16(tO + cb * 32 + hf * 16, o);
          }
        }
        tc::tmem_wait_st();
      }
      if (active) {
        const float inv_l = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
        for (int cb = 0; cb < D / 32; ++cb) {
          float o[32];
          tc::tmem_ld32(tO + cb * 32, *reinterpret_cast<uint32_t(*)[32]>(o));
          tc::tmem_wait_ld();
          if (!valid) continue;
          if (!(pc.sums & LEAVES)) {
            uint4 pk[4];
            uint32_t* pw = reinterpret_cast<uint32_t*>(pk);
#pragma unroll
            for (int k = 0; k < 16; ++k) pw[k] = pack16<F16>(o[2 * k] * inv_l, o[2 * k + 1] * inv_l);
#pragma unroll
            for (int k = 0; k < 4; ++k) reinterpret_cast<uint4*>(orow + cb * 32)[k] = pk[k];
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<float4*>(p.ws_o + ws_index<D, NQ>(slot, i, cb * 8 + k, row)) =
                  make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        }
        if (valid && (pc.sums & LEAVES))
          *ml = make_float2(m_used, l);
        else if (valid && a.lse)
          a.lse[(size_t)hq * a.n_tok + trow] = l == 0.f ? -INFINITY : (m_used + __log2f(l)) * 0.69314718055994531f;
      }
      // O is read out: the next piece's first P V may overwrite it
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(B::OFREE + i));
    }
    if (!ok && lane == 0) set_status(a.status, SKV_DEV_TIMEOUT);
  }

  tc::tc_fence_before();
  __syncthreads();
  if (warp == C::WARP_K) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// SM count per device ordinal, asked once (threads that race store the same value)
std::atomic<int> g_sms[64];

int sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  int n = g_sms[dev].load(std::memory_order_relaxed);
  if (!n) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 152;
    g_sms[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

template <typename K>
cudaError_t set_smem_once(K kernel, int bytes, int variant) {
  static std::atomic<int> done[64][32];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && done[dev][variant].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev][variant].store(1, std::memory_order_relaxed);
  return e;
}

// Workspace: the shared units (a word of four per CTA), then (m, sum) and O of
// two pieces per CTA, the first and the last of its share (any piece between
// is a whole unit), at the larger form's rows and head size.
constexpr int MAX_CTAS = 512;
constexpr size_t WS_HEAD = MAX_CTAS * sizeof(int4);
size_t ws_ml_bytes() { return (size_t)2 * sm_count() * 2 * BM * 2 * sizeof(float); }

bool encode_3d(CUtensorMap* m, bool f16, const void* base, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
               const cuuint32_t (&box)[3]) {
  auto fn = tmap_encode_fn();
  const cuuint32_t es[3] = {1, 1, 1};
  return fn && fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                  const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t ragged_ws_bytes() { return WS_HEAD + ws_ml_bytes() + (size_t)2 * sm_count() * 2 * BM * 128 * sizeof(float); }

cudaError_t launch_ragged_attn(const RaggedArgs& a, int d, bool f16, cudaStream_t st) {
  RParams p;
  p.a = a;
  p.G = a.Hq / a.Hkv;
  p.TQ = BM / p.G;
  const bool paged = a.k_start == nullptr;
  // More tokens than one query tile per request holds, on average: two tiles
  // per unit (a request that needs one leaves the second idle).  d = 128, 32
  // query and 8 kv heads, 4 k keys: one chunk of 512 tokens 44 us wide, 54
  // narrow; four of 100, 44 and 49; 16 of 20, 57 and 51; d = 64, six requests of
  // long encodings, 202 and 333.  The host has no lengths, so padding rows and
  // idle requests count: 64 single tokens take 172 us, and 179 in 4,096 rows; a
  // chunk of 512 tokens 38, and 48 among 16 to 256 requests that are idle, one
  // of 4,096 122, and 190 to 197 among 256.
  const bool wide = a.n_tok > (long long)a.n_req * p.TQ;
  p.TB = (wide ? 2 : 1) * p.TQ;
  const int grid = min(sm_count(), MAX_CTAS);
  // what a piece's queries, first scores and epilogue take, in key tiles (0
  // instead: 68 us against 62 in a mixed batch of chunks at d = 64, 14.2
  // against 13.0 in decode of one request)
  p.unit_cost = wide ? 2 : 1;
  p.whole_slack = wide ? 8 : 6;
  p.BR = BN;
  if (paged)
    while (a.page_size % p.BR) p.BR /= 2;
  p.boxes = BN / p.BR;
  p.scale_log2 = a.sm_scale * kLog2e;
  // in cycles at the 2.07 GHz maximum clock: a slower one only lengthens it
  p.wait_cycles = (uint64_t)(min(a.wait_ns, (uint64_t)1 << 62) * 2.07);
  p.wait_poll = a.wait_ns < tc::kSuspendHintNs;
  char* ws = static_cast<char*>(a.ws);
  p.ws_unit = reinterpret_cast<int4*>(ws);
  p.ws_ml = reinterpret_cast<float*>(ws + WS_HEAD);
  p.ws_o = reinterpret_cast<float*>(ws + WS_HEAD + ws_ml_bytes());

  CUtensorMap tq, tk, tv;
  const cuuint64_t dd = (cuuint64_t)d;
  if (!encode_3d(&tq, f16, a.q, {dd, (cuuint64_t)a.Hq, (cuuint64_t)a.n_tok}, {dd * 2, (cuuint64_t)a.q_stride * 2},
                 {64, (cuuint32_t)p.G, (cuuint32_t)p.TQ}))
    return cudaErrorInvalidValue;
  for (int i = 0; i < 2; ++i) {
    const void* base = i ? a.v : a.k;
    bool ok;
    if (paged) {
      ok = encode_3d(i ? &tv : &tk, f16, base, {dd, (cuuint64_t)a.page_size, (cuuint64_t)a.n_page * a.Hkv},
                     {dd * 2, dd * 2 * a.page_size}, {64, (cuuint32_t)p.BR, 1});
    } else if (a.n_key > 0) {
      ok = encode_3d(i ? &tv : &tk, f16, base, {dd, (cuuint64_t)a.Hkv, (cuuint64_t)a.n_key},
                     {dd * 2, (cuuint64_t)(i ? a.v_stride : a.k_stride) * 2}, {64, 1, (cuuint32_t)BN});
    } else {
      (i ? tv : tk) = tq;      // no states at all: the map is never read
      ok = true;
    }
    if (!ok) return cudaErrorInvalidValue;
  }
  auto launch = [&](auto kernel, auto merge, int smem, int threads, int variant) -> cudaError_t {
    cudaError_t e = set_smem_once(kernel, smem, variant);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kernel, dim3(grid), threads, smem, st, tq, tk, tv, p);
    if (e != cudaSuccess) return e;
    return launch_dependent(merge, dim3(grid, wide ? 2 : 1, MERGE_PARTS), MT, 0, st, p);
  };
#define SKV_RAGGED(DD, FF, NN, PP, VAR)                                                                        \
  (a.wait_ns ? launch(ragged_attn_kernel<DD, FF, NN, PP, true>, merge_kernel<DD, FF, NN>, RCfg<DD, NN>::ALLOC, \
                      RCfg<DD, NN>::NT, 16 + (VAR))                                                            \
             : launch(ragged_attn_kernel<DD, FF, NN, PP, false>, merge_kernel<DD, FF, NN>, RCfg<DD, NN>::ALLOC, \
                      RCfg<DD, NN>::NT, VAR))
#define SKV_RAGGED_FORMS(DD, FF, VAR)                                                                    \
  (wide ? (paged ? SKV_RAGGED(DD, FF, 2, true, VAR) : SKV_RAGGED(DD, FF, 2, false, VAR + 1))             \
        : (paged ? SKV_RAGGED(DD, FF, 1, true, VAR + 2) : SKV_RAGGED(DD, FF, 1, false, VAR + 3)))
  if (d == 128) return f16 ? SKV_RAGGED_FORMS(128, true, 0) : SKV_RAGGED_FORMS(128, false, 4);
  return f16 ? SKV_RAGGED_FORMS(64, true, 8) : SKV_RAGGED_FORMS(64, false, 12);
#undef SKV_RAGGED_FORMS
#undef SKV_RAGGED
}

}  // namespace skv
