// verify_sampled: drafted tokens accepted by the target's and the drafter's
// probabilities, and the token that follows them, from given random numbers.
//
//   draft x after row i is accepted iff u_i q_i(x) < p_i(x);
//   the token after the last accepted draft is the smallest index whose
//   running sum of w passes r sum w, with w = max(p - q, 0) of the row where a
//   draft was rejected, w = p of the last row where none was
//
// The comparison is exact: the product of two 24-bit significands fits a
// double.  So are the sums, up to 2^-55 per entry: probabilities are summed as
// whole numbers of 2^-55, which come out the same in any order, and r times
// their sum is cut to a whole number without rounding, so that the
// token does not depend on how a row is split over threads (sums in fp32 would
// move the borders between tokens by about 1e-9, and one draw in some
// thousands over a vocabulary of 151,936 lies nearer to one than that).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"
#include "evict.h"
#include "skv.h"
#include "tc.cuh"

namespace skv {

namespace {

constexpr int VT = 512;               // threads per CTA, at most
constexpr int NW = VT / 32;
constexpr int MAX_CLUSTER = 16;       // CTAs of a request, at most
constexpr float MOST = 2.f;                     // an entry above is no probability
constexpr uint64_t LIMIT = 1ull << 58;          // nor a row whose sum passes 8

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float value(__half x) { return __half2float(x); }

__device__ __forceinline__ bool is_prob(float x) { return x >= 0.f && x <= MOST; }   // false for NaN
__device__ __forceinline__ float prob(float x) { return is_prob(x) ? x : 0.f; }

// An entry in units of 2^-55, cut: its 24-bit significand shifted by its
// exponent.  Sets odd and gives 0 for what is no probability.
__device__ __forceinline__ long long fixed(float x, bool& odd) {
  const uint32_t u = __float_as_uint(x);
  const bool ok = u <= __float_as_uint(MOST);          // not for a sign, nor NaN
  odd |= !ok && u != 0x80000000u;                      // -0 is 0
  const uint32_t top = ((u & 0x7FFFFFu) | 0x800000u) << 1;
  const uint32_t s = min(128u - (u >> 23), 63u);       // zeros and subnormals go out
  return ok ? (long long)(((uint64_t)top << 32) >> s) : 0;
}

// The same for many entries in [0, 2], as three whole numbers of 32 bits in
// units of 2^-19, 2^-42 and 2^-55 that sums are taken of one by one.  Added
// to 16 and cut, an entry leaves its first part in the sum's low bits; what it
// lacks is exact, and goes on to 2^-19 and 2^-32.  Seven additions and no
// 64-bit arithmetic: fixed() takes 17 instructions, and a conversion to 64 bits
// ten times as long (64 requests over 151,936 entries: 55 us with the
// conversion, 34 with fixed(), 20.8 so).
struct Limbs {
  uint32_t a, b, c;
};
__device__ __forceinline__ Limbs limbs(float x) {
  const float a = __fadd_rz(x, 16.f), r = x - (a - 16.f);
  const float b = __fadd_rz(r, 0x1p-19f), q = r - (b - 0x1p-19f);
  return {__float_as_uint(a), __float_as_uint(b), __float_as_uint(__fadd_rz(q, 0x1p-32f))};
}

// The whole part of r total, exact, for r below 1 (of r <= 0: 0) and total up to 2^58:
// r is its significand times 2^-s, s at least 24.  In doubles the product would be off
// by up to 6, a total of 2^55 having 56 bits.
__device__ __forceinline__ unsigned long long share_of(unsigned long long total, float r) {
  if (!(r > 0.f)) return 0;
  const uint32_t u = __float_as_uint(r), e = max(u >> 23, 1u), s = 150 - e;
  const unsigned long long m = (u & 0x7FFFFFu) | (u >> 23 ? 0x800000u : 0u);
  const unsigned long long lo = total * m, hi = __umul64hi(total, m);      // hi below 2^18
  return s < 64 ? hi << (64 - s) | lo >> s : s < 128 ? hi >> (s - 64) : 0;
}

enum Mode { REST, FULL, WITHOUT };    // max(p - q, 0); p; p but for the rejected token

// One cluster per request: its CTAs' warps take runs of the row and sum them;
// the CTA whose part holds the draw goes over one warp's run once more, out of
// L1 or L2.  One request is bound by latency (9.7 us for 8 drafts over 151,936
// entries), many by that chain and HBM (64 requests 20.8 us, 0.55 of its rate).
// VEC: rows start on 16-byte boundaries and are read 16 bytes a lane; else an
// entry a lane.
template <typename T, bool VEC>
__global__ void __launch_bounds__(VT, 2) verify_sampled_kernel(const SampleArgs a) {
  constexpr int W = VEC ? 16 / (int)sizeof(T) : 1;   // entries of a lane at a time
  constexpr int U = VEC ? (sizeof(T) == 4 ? 4 : 2) : 8;   // loads of each row in flight
  __shared__ unsigned long long s_warp[NW], s_part[NW];
  __shared__ unsigned long long s_total[2][MAX_CLUSTER];
  const int nw = blockDim.x >> 5;                    // warps of the CTA
  const int ctas = a.ctas, rank = ctas > 1 ? (int)tc::cluster_ctarank() : 0;
  const int b = blockIdx.x / ctas, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (ctas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // it has started
  tc::grid_dep_wait();
  const int lo = a.q_start[b], hi = a.q_start[b + 1];
  const bool bad = lo < 0 || hi < lo || hi > a.n_tok;
  const int n = bad ? 0 : hi - lo;
  if (n == 0) {
    if (ctas > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (tid == 0 && rank == 0) {
      if (bad) set_status(a.status, SKV_DEV_BAD_LEN);
      a.accept_len[b] = 0;
      a.next_token[b] = -1;
      if (a.held) a.held[b] = a.kv_len[b];
    }
    return;
  }
  const T* P = static_cast<const T*>(a.p);
  const T* Q = static_cast<const T*>(a.q);
  const float r = a.r[b];

  // accepted drafts: every warp finds out for itself, a lane per draft
  int acc = n - 1, x = -1;            // x: the draft that was rejected
  for (int j0 = 0; j0 < n - 1; j0 += 32) {
    const int j = j0 + lane;
    int t = -1;
    bool ok = true;
    if (j < n - 1) {
      t = a.token[lo + j + 1];
      ok = false;
      if (t >= 0 && t < a.n_vocab) {
        const float pt = prob(value(P[(lo + j) * a.p_stride + t]));
        const float qt = Q ? prob(value(Q[(lo + j) * a.q_stride + t])) : 1.f;
        ok = (double)a.u[lo + j] * (double)qt < (double)pt;
      }
    }
    const uint32_t no = __ballot_sync(0xffffffffu, !ok);
    if (no) {
      const int l = __ffs(no) - 1;
      acc = j0 + l;
      x = __shfl_sync(0xffffffffu, t, l);
      break;
    }
  }
  if (tid == 0 && rank == 0) {
    if (acc < n - 1 && (x < 0 || x >= a.n_vocab)) set_status(a.status, SKV_DEV_BAD_TOKEN);
    a.accept_len[b] = acc;
    if (a.held) a.held[b] = a.kv_len[b] - n + acc + 1;
  }

  const T* prow = P + (lo + acc) * a.p_stride;
  const T* qrow = Q ? Q + (lo + acc) * a.q_stride : nullptr;
  int mode = acc == n - 1 ? FULL : Q ? REST : WITHOUT;
  bool odd = false;                   // an entry that is no probability
  // entries [i, i + W) of a row; those past its end are 0
  struct Entries {
    T v[W];
  };
  auto load = [&](const T* row, int i) {
    Entries e{};
    if (i + W <= a.n_vocab) {
      if constexpr (VEC) {
        const uint4 raw = *reinterpret_cast<const uint4*>(row + i);
        e = *reinterpret_cast<const Entries*>(&raw);
      } else {
        e.v[0] = row[i];
      }
    } else if (VEC && i < a.n_vocab) {
#pragma unroll
      for (int k = 0; k < W; ++k)
        if (i + k < a.n_vocab) e.v[k] = row[i + k];
    }
    return e;
  };
  // entry i + k of the distribution, in units of 2^-55
  auto weight = [&](const Entries& pe, const Entries& qe, int i, int k) -> unsigned long long {
    long long w = fixed(value(pe.v[k]), odd);
    if (mode == REST) w = max(w - fixed(value(qe.v[k]), odd), 0LL);
    return mode == WITHOUT && i + k == x ? 0ull : (unsigned long long)w;
  };
  // this warp's run: chunks [c0, c1) of 32 W entries
  const int chunks = (a.n_vocab + 32 * W - 1) / (32 * W), warps = ctas * nw, gw = rank * nw + warp;
  const int c0 = (int)((long long)gw * chunks / warps), c1 = (int)((long long)(gw + 1) * chunks / warps);
  for (int round = 0;; ++round) {
    unsigned long long s = 0;
    bool over = false;
    uint32_t most = 0;                // of the entries' bits: above those of 2 with a sign, a NaN or a large one
    for (int c = c0; c < c1; c += U) {
      Entries pe[U], qe[U];
#pragma unroll
      for (int v = 0; v < U; ++v) {
        const int i = c + v < c1 ? ((c + v) * 32 + lane) * W : a.n_vocab;
        pe[v] = load(prow, i);
        qe[v] = mode == REST ? load(qrow, i) : Entries{};
      }
      int da = 0, db = 0, dc = 0;
#pragma unroll
      for (int v = 0; v < U; ++v)
#pragma unroll
        for (int k = 0; k < W; ++k) {
          const float pv = value(pe[v].v[k]), qv = value(qe[v].v[k]);
          most = max(max(most, __float_as_uint(pv)), __float_as_uint(qv));
          const Limbs x1 = limbs(pv), x2 = limbs(fminf(pv, qv));     // max(p - q, 0) = p - min(p, q)
          da += x1.a - x2.a;
          db += x1.b - x2.b;
          dc += x1.c - x2.c;
        }
      s += ((long long)da << 36) + ((long long)db << 13) + dc;
      if (s > LIMIT) {
        over = true;
        s = 0;
      }
    }
    if (most > __float_as_uint(MOST)) {
      // once more, entry by entry
      s = 0;
      over = false;
      for (int c = c0; c < c1; ++c) {
        const int i = (c * 32 + lane) * W;
        const Entries pe = load(prow, i), qe = mode == REST ? load(qrow, i) : Entries{};
#pragma unroll
        for (int k = 0; k < W; ++k) s += weight(pe, qe, i, k);
        if (s > LIMIT) {
          over = true;
          s = 0;
        }
      }
    } else if (mode == WITHOUT && x >= 0 && x < a.n_vocab && x / W / 32 >= c0 && x / W / 32 < c1 && x / W % 32 == lane) {
      s -= fixed(value(prow[x]), odd);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    over = __any_sync(0xffffffffu, over) || s > LIMIT;
    if (over) s = LIMIT + 1;
    if (lane == 0) s_warp[warp] = s;
    __syncthreads();
    // sums of the CTA's warps, then of the cluster's CTAs; a sum that is too
    // large stays so
    unsigned long long mine = 0, before = 0;     // of this CTA, and of those before it
    for (int w = 0; w < nw; ++w) mine += s_warp[w];
    mine = min(mine, (unsigned long long)LIMIT + 1);
    unsigned long long total = mine;
    if (ctas > 1) {
      if (round == 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // all have started
      if (tid < ctas) {
        const uint32_t to = tc::map_to_cta(tc::smem_u32(&s_total[round][rank]), (uint32_t)tid);
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(mine) : "memory");
      }
      tc::cluster_sync();
      total = 0;
      for (int c = 0; c < ctas; ++c) {
        if (c == rank) before = total;
        total += s_total[round][c];
      }
    }
    if (total == 0 && mode != FULL) {   // nothing is left of p: p itself
      mode = FULL;
      __syncthreads();
      continue;
    }
    if (total == 0 || total > LIMIT) {
      if (tid == 0 && rank == 0) {
        a.next_token[b] = -1;
        set_status(a.status, SKV_DEV_BAD_PROB);
      }
      break;
    }
    // a running sum passes r total iff it passes its whole part; NaN: the first entry
    const unsigned long long at = r < 1.f ? share_of(total, r) : r >= 1.f ? total - 1 : 0ull;
    if (at >= before && at - before < mine) {
      // This CTA's part of the row has it.  The run of the warp that it falls
      // in is gone over by all warps, SU chunks each at a time: by that warp
      // alone, a load's latency for every chunk, it took 12 of 38 us.
      constexpr int SU = 2;
      unsigned long long run = before;
      int w = 0;
      while (at - run >= s_warp[w]) run += s_warp[w++];
      const int first = (int)((long long)(rank * nw + w) * chunks / warps);
      const int last = (int)((long long)(rank * nw + w + 1) * chunks / warps);
      for (int c = first; c < last; c += nw * SU) {
        unsigned long long part[SU][W], sum = 0;
        const int mc = c + warp * SU;
        Entries pe[SU], qe[SU];
#pragma unroll
        for (int v = 0; v < SU; ++v) {
          const int i = mc + v < last ? ((mc + v) * 32 + lane) * W : a.n_vocab;
          pe[v] = load(prow, i);
          qe[v] = mode == REST ? load(qrow, i) : Entries{};
        }
        unsigned long long chunk_sum[SU];
#pragma unroll
        for (int v = 0; v < SU; ++v) {
          chunk_sum[v] = 0;
#pragma unroll
          for (int k = 0; k < W; ++k) {
            part[v][k] = weight(pe[v], qe[v], ((mc + v) * 32 + lane) * W, k);
            chunk_sum[v] += part[v][k];
          }
          sum += chunk_sum[v];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s_part[warp] = sum;
        __syncthreads();
        int f = 0;                       // the warp whose chunks hold it
        while (f < nw && at - run >= s_part[f]) run += s_part[f++];
        if (f == warp) {
#pragma unroll
          for (int v = 0; v < SU; ++v) {
            unsigned long long incl = chunk_sum[v];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const unsigned long long t = __shfl_up_sync(0xffffffffu, incl, o);
              if (lane >= o) incl += t;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, run + incl > at);
            if (past) {
              if (lane == __ffs(past) - 1) {
                unsigned long long cum = run + incl - chunk_sum[v];
                int found = ((mc + v) * 32 + lane) * W;
#pragma unroll
                for (int k = 0; k < W; ++k) {
                  cum += part[v][k];
                  found += cum <= at;    // the first that passes, and none after it counts
                }
                a.next_token[b] = found;
              }
              break;
            }
            run += __shfl_sync(0xffffffffu, incl, 31);
          }
        }
        if (f < nw) break;
        __syncthreads();
      }
    }
    break;
  }
  if (__any_sync(0xffffffffu, odd) && lane == 0) set_status(a.status, SKV_DEV_BAD_PROB);
}

// CTAs that a cluster may have: 16 where the device can hold one so large (more
// than 8 is not portable), asked once per device and kernel.
template <typename T, typename K>
cudaError_t largest_cluster(K kernel, int variant, int& most) {
  static std::atomic<int> known[64][2];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  most = dev >= 0 && dev < 64 ? known[dev][variant].load(std::memory_order_relaxed) : 0;
  if (most) return cudaSuccess;
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = MAX_CLUSTER;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3(MAX_CLUSTER);
  cfg.blockDim = dim3(VT);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int fit = 0;
  e = cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg);
  if (e != cudaSuccess) return e;
  most = fit > 0 ? MAX_CLUSTER : 8;
  if (dev >= 0 && dev < 64) known[dev][variant].store(most, std::memory_order_relaxed);
  return cudaSuccess;
}

template <typename T>
cudaError_t launch(const SampleArgs& in, cudaStream_t st) {
  SampleArgs a = in;
  const bool vec = ((uintptr_t)a.p | (uintptr_t)a.q) % 16 == 0 && a.p_stride * sizeof(T) % 16 == 0 &&
                   (!a.q || a.q_stride * sizeof(T) % 16 == 0);
  // Few requests: large CTAs and clusters (one request in a cluster of 8 13.4 us,
  // of 16 9.3); many: all CTAs at once (64 requests with clusters of 4 and 256
  // threads 50 us, of 8 38).  304: two CTAs for each of the 152 SMs.
  const int threads = a.n_req < 16 ? VT : VT / 2;
  auto kernel = vec ? verify_sampled_kernel<T, true> : verify_sampled_kernel<T, false>;
  int most = 8;
  if (a.n_req * 8 < 304) {
    const cudaError_t e = largest_cluster<T>(kernel, vec, most);
    if (e != cudaSuccess) return e;
  }
  a.ctas = 1;
  while (a.ctas < most && a.ctas * a.n_req < 304 && a.n_vocab > a.ctas * 2048) a.ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)a.n_req * a.ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = a.ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_verify_sampled(const SampleArgs& a, int dtype, cudaStream_t st) {
  if (dtype == SKV_FP32) return launch<float>(a, st);
  return dtype == SKV_FP16 ? launch<__half>(a, st) : launch<__nv_bfloat16>(a, st);
}

}  // namespace skv
