// verify_sampled: drafted tokens accepted by the target's and the drafter's
// probabilities, and the token that follows them, from given random numbers.
//
//   draft x after row i is accepted iff u_i q_i(x) < p_i(x);
//   the token after the last accepted draft is the smallest index whose
//   running sum of w passes r sum w, with w = max(p - q, 0) of the row where a
//   draft was rejected, w = p of the last row where none was
//
// The comparison is exact: the product of two 24-bit significands fits a
// double.  So are the sums, up to 2^-56 per entry: probabilities are summed as
// whole numbers of 2^-55, which come out the same in any order, so that the
// token does not depend on how a row is split over threads (sums in fp32 would
// move the borders between tokens by about 1e-9, and one draw in some
// thousands over a vocabulary of 151,936 lies nearer to one than that).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "evict.h"
#include "skv.h"
#include "tc.cuh"

namespace skv {

namespace {

constexpr int VT = 512;               // threads per CTA
constexpr int NW = VT / 32;
constexpr float FIX = 36028797018963968.f;      // 2^55: the unit of the sums
constexpr float MOST = 2.f;                     // an entry above is no probability
constexpr uint64_t LIMIT = 1ull << 58;          // nor a row whose sum passes 8

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float value(__half x) { return __half2float(x); }

__device__ __forceinline__ bool is_prob(float x) { return x >= 0.f && x <= MOST; }   // false for NaN
__device__ __forceinline__ float prob(float x) { return is_prob(x) ? x : 0.f; }
__device__ __forceinline__ long long fixed(float x) { return __float2ll_rn(x * FIX); }

enum Mode { REST, FULL, WITHOUT };    // max(p - q, 0); p; p but for the rejected token

template <typename T>
__global__ void __launch_bounds__(VT) verify_sampled_kernel(const SampleArgs a) {
  __shared__ unsigned long long s_warp[NW];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  tc::grid_dep_wait();
  const int lo = a.q_start[b], hi = a.q_start[b + 1];
  const bool bad = lo < 0 || hi < lo || hi > a.n_tok;
  const int n = bad ? 0 : hi - lo;
  if (n == 0) {
    if (tid == 0) {
      if (bad) set_status(a.status, SKV_DEV_BAD_LEN);
      a.accept_len[b] = 0;
      a.next_token[b] = -1;
      if (a.held) a.held[b] = a.kv_len[b];
    }
    return;
  }
  const T* P = static_cast<const T*>(a.p);
  const T* Q = static_cast<const T*>(a.q);

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
  if (tid == 0) {
    if (acc < n - 1 && (x < 0 || x >= a.n_vocab)) set_status(a.status, SKV_DEV_BAD_TOKEN);
    a.accept_len[b] = acc;
    if (a.held) a.held[b] = a.kv_len[b] - n + acc + 1;
  }

  const T* prow = P + (lo + acc) * a.p_stride;
  const T* qrow = Q ? Q + (lo + acc) * a.q_stride : nullptr;
  int mode = acc == n - 1 ? FULL : Q ? REST : WITHOUT;
  // entry i of the distribution, in units of 2^-55
  bool odd = false;                   // an entry that is no probability
  auto entry = [&](int i) -> unsigned long long {
    const float pv = value(prow[i]);
    odd |= !is_prob(pv);
    long long w = fixed(prob(pv));
    if (mode == REST) {
      const float qv = value(qrow[i]);
      odd |= !is_prob(qv);
      w = max(w - fixed(prob(qv)), 0LL);
    }
    return mode == WITHOUT && i == x ? 0ull : (unsigned long long)w;
  };
  // a warp takes a run of the vocabulary
  const int per = (a.n_vocab + NW * 32 - 1) / (NW * 32) * 32;
  const int i0 = min((long long)a.n_vocab, (long long)warp * per), i1 = min((long long)a.n_vocab, (long long)i0 + per);
  for (;;) {
    unsigned long long s = 0;
    bool over = false;
    for (int i = i0 + lane; i < i1; i += 32) {
      s += entry(i);
      if (s > LIMIT) {
        over = true;
        s = 0;
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    over = __any_sync(0xffffffffu, over) || s > LIMIT;
    __syncthreads();
    if (lane == 0) s_warp[warp] = over ? LIMIT + 1 : s;
    __syncthreads();
    unsigned long long total = 0, before = 0;
    for (int w = 0; w < NW; ++w) {
      if (w == warp) before = total;
      total += s_warp[w];
      over |= s_warp[w] > LIMIT;
    }
    if (total == 0 && mode != FULL) {   // nothing is left of p: p itself
      mode = FULL;
      continue;
    }
    if (over || total == 0 || total > LIMIT) {
      if (tid == 0) {
        a.next_token[b] = -1;
        set_status(a.status, SKV_DEV_BAD_PROB);
      }
      break;
    }
    const float r = a.r[b];
    // a running sum passes r total iff it passes its whole part; NaN: the first entry
    const unsigned long long at = r > 0.f ? min(total - 1, (unsigned long long)((double)total * (double)fminf(r, 1.f))) : 0ull;
    if (at >= before && at - before < s) {
      unsigned long long run = before;
      for (int i = i0 + lane;; i += 32) {
        const unsigned long long w = i < i1 ? entry(i) : 0ull;
        unsigned long long incl = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long t = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += t;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, run + incl > at);
        if (past) {
          if (lane == __ffs(past) - 1) a.next_token[b] = i;
          break;
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    break;
  }
  if (__any_sync(0xffffffffu, odd) && lane == 0) set_status(a.status, SKV_DEV_BAD_PROB);
}

}  // namespace

cudaError_t launch_verify_sampled(const SampleArgs& a, int dtype, cudaStream_t st) {
  auto launch = [&](auto kernel) { return launch_dependent(kernel, dim3((unsigned)a.n_req), VT, 0, st, a); };
  if (dtype == SKV_FP32) return launch(verify_sampled_kernel<float>);
  return dtype == SKV_FP16 ? launch(verify_sampled_kernel<__half>) : launch(verify_sampled_kernel<__nv_bfloat16>);
}

}  // namespace skv
