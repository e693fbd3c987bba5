// paged_attn_weight: the attention weight that each cached key has got from a
// step's rows, added to what it had.
//
//   w[h][j] = sum over rows i that see key j and query heads g of kv head h of
//             exp(scale q_ig . k_j - lse_ig)
#include <math.h>

#include "common.cuh"
#include "evict.h"
#include "skv.h"
#include "tc.cuh"

namespace skv {

namespace {

constexpr int KT = 128;   // keys of a tile, a thread each

template <bool F16>
__device__ __forceinline__ void unpack(uint32_t w, float& lo, float& hi) {
  if constexpr (F16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    lo = f.x;
    hi = f.y;
  } else {
    lo = bf16_lo(w);
    hi = bf16_hi(w);
  }
}

template <int D, bool F16>
__global__ void __launch_bounds__(KT) attn_weight_kernel(const WeightArgs a) {
  const RaggedArgs& r = a.r;
  const int tid = threadIdx.x, G = r.Hq / r.Hkv;
  tc::grid_dep_wait();
  long long first = 0;                       // tiles of the requests before
  for (int b = 0; b < r.n_req; ++b) {
    const Span s = request_span(r, b);
    if (s.bad && blockIdx.x == 0 && tid == 0) set_status(r.status, SKV_DEV_BAD_LEN);
    if (s.L == 0 || s.kv == 0) continue;
    const int tiles = (s.kv + KT - 1) / KT;
    const long long n = (long long)tiles * r.Hkv;
    long long t = (blockIdx.x - first % gridDim.x + gridDim.x) % gridDim.x;
    first += n;
    for (; t < n; t += gridDim.x) {
      const int h = (int)(t / tiles), j = (int)(t % tiles) * KT + tid;
      if (j >= s.kv) continue;
      const int page = r.table[(size_t)b * r.max_block + j / r.page_size];
      if (page < 0 || page >= r.n_page) {
        set_status(r.status, SKV_DEV_BAD_PAGE);
        continue;
      }
      const size_t at = ((size_t)page * r.Hkv + h) * r.page_size + j % r.page_size;
      const uint4* kr = reinterpret_cast<const uint4*>(r.k + at * D);
      const int old = s.kv - s.L;            // keys before the step
      float w = 0.f;
      for (int i = max(0, j - old); i < s.L; ++i)
        for (int g = 0; g < G; ++g) {
          const uint4* qr = reinterpret_cast<const uint4*>(r.q + (s.q0 + i) * r.q_stride + (size_t)(h * G + g) * D);
          const float l = a.lse[(size_t)(h * G + g) * r.n_tok + s.q0 + i];
          float dot = 0.f;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint4 x = kr[c], y = qr[c];
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float x0, x1, y0, y1;
              unpack<F16>(xs[e], x0, x1);
              unpack<F16>(ys[e], y0, y1);
              dot += x0 * y0 + x1 * y1;
            }
          }
          if (isfinite(l)) w += expf(r.sm_scale * dot - l);
        }
      if (j >= old) a.pos[at] = a.position[s.q0 + j - old];
      a.score[at] = j < old && a.add ? a.add[at] + w : w;
    }
  }
}

}  // namespace

cudaError_t launch_attn_weight(const WeightArgs& a, int d, bool f16, cudaStream_t st) {
  auto launch = [&](auto kernel) { return launch_dependent(kernel, dim3(152 * 8), KT, 0, st, a); };
  if (d == 128) return f16 ? launch(attn_weight_kernel<128, true>) : launch(attn_weight_kernel<128, false>);
  return f16 ? launch(attn_weight_kernel<64, true>) : launch(attn_weight_kernel<64, false>);
}

}  // namespace skv
