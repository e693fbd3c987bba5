// paged_attn and cross_attn: attention of packed queries over each request's
// pages or packed states.
//
// One warp per (token, query head): a lane holds d/32 dimensions of the query
// and the output, every key is one dot product across the warp, and the
// softmax keeps a running maximum and sum.
#include <math.h>

#include "common.cuh"
#include "ragged.h"
#include "skv.h"

namespace skv {

namespace {

constexpr int NT = 256;

template <bool F16>
__device__ __forceinline__ float to_f32(uint16_t x) {
  return F16 ? __half2float(__ushort_as_half(x)) : __uint_as_float((uint32_t)x << 16);
}

template <int D, bool F16>
__global__ void __launch_bounds__(NT) ragged_attn_kernel(const RaggedArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = blockIdx.x * (long long)(NT / 32) + (threadIdx.x >> 5);
  const int tok = (int)(w / a.Hq), hq = (int)(w % a.Hq);
  if (tok >= a.n_tok) return;
  int b = -1;
  Span s{};
  for (int i = 0; i < a.n_req; ++i) {
    const Span t = request_span(a, i);
    if (t.bad && w == 0 && lane == 0) set_status(a.status, SKV_DEV_BAD_LEN);
    if (tok >= t.q0 && tok < t.q0 + t.L) {
      b = i;
      s = t;
    }
  }
  if (b < 0) return;
  const int h = hq / (a.Hq / a.Hkv);
  const int n = a.k_start ? s.kv : min(s.kv, s.kv - s.L + (tok - s.q0) + 1);
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = to_f32<F16>(a.q[tok * a.q_stride + (size_t)hq * D + lane * E + e]);
    o[e] = 0.f;
  }
  for (int j = 0; j < n; ++j) {
    const uint16_t *k = nullptr, *v = nullptr;
    if (a.k_start) {
      const long long r = (long long)a.k_start[b] + j;
      k = a.k + r * a.k_stride + (size_t)h * D;
      v = a.v + r * a.v_stride + (size_t)h * D;
    } else {
      const int page = a.table[(size_t)b * a.max_block + j / a.page_size];
      if (page >= 0 && page < a.n_page) {
        const size_t r = (((size_t)page * a.Hkv + h) * a.page_size + j % a.page_size) * D;
        k = a.k + r;
        v = a.v + r;
      } else if (lane == 0) {
        set_status(a.status, SKV_DEV_BAD_PAGE);
      }
    }
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) z += k ? q[e] * to_f32<F16>(k[lane * E + e]) : 0.f;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
    z *= a.sm_scale;
    const float m_new = fmaxf(m, z), al = expf(m - m_new), p = expf(z - m_new);
    l = l * al + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * al + (v ? p * to_f32<F16>(v[lane * E + e]) : 0.f);
    m = m_new;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float x = o[e] * inv;
    a.out[((size_t)tok * a.Hq + hq) * D + lane * E + e] =
        F16 ? __half_as_ushort(__float2half_rn(x)) : __bfloat16_as_ushort(__float2bfloat16_rn(x));
  }
  if (a.lse && lane == 0) a.lse[(size_t)hq * a.n_tok + tok] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t ragged_ws_bytes() { return 0; }

cudaError_t launch_ragged_attn(const RaggedArgs& a, int d, bool f16, cudaStream_t st) {
  const long long warps = (long long)a.n_tok * a.Hq;
  const unsigned grid = (unsigned)((warps + NT / 32 - 1) / (NT / 32));
  auto launch = [&](auto kernel) { kernel<<<grid, NT, 0, st>>>(a); };
  if (d == 128) f16 ? launch(ragged_attn_kernel<128, true>) : launch(ragged_attn_kernel<128, false>);
  else f16 ? launch(ragged_attn_kernel<64, true>) : launch(ragged_attn_kernel<64, false>);
  return cudaGetLastError();
}

}  // namespace skv
