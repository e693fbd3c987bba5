// Arguments of the calls over requests of different lengths (paged cache and
// cross attention), and their host-side launchers (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "skv.h"

namespace skv {

struct PlanArgs {
  int n_req, n_tok, n_page, page_size, max_block;
  uint32_t ps_m;            // fastdiv multiplier of page_size
  const int32_t* state;     // [n_req + 2] held tokens, queue head, queue count
  const int32_t* new_len;   // [n_req]
  int32_t* queue;           // [n_page] ring of free pages
  int32_t* table;           // [n_req][max_block]
  int32_t* q_start;         // [n_req + 1]
  int32_t* kv_len;          // [n_req]
  int32_t* next_state;      // [n_req + 2]
  int32_t* position;        // [n_tok]
  int32_t* slot;            // [n_tok]
  int32_t* status;
};
cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t st);

struct WriteArgs {
  int n_tok, Hq, Hkv, n_page, page_size, rope_len;
  uint32_t ps_m;            // fastdiv multiplier of page_size
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride;   // elements per token
  const int32_t *position, *slot;
  const float2* rope;       // null: copy
  uint16_t *q_out, *k_pages, *v_pages;
  int32_t* status;
};
cudaError_t launch_paged_write(const WriteArgs& a, int d, bool f16, cudaStream_t st);

// Attention of packed queries over each request's keys: pages (table given)
// or packed states (k_start given).
struct RaggedArgs {
  int n_req, n_tok, Hq, Hkv;
  const uint16_t* q;
  long long q_stride;
  const int32_t* q_start;   // [n_req + 1]
  const int32_t* kv_len;    // [n_req]
  const uint16_t *k, *v;
  int n_page, page_size, max_block;
  const int32_t* table;
  long long k_stride, v_stride;
  const int32_t* k_start;   // [n_req], null: paged
  int n_key;
  uint16_t* out;
  float* lse;
  void* ws;
  int32_t* status;
  float sm_scale;
  uint64_t wait_ns;         // limit of a wait, 0: two seconds
};
constexpr float kLog2e = 1.4426950408889634f;   // the softmax works to base two: its scale times this
cudaError_t launch_ragged_attn(const RaggedArgs& a, int d, bool f16, cudaStream_t st);
size_t ragged_ws_bytes();

// Launch as a programmatic dependent of the kernel before it on the stream:
// its CTAs may start as that one's last ones leave, and wait for it
// (grid_dep_wait) before they read or write anything of the caller's.  They
// read none of it through the read-only path: it may change after they start.
// The kernels themselves give no early signal to the ones after them: CTAs that
// start only to wait took SM slots and launch bandwidth (a plan of 2048
// requests 15.7 us in a row of plans, 8.2 without; a decode call 13.6 and 12.9,
// 17.1 without the dependent launch).
template <typename... K, typename... A>
cudaError_t launch_dependent(void (*kernel)(K...), dim3 grid, int threads, int smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// One request as the attention sees it: rows [q0, q0 + L) of the queries, kv
// keys; row t sees the first kv - L + t + 1 of them (paged) or all (states).
// Lengths out of range make it harmless: a bad span has no rows, bad keys
// are none.  The limit on a request's keys keeps every index in 32 bits, and a
// unit's stay in one CTA (half a million key tiles) under the two seconds
// after which a wait gives up.
constexpr int kMaxKeys = SKV_MAX_KEYS;
struct Span {
  int q0, L, kv;
  bool bad;
};
__device__ __forceinline__ Span request_span(const RaggedArgs& a, int b) {
  Span s;
  const int lo = a.q_start[b], hi = a.q_start[b + 1];
  s.bad = lo < 0 || hi < lo || hi > a.n_tok;
  s.q0 = s.bad ? 0 : lo;
  s.L = s.bad ? 0 : hi - lo;
  s.kv = a.kv_len[b];
  bool kv_ok;
  if (a.k_start) {
    const int k0 = a.k_start[b];
    kv_ok = k0 >= 0 && s.kv >= 0 && s.kv <= kMaxKeys && (long long)k0 + s.kv <= a.n_key;
  } else {
    kv_ok = s.kv == 0 || (s.kv >= s.L && s.kv <= min((long long)a.max_block * a.page_size, (long long)kMaxKeys));
  }
  if (!kv_ok) {
    s.kv = 0;
    s.bad = true;
  }
  return s;
}

}  // namespace skv
