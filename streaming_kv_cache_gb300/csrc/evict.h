// Arguments of sampled verification and of eviction from the paged cache, and
// their host-side launchers (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ragged.h"

namespace skv {

struct SampleArgs {
  int n_req, n_tok, n_vocab;
  int ctas;                   // of a request (a cluster)
  const int32_t* q_start;     // [n_req + 1]
  const int32_t* token;       // [n_tok]
  const void *p, *q;          // [n_tok][n_vocab]; q null: drafts without probabilities
  long long p_stride, q_stride;
  const float *u, *r;         // [n_tok], [n_req]
  const int32_t* kv_len;      // [n_req], null with held
  int32_t *accept_len, *next_token, *held;
  int32_t* status;
};
cudaError_t launch_verify_sampled(const SampleArgs& a, int dtype, cudaStream_t st);

struct EvictArgs {
  int n_layer, n_req, Hkv, n_page, page_size, max_block;
  uint32_t ps_m;              // fastdiv multiplier of page_size
  const int32_t* table;       // [n_req][max_block]
  const int32_t* kv_len;      // [n_req]
  const int32_t *keep, *evicted;
  int n_sink, n_recent;
  int parts;                  // CTAs of a (layer, request, kv head)
  int per_cta;                // of a plan: tokens that one of them holds
  float* score;               // pools [n_layer][n_page][Hkv][page_size]
  int32_t* pos;
  int32_t* move;
  int32_t* n_move;            // [n_layer][n_req][Hkv]
  uint16_t *k, *v;            // [n_layer][n_page][Hkv][page_size][d]
  int32_t* status;
};
cudaError_t launch_evict_plan(const EvictArgs& a, cudaStream_t st);
cudaError_t launch_evict_move(const EvictArgs& a, int d, cudaStream_t st);

// Attention weights: the queries and spans of RaggedArgs (out and v unused),
// what their attention left, and the pools of one layer.
struct WeightArgs {
  RaggedArgs r;
  const float* lse;           // [Hq][n_tok]
  const int32_t* position;    // [n_tok]
  const float* add;           // null: the weights alone
  float* score;
  int32_t* pos;
};
cudaError_t launch_attn_weight(const WeightArgs& a, int d, bool f16, cudaStream_t st);

}  // namespace skv
