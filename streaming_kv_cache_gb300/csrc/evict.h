// Arguments of sampled verification and of eviction from the paged cache, and
// their host-side launchers (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ragged.h"

namespace skv {

struct SampleArgs {
  int n_req, n_tok, n_vocab;
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

}  // namespace skv
