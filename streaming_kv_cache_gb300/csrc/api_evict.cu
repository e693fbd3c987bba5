// C-ABI entry points of sampled verification and of eviction from the paged
// cache: argument validation and kernel launches.  Nothing here allocates
// device memory or synchronises the stream.
#include <math.h>
#include <stdint.h>

#include "evict.h"
#include "kernels.h"
#include "skv.h"

namespace {

bool aligned(const void* p, unsigned n) { return p && ((uintptr_t)p & (n - 1)) == 0; }

// n words of 32 bits
struct Range {
  const void* p;
  size_t n;
};
bool overlap(const Range& a, const Range& b) {
  const char *a0 = (const char*)a.p, *b0 = (const char*)b.p;
  return a.n && b.n && a0 < b0 + 4 * b.n && b0 < a0 + 4 * a.n;
}

int launched(cudaError_t e) { return e == cudaSuccess ? SKV_OK : skv::record_cuda_error(e); }

}  // namespace

extern "C" {

int verify_sampled(int32_t n_req, int32_t n_tok, int32_t n_vocab, int32_t dtype, const int32_t* q_start,
                   const int32_t* token, const void* p, int64_t p_stride, const void* q, int64_t q_stride,
                   const float* u, const float* r, const int32_t* kv_len, int32_t* accept_len,
                   int32_t* next_token, int32_t* held, int32_t* status, void* stream) {
  if (n_req < 0 || n_tok < 0 || n_vocab < 1) return SKV_ERR_INVALID;
  if (dtype != SKV_BF16 && dtype != SKV_FP16 && dtype != SKV_FP32) return SKV_ERR_INVALID;
  if (n_req > SKV_MAX_SAMPLED || n_tok > (1 << 30) || n_vocab > (1 << 30)) return SKV_ERR_UNSUPPORTED;
  if (!aligned(status, 4) || (!kv_len != !held)) return SKV_ERR_INVALID;
  if (n_req == 0) return SKV_OK;
  if (!aligned(q_start, 4) || !aligned(r, 4) || !aligned(accept_len, 4) || !aligned(next_token, 4)) return SKV_ERR_INVALID;
  if (held && (!aligned(held, 4) || !aligned(kv_len, 4))) return SKV_ERR_INVALID;
  if (n_tok) {
    const unsigned size = dtype == SKV_FP32 ? 4 : 2;
    if (!aligned(token, 4) || !aligned(u, 4) || !aligned(p, size) || p_stride < n_vocab) return SKV_ERR_INVALID;
    if (q && (!aligned(q, size) || q_stride < n_vocab)) return SKV_ERR_INVALID;
  }
  // a request's answer is written while others still read their inputs
  const size_t req = (size_t)n_req, tok = (size_t)n_tok;
  const Range used[] = {{q_start, req + 1}, {token, tok}, {u, tok}, {r, req}, {kv_len, held ? req : 0},
                        {accept_len, req}, {next_token, req}, {held, held ? req : 0}, {status, 1}};
  for (int i = 5; i < 9; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(used[i], used[j]) && !(i == 7 && j == 4 && held == kv_len)) return SKV_ERR_INVALID;
  int rc = skv::check_device();
  if (rc) return rc;
  skv::SampleArgs a{};
  a.n_req = n_req;
  a.n_tok = n_tok;
  a.n_vocab = n_vocab;
  a.q_start = q_start;
  a.token = token;
  a.p = p;
  a.q = q;
  a.p_stride = p_stride;
  a.q_stride = q_stride;
  a.u = u;
  a.r = r;
  a.kv_len = kv_len;
  a.accept_len = accept_len;
  a.next_token = next_token;
  a.held = held;
  a.status = status;
  return launched(skv::launch_verify_sampled(a, dtype, (cudaStream_t)stream));
}

}  // extern "C"
