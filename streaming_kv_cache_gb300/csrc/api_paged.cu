// C-ABI entry points of the paged cache and cross attention: argument
// validation and kernel launches.  Nothing here allocates device memory or
// synchronises the stream.
#include <math.h>
#include <stdint.h>

#include "kernels.h"
#include "ragged.h"
#include "skv.h"

namespace {

bool aligned(const void* p, unsigned n) { return p && ((uintptr_t)p & (n - 1)) == 0; }

// a token-major tensor of `heads` heads: its pointer and token stride
bool tensor_ok(const void* p, int64_t stride, int64_t heads, int d) {
  return aligned(p, 16) && stride >= heads * d && (stride & 7) == 0;
}

// n rows of `row` elements, `stride` apart, and the contiguous output's n rows
// of out_row elements share no byte
bool apart(const void* x, int64_t stride, int64_t row, const void* out, int64_t out_row, int64_t n) {
  const char *x0 = (const char*)x, *o0 = (const char*)out;
  return o0 >= x0 + 2 * ((n - 1) * stride + row) || x0 >= o0 + 2 * n * out_row;
}

// the output is the input itself, row for row, or apart from it
bool in_place_or_apart(const void* x, int64_t stride, int64_t row, const void* out, int64_t n) {
  return (x == out && (stride == row || n == 1)) || apart(x, stride, row, out, row, n);
}

// n words of 32 bits
struct Range {
  const void* p;
  size_t n;
};
bool overlap(const Range& a, const Range& b) {
  const char *a0 = (const char*)a.p, *b0 = (const char*)b.p;
  return a.n && b.n && a0 < b0 + 4 * b.n && b0 < a0 + 4 * a.n;
}

// What every paged call needs of the pool; k, v and rope belong to some calls only.
int check_pool(const skv_paged* c) {
  if (!c) return SKV_ERR_INVALID;
  if (c->n_page < 1 || c->page_size < 16 || (c->page_size & 15) || c->max_block < 1) return SKV_ERR_INVALID;
  if ((long long)c->n_page * c->page_size > 0x7FFFFFFFLL) return SKV_ERR_INVALID;
  if (!aligned(c->block_table, 4) || !aligned(c->status, 4)) return SKV_ERR_INVALID;
  return SKV_OK;
}

int check_heads(int n_kv_head, int head_dim, int dtype) {
  if (n_kv_head < 1 || (head_dim != 64 && head_dim != 128)) return SKV_ERR_INVALID;
  if (dtype != SKV_BF16 && dtype != SKV_FP16) return SKV_ERR_INVALID;
  return SKV_OK;
}

int check_pages(const skv_paged* c) {
  int rc = check_pool(c);
  if (rc) return rc;
  if ((rc = check_heads(c->n_kv_head, c->head_dim, c->dtype))) return rc;
  if ((long long)c->n_page * c->n_kv_head > 0x7FFFFFFFLL) return SKV_ERR_INVALID;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return SKV_ERR_INVALID;
  return SKV_OK;
}

// The checks that paged_attn and cross_attn share.  SKV_OK with *empty set:
// nothing to do.
int check_attn(int n_q_head, int n_kv_head, int d, int n_req, int n_tok, const void* q, int64_t q_stride,
               const int32_t* q_start, const void* out, const float* lse, const void* ws, size_t ws_bytes,
               float sm_scale, bool* empty) {
  *empty = false;
  if (n_q_head < 1 || n_q_head % n_kv_head) return SKV_ERR_INVALID;
  if (n_q_head / n_kv_head > 128) return SKV_ERR_UNSUPPORTED;
  if (n_req < 0 || n_tok < 0) return SKV_ERR_INVALID;
  if (n_req > (1 << 30) || n_tok > (1 << 30) || (long long)n_tok * n_q_head > 0x7FFFFFFFLL) return SKV_ERR_UNSUPPORTED;
  if (!(sm_scale > 0.f) || isinf(sm_scale * skv::kLog2e)) return SKV_ERR_INVALID;
  if (n_req == 0 || n_tok == 0) {
    *empty = true;
    return SKV_OK;
  }
  if (!tensor_ok(q, q_stride, n_q_head, d) || !aligned(out, 16) || !aligned(q_start, 4)) return SKV_ERR_INVALID;
  // a unit's rows are written once its queries have been read
  if (!in_place_or_apart(q, q_stride, (int64_t)n_q_head * d, out, n_tok)) return SKV_ERR_INVALID;
  if (lse && !aligned(lse, 4)) return SKV_ERR_INVALID;
  const size_t need = skv::ragged_ws_bytes();
  if (ws_bytes < need || (need && !aligned(ws, 16))) return SKV_ERR_INVALID;
  return SKV_OK;
}

}  // namespace

extern "C" {

int kv_paged_plan(const skv_paged* cache, int32_t n_req, int32_t n_tok, const int32_t* state,
                  const int32_t* new_len, int32_t* queue, int32_t* q_start, int32_t* kv_len,
                  int32_t* next_state, int32_t* position, int32_t* slot, void* stream) {
  int rc = check_pool(cache);
  if (rc) return rc;
  if (n_req < 0 || n_tok < 0 || n_tok > (1 << 30)) return SKV_ERR_INVALID;
  if (n_req > SKV_PAGED_MAX_REQUESTS) return SKV_ERR_UNSUPPORTED;
  if (!aligned(state, 4) || !aligned(queue, 4) || !aligned(q_start, 4) || !aligned(next_state, 4))
    return SKV_ERR_INVALID;
  if (n_req && (!aligned(new_len, 4) || !aligned(kv_len, 4))) return SKV_ERR_INVALID;
  if (n_tok && (!aligned(position, 4) || !aligned(slot, 4))) return SKV_ERR_INVALID;
  // every CTA reads the lengths, the queue and the table while others write
  // already, so what is written shares no byte with anything else
  const size_t req = (size_t)n_req, tok = (size_t)n_tok;
  const Range used[] = {{state, req + 2}, {new_len, req}, {queue, (size_t)cache->n_page},
                        {cache->block_table, req * (size_t)cache->max_block}, {q_start, req + 1}, {kv_len, req},
                        {next_state, req + 2}, {position, tok}, {slot, tok}, {cache->status, 1}};
  for (int i = 2; i < 10; ++i)                     // the first two are only read
    for (int j = 0; j < i; ++j)
      if (overlap(used[i], used[j])) return SKV_ERR_INVALID;
  if ((rc = skv::check_device())) return rc;
  skv::PlanArgs a{};
  a.n_req = n_req;
  a.n_tok = n_tok;
  a.n_page = cache->n_page;
  a.page_size = cache->page_size;
  a.ps_m = skv::fastdiv_m((uint32_t)cache->page_size);
  a.max_block = cache->max_block;
  a.state = state;
  a.new_len = new_len;
  a.queue = queue;
  a.table = cache->block_table;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.next_state = next_state;
  a.position = position;
  a.slot = slot;
  a.status = cache->status;
  const cudaError_t e = skv::launch_paged_plan(a, (cudaStream_t)stream);
  return e == cudaSuccess ? SKV_OK : skv::record_cuda_error(e);
}

int kv_paged_write(const skv_paged* cache, int32_t n_q_head, int32_t n_tok, const void* q,
                   int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                   int64_t v_stride, const int32_t* position, const int32_t* slot, void* q_out,
                   void* stream) {
  int rc = check_pages(cache);
  if (rc) return rc;
  if (n_tok < 0 || n_q_head < 0 || (!q != !q_out) || (q && n_q_head < 1)) return SKV_ERR_INVALID;
  if (cache->rope ? (cache->rope_len < 1 || !aligned(cache->rope, 16)) : cache->rope_len != 0) return SKV_ERR_INVALID;
  if (n_tok == 0) return SKV_OK;
  const int d = cache->head_dim;
  if (!tensor_ok(k, k_stride, cache->n_kv_head, d) || !tensor_ok(v, v_stride, cache->n_kv_head, d))
    return SKV_ERR_INVALID;
  if (!aligned(slot, 4) || (cache->rope && !aligned(position, 4))) return SKV_ERR_INVALID;
  if (q) {
    if (!tensor_ok(q, q_stride, n_q_head, d) || !aligned(q_out, 16)) return SKV_ERR_INVALID;
    const int64_t row = (int64_t)n_q_head * d, kv_row = (int64_t)cache->n_kv_head * d;
    if (!in_place_or_apart(q, q_stride, row, q_out, n_tok) || !apart(k, k_stride, kv_row, q_out, row, n_tok) ||
        !apart(v, v_stride, kv_row, q_out, row, n_tok))
      return SKV_ERR_INVALID;
  }
  if ((rc = skv::check_device())) return rc;
  skv::WriteArgs a{};
  a.n_tok = n_tok;
  a.Hq = n_q_head;
  a.Hkv = cache->n_kv_head;
  a.n_page = cache->n_page;
  a.page_size = cache->page_size;
  a.rope_len = cache->rope_len;
  a.ps_m = skv::fastdiv_m((uint32_t)cache->page_size);
  a.q = (const uint16_t*)q;
  a.k = (const uint16_t*)k;
  a.v = (const uint16_t*)v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.position = position;
  a.slot = slot;
  a.rope = (const float2*)cache->rope;
  a.q_out = (uint16_t*)q_out;
  a.k_pages = (uint16_t*)cache->k;
  a.v_pages = (uint16_t*)cache->v;
  a.status = cache->status;
  const cudaError_t e = skv::launch_paged_write(a, d, cache->dtype == SKV_FP16, (cudaStream_t)stream);
  return e == cudaSuccess ? SKV_OK : skv::record_cuda_error(e);
}

size_t skv_attn_workspace_bytes(void) { return skv::ragged_ws_bytes(); }

int paged_attn(const skv_paged* cache, int32_t n_q_head, int32_t n_req, int32_t n_tok,
               const void* q, int64_t q_stride, const int32_t* q_start, const int32_t* kv_len,
               void* out, float* lse, void* ws, size_t ws_bytes, float sm_scale, void* stream) {
  int rc = check_pages(cache);
  if (rc) return rc;
  bool empty;
  rc = check_attn(n_q_head, cache->n_kv_head, cache->head_dim, n_req, n_tok, q, q_stride, q_start, out, lse, ws,
                  ws_bytes, sm_scale, &empty);
  if (rc || empty) return rc;
  if (!aligned(kv_len, 4)) return SKV_ERR_INVALID;
  if ((rc = skv::check_device())) return rc;
  skv::RaggedArgs a{};
  a.n_req = n_req;
  a.n_tok = n_tok;
  a.Hq = n_q_head;
  a.Hkv = cache->n_kv_head;
  a.q = (const uint16_t*)q;
  a.q_stride = q_stride;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.k = (const uint16_t*)cache->k;
  a.v = (const uint16_t*)cache->v;
  a.n_page = cache->n_page;
  a.page_size = cache->page_size;
  a.max_block = cache->max_block;
  a.table = cache->block_table;
  a.out = (uint16_t*)out;
  a.lse = lse;
  a.ws = ws;
  a.status = cache->status;
  a.sm_scale = sm_scale;
  a.wait_ns = cache->wait_ns;
  const cudaError_t e = skv::launch_ragged_attn(a, cache->head_dim, cache->dtype == SKV_FP16, (cudaStream_t)stream);
  return e == cudaSuccess ? SKV_OK : skv::record_cuda_error(e);
}

int cross_attn(const skv_states* states, int32_t n_q_head, int32_t n_req, int32_t n_tok,
               const void* q, int64_t q_stride, const int32_t* q_start, void* out, float* lse,
               void* ws, size_t ws_bytes, float sm_scale, void* stream) {
  const skv_states* s = states;
  if (!s) return SKV_ERR_INVALID;
  int rc = check_heads(s->n_kv_head, s->head_dim, s->dtype);
  if (rc) return rc;
  if (s->n_key < 0 || !aligned(s->status, 4)) return SKV_ERR_INVALID;
  if (s->n_key > (1 << 30)) return SKV_ERR_UNSUPPORTED;
  bool empty;
  rc = check_attn(n_q_head, s->n_kv_head, s->head_dim, n_req, n_tok, q, q_stride, q_start, out, lse, ws, ws_bytes,
                  sm_scale, &empty);
  if (rc || empty) return rc;
  if (s->n_key && (!tensor_ok(s->k, s->k_stride, s->n_kv_head, s->head_dim) ||
                   !tensor_ok(s->v, s->v_stride, s->n_kv_head, s->head_dim)))
    return SKV_ERR_INVALID;
  if (!aligned(s->k_start, 4) || !aligned(s->k_len, 4)) return SKV_ERR_INVALID;
  if ((rc = skv::check_device())) return rc;
  skv::RaggedArgs a{};
  a.n_req = n_req;
  a.n_tok = n_tok;
  a.Hq = n_q_head;
  a.Hkv = s->n_kv_head;
  a.q = (const uint16_t*)q;
  a.q_stride = q_stride;
  a.q_start = q_start;
  a.kv_len = s->k_len;
  a.k = (const uint16_t*)s->k;
  a.v = (const uint16_t*)s->v;
  a.k_stride = s->k_stride;
  a.v_stride = s->v_stride;
  a.k_start = s->k_start;
  a.n_key = s->n_key;
  a.out = (uint16_t*)out;
  a.lse = lse;
  a.ws = ws;
  a.status = s->status;
  a.sm_scale = sm_scale;
  a.wait_ns = s->wait_ns;
  const cudaError_t e = skv::launch_ragged_attn(a, s->head_dim, s->dtype == SKV_FP16, (cudaStream_t)stream);
  return e == cudaSuccess ? SKV_OK : skv::record_cuda_error(e);
}

}  // extern "C"
