// C-ABI entry points of sampled verification and of eviction from the paged
// cache: argument validation and kernel launches.  Nothing here allocates
// device memory or synchronises the stream.
#include <math.h>
#include <stdint.h>

#include "checks.h"
#include "evict.h"
#include "kernels.h"
#include "skv.h"

using namespace skv::checks;

namespace {

// entries of a pool of one word per token and kv head
size_t pool_words(const skv_paged* c) { return (size_t)c->n_page * c->n_kv_head * c->page_size; }

// no output shares a byte with anything else of the call; used: inputs, then outputs
template <int N>
bool apart(const Range (&used)[N], int n_in) {
  for (int i = n_in; i < N; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(used[i], used[j])) return false;
  return true;
}

// the pool as the eviction calls use it, and how many (layer, request, kv head) there are
int check_layers(const skv_paged* c, int32_t n_layer, int32_t n_req) {
  int rc = check_pool(c);
  if (rc) return rc;
  if (c->n_kv_head < 1 || (long long)c->n_page * c->n_kv_head > 0x7FFFFFFFLL || n_layer < 0 || n_req < 0)
    return SKV_ERR_INVALID;
  if ((double)n_layer * n_req * c->n_kv_head > (1 << 26)) return SKV_ERR_UNSUPPORTED;
  return SKV_OK;
}

skv::EvictArgs evict_args(const skv_paged* c, int32_t n_layer, int32_t n_req, const int32_t* kv_len) {
  skv::EvictArgs a{};
  a.n_layer = n_layer;
  a.n_req = n_req;
  a.Hkv = c->n_kv_head;
  a.n_page = c->n_page;
  a.page_size = c->page_size;
  a.max_block = c->max_block;
  a.ps_m = skv::fastdiv_m((uint32_t)c->page_size);
  a.table = c->block_table;
  a.kv_len = kv_len;
  a.status = c->status;
  return a;
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
  // a request's answer is written while others still read their inputs; held
  // in place of kv_len is read and written by one thread
  const size_t req = (size_t)n_req, tok = (size_t)n_tok;
  const Range used[] = {{q_start, req + 1}, {token, tok}, {u, tok}, {r, req}, {kv_len, held && held != kv_len ? req : 0},
                        {accept_len, req}, {next_token, req}, {held, held ? req : 0}, {status, 1}};
  if (!apart(used, 5)) return SKV_ERR_INVALID;
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

int paged_attn_weight(const skv_paged* cache, int32_t n_q_head, int32_t n_req, int32_t n_tok, const void* q,
                      int64_t q_stride, const int32_t* q_start, const int32_t* kv_len, const float* lse,
                      const int32_t* position, const float* add, float* score, int32_t* pos, void* ws,
                      size_t ws_bytes, float sm_scale, void* stream) {
  const skv_paged* c = cache;
  int rc = check_pool(c);
  if (rc) return rc;
  if ((rc = check_heads(c->n_kv_head, c->head_dim, c->dtype))) return rc;
  if ((long long)c->n_page * c->n_kv_head > 0x7FFFFFFFLL || !aligned(c->k, 16)) return SKV_ERR_INVALID;
  if (n_q_head < 1 || n_q_head % c->n_kv_head || n_req < 0 || n_tok < 0) return SKV_ERR_INVALID;
  if (n_q_head / c->n_kv_head > 128 || n_req > SKV_PAGED_MAX_REQUESTS) return SKV_ERR_UNSUPPORTED;
  // a unit's query tiles, a microsecond or two each, end long before a wait gives up
  if (n_tok > (1 << 18) * (128 / (n_q_head / c->n_kv_head)) || (long long)n_tok * n_q_head > 0x7FFFFFFFLL)
    return SKV_ERR_UNSUPPORTED;
  if (!(sm_scale > 0.f) || isinf(sm_scale * skv::kLog2e)) return SKV_ERR_INVALID;
  if (n_req == 0 || n_tok == 0) return SKV_OK;
  if (!tensor_ok(q, q_stride, n_q_head, c->head_dim) || !aligned(q_start, 4) || !aligned(kv_len, 4)) return SKV_ERR_INVALID;
  if (!aligned(lse, 4) || !aligned(position, 4) || !aligned(score, 4) || !aligned(pos, 4)) return SKV_ERR_INVALID;
  if (add && !aligned(add, 4)) return SKV_ERR_INVALID;
  const size_t need = skv::ragged_ws_bytes();
  if (ws_bytes < need || (need && !aligned(ws, 16))) return SKV_ERR_INVALID;
  const size_t pool = pool_words(c), req = (size_t)n_req, tok = (size_t)n_tok;
  // weights are added in place by the thread that reads them, or apart
  const Range used[] = {{q, ((tok - 1) * (size_t)q_stride + (size_t)n_q_head * c->head_dim) / 2},
                        {c->k, pool * c->head_dim / 2}, {q_start, req + 1}, {kv_len, req}, {lse, tok * n_q_head},
                        {position, tok}, {add, add && add != score ? pool : 0}, {c->block_table, req * (size_t)c->max_block},
                        {score, pool}, {pos, pool}, {ws, need / 4}, {c->status, 1}};
  if (!apart(used, 8)) return SKV_ERR_INVALID;
  if ((rc = skv::check_device())) return rc;
  skv::WeightArgs a{};
  a.r.n_req = n_req;
  a.r.n_tok = n_tok;
  a.r.Hq = n_q_head;
  a.r.Hkv = c->n_kv_head;
  a.r.q = (const uint16_t*)q;
  a.r.q_stride = q_stride;
  a.r.q_start = q_start;
  a.r.kv_len = kv_len;
  a.r.k = (const uint16_t*)c->k;
  a.r.n_page = c->n_page;
  a.r.page_size = c->page_size;
  a.r.max_block = c->max_block;
  a.r.table = c->block_table;
  a.r.ws = ws;
  a.r.status = c->status;
  a.r.sm_scale = sm_scale;
  a.r.wait_ns = c->wait_ns;
  a.lse = lse;
  a.position = position;
  a.add = add;
  a.score = score;
  a.pos = pos;
  return launched(skv::launch_attn_weight(a, c->head_dim, c->dtype == SKV_FP16, (cudaStream_t)stream));
}

int kv_evict_plan(const skv_paged* cache, int32_t n_layer, int32_t n_req, const int32_t* kv_len,
                  const int32_t* keep, const int32_t* evicted, int32_t n_sink, int32_t n_recent,
                  const float* score, const int32_t* pos, int32_t* move, int32_t* n_move, void* stream) {
  int rc = check_layers(cache, n_layer, n_req);
  if (rc) return rc;
  if (n_sink < 0 || n_recent < 0) return SKV_ERR_INVALID;
  if (n_layer == 0 || n_req == 0) return SKV_OK;
  if (!aligned(kv_len, 4) || !aligned(keep, 4) || (evicted && !aligned(evicted, 4))) return SKV_ERR_INVALID;
  // tokens are read four at a time, moves written as pairs
  if (!aligned(score, 16) || !aligned(pos, 16) || !aligned(move, 16) || !aligned(n_move, 4)) return SKV_ERR_INVALID;
  const size_t pool = n_layer * pool_words(cache), req = (size_t)n_req;
  const Range used[] = {{score, pool}, {pos, pool}, {kv_len, req}, {keep, req}, {evicted, evicted ? req : 0},
                        {cache->block_table, req * (size_t)cache->max_block}, {move, pool},
                        {n_move, n_layer * req * cache->n_kv_head}, {cache->status, 1}};
  if (!apart(used, 6)) return SKV_ERR_INVALID;
  if ((rc = skv::check_device())) return rc;
  skv::EvictArgs a = evict_args(cache, n_layer, n_req, kv_len);
  a.keep = keep;
  a.evicted = evicted;
  a.n_sink = n_sink;
  a.n_recent = n_recent;
  a.score = const_cast<float*>(score);
  a.pos = const_cast<int32_t*>(pos);
  a.move = move;
  a.n_move = n_move;
  return launched(skv::launch_evict_plan(a, (cudaStream_t)stream));
}

int kv_evict_move(const skv_paged* cache, int32_t n_layer, int32_t n_req, const int32_t* kv_len,
                  const int32_t* move, const int32_t* n_move, float* score, int32_t* pos, void* stream) {
  int rc = check_layers(cache, n_layer, n_req);
  if (rc) return rc;
  if ((rc = check_pages(cache))) return rc;
  if (n_layer == 0 || n_req == 0) return SKV_OK;
  if (!aligned(kv_len, 4) || !aligned(move, 16) || !aligned(n_move, 4) || !aligned(score, 16) || !aligned(pos, 16))
    return SKV_ERR_INVALID;
  const size_t pool = n_layer * pool_words(cache), req = (size_t)n_req, rows = pool * cache->head_dim / 2;
  const Range used[] = {{kv_len, req}, {move, pool}, {n_move, n_layer * req * cache->n_kv_head},
                        {cache->block_table, req * (size_t)cache->max_block}, {cache->k, rows}, {cache->v, rows},
                        {score, pool}, {pos, pool}, {cache->status, 1}};
  if (!apart(used, 4)) return SKV_ERR_INVALID;
  if ((rc = skv::check_device())) return rc;
  skv::EvictArgs a = evict_args(cache, n_layer, n_req, kv_len);
  a.move = const_cast<int32_t*>(move);
  a.n_move = const_cast<int32_t*>(n_move);
  a.score = score;
  a.pos = pos;
  a.k = (uint16_t*)cache->k;
  a.v = (uint16_t*)cache->v;
  return launched(skv::launch_evict_move(a, cache->head_dim, (cudaStream_t)stream));
}

}  // extern "C"
