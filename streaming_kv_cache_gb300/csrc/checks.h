// Argument checks that the entry points of the paged cache share.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "skv.h"

namespace skv {
namespace checks {

inline bool aligned(const void* p, unsigned n) { return p && ((uintptr_t)p & (n - 1)) == 0; }

// a token-major tensor of `heads` heads: its pointer and token stride
inline bool tensor_ok(const void* p, int64_t stride, int64_t heads, int d) {
  return aligned(p, 16) && stride >= heads * d && (stride & 7) == 0;
}

// n words of 32 bits
struct Range {
  const void* p;
  size_t n;
};
inline bool overlap(const Range& a, const Range& b) {
  const char *a0 = (const char*)a.p, *b0 = (const char*)b.p;
  return a.n && b.n && a0 < b0 + 4 * b.n && b0 < a0 + 4 * a.n;
}

// What every paged call needs of the pool; k, v and rope belong to some calls only.
inline int check_pool(const skv_paged* c) {
  if (!c) return SKV_ERR_INVALID;
  if (c->n_page < 1 || c->page_size < 16 || (c->page_size & 15) || c->max_block < 1) return SKV_ERR_INVALID;
  if ((long long)c->n_page * c->page_size > 0x7FFFFFFFLL) return SKV_ERR_INVALID;
  if (!aligned(c->block_table, 4) || !aligned(c->status, 4)) return SKV_ERR_INVALID;
  return SKV_OK;
}

inline int check_heads(int n_kv_head, int head_dim, int dtype) {
  if (n_kv_head < 1 || (head_dim != 64 && head_dim != 128)) return SKV_ERR_INVALID;
  if (dtype != SKV_BF16 && dtype != SKV_FP16) return SKV_ERR_INVALID;
  return SKV_OK;
}

inline int check_pages(const skv_paged* c) {
  int rc = check_pool(c);
  if (rc) return rc;
  if ((rc = check_heads(c->n_kv_head, c->head_dim, c->dtype))) return rc;
  if ((long long)c->n_page * c->n_kv_head > 0x7FFFFFFFLL) return SKV_ERR_INVALID;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return SKV_ERR_INVALID;
  return SKV_OK;
}

}  // namespace checks
}  // namespace skv
