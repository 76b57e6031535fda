// What the operators of the paged 8-bit cache share: the checks of its description, and where a
// packed row or a block of positions belongs.
#pragma once

#include <cmath>

#include "qd_internal.cuh"

namespace qd {
namespace paged {

struct Cache {
  uint8_t *k, *v;
  float *ks, *vs;
  const int32_t* table;
  int n_pages, page_tokens, per_page;  // per_page: blocks
  uint32_t per_magic;                  // 2^32 / per_page rounded up (0 for one block)
  int n_kv, max_pages, capacity;       // capacity: positions of a sequence
};

inline Cache cache_of(const qd_paged_kv* kv) {
  Cache c;
  c.k = static_cast<uint8_t*>(kv->k_pages);
  c.v = static_cast<uint8_t*>(kv->v_pages);
  c.ks = kv->k_scale;
  c.vs = kv->v_scale;
  c.table = kv->page_table;
  c.n_pages = kv->n_pages;
  c.page_tokens = kv->page_tokens;
  c.per_page = kv->page_tokens / QD_KV_BLOCK;
  c.per_magic = c.per_page == 1 ? 0u : (uint32_t)(((1ull << 32) + c.per_page - 1) / c.per_page);
  c.n_kv = kv->n_kv_heads;
  c.max_pages = kv->max_pages;
  c.capacity = kv->max_pages * kv->page_tokens;
  return c;
}

// QD_OK, or what is wrong with the description itself.
inline qd_status cache_status(const qd_paged_kv* kv, int n_seqs) {
  if (!kv) return QD_ERR_INVALID_ARG;
  if (!kv->k_pages || !kv->v_pages || !kv->k_scale || !kv->v_scale || !kv->page_table) return QD_ERR_INVALID_ARG;
  if (kv->fmt != QD_KV_I8 && kv->fmt != QD_KV_E4M3) return QD_ERR_UNSUPPORTED;
  if (kv->head_dim != 64 && kv->head_dim != 128) return QD_ERR_UNSUPPORTED;
  if (kv->n_pages < 1 || kv->page_tokens < QD_KV_BLOCK || kv->page_tokens > 1024 || kv->page_tokens % QD_KV_BLOCK ||
      kv->n_kv_heads < 1 || kv->n_kv_heads > 4096 || kv->max_pages < 1 || kv->max_seqs < 1 ||
      kv->max_seqs > QD_MAX_SEQS || (int64_t)kv->max_pages * kv->page_tokens > (1ll << 30) ||
      (int64_t)kv->n_pages * kv->n_kv_heads > ((1ll << 31) - 1) / (kv->page_tokens / QD_KV_BLOCK) || n_seqs < 1 ||
      n_seqs > kv->max_seqs)
    return QD_ERR_SHAPE;
  if (!aligned16(kv->k_pages) || !aligned16(kv->v_pages) || !aligned4(kv->k_scale) || !aligned4(kv->v_scale) ||
      !aligned4(kv->page_table))
    return QD_ERR_ALIGN;
  return QD_OK;
}

// The page of a block (of QD_KV_BLOCK positions) in a sequence's row of the table, -1 if there is
// none, and the block's place in it.  block / per_page by a multiplication: with at most 2^26 blocks and
// 64 to a page, block (ceil(2^32 / per) / 2^32 - 1 / per) < 2^-6 <= 1 / per, so the floor is the quotient.
__device__ __forceinline__ int page_of(const Cache& c, const int32_t* row, int block, int& in_page) {
  const int at = c.per_magic ? (int)__umulhi((uint32_t)block, c.per_magic) : block;
  in_page = block - at * c.per_page;
  const int page = __ldg(row + at);
  return (unsigned)page < (unsigned)c.n_pages ? page : -1;
}
__device__ __forceinline__ const int32_t* table_row(const Cache& c, int b) { return c.table + (int64_t)b * c.max_pages; }
// Scale index of (page, head, block in the page); times 16 * head_dim: its first code.
__device__ __forceinline__ int64_t block_index(const Cache& c, int page, int head, int in_page) {
  return ((int64_t)page * c.n_kv + head) * c.per_page + in_page;
}

// Rows of sequence b, whatever row_start holds: [first, first + count) within [0, n_tokens).
__device__ __forceinline__ int rows_of(const int32_t* row_start, int b, int n_tokens, int& first) {
  first = min(max(row_start[b], 0), n_tokens);
  return max(min(max(row_start[b + 1], 0), n_tokens) - first, 0);
}

}  // namespace paged
}  // namespace qd
