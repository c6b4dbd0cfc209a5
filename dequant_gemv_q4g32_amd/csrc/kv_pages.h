// Layout of a paged key-value cache, shared by the host and the device sources.
//
// A pool is [layers][num_pages] page records. A page record holds page_tokens (T) consecutive
// tokens of one sequence for every KV head; the part of one head (D = head_dim) is contiguous:
//   QG_KV_Q8   K codes int8 [T][D], V codes int8 [T][D], K scales fp16 [T][D/32],
//              V scales fp16 [D/32][T]
//   QG_KV_F16  K fp16 [T][D], V fp16 [T][D]
// The codes and scales are those of qg_kv_quantize. Head parts are contiguous because a
// decode-attention wave reads one head of one sequence: T tokens of K, V and scales are then
// one run of memory. The two scale arrays follow how the matrix-core operands meet them: a
// lane holds one token of K (its D/32 scales are neighbours) but several consecutive tokens of
// one group of V (its tokens are neighbours).
#pragma once
#include <stdint.h>

#include "../../include/qgemv.h"

namespace qg {

struct KvLayout {
  int64_t head_bytes;    // one head's part of a page record
  int64_t page_bytes;    // kv_heads * head_bytes
  int32_t v_off;         // byte offsets within a head's part (K starts at 0)
  int32_t ks_off;
  int32_t vs_off;
};

inline int kv_layout(int kind, int64_t kv_heads, int64_t head_dim, int64_t page_tokens, KvLayout *out) {
  if (kind != QG_KV_Q8 && kind != QG_KV_F16) return QG_ERR_FORMAT;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return QG_ERR_SHAPE;
  if (page_tokens < 16 || page_tokens > 256 || (page_tokens & (page_tokens - 1))) return QG_ERR_SHAPE;
  if (kv_heads < 1 || kv_heads > 1024) return QG_ERR_SHAPE;
  const int64_t td = page_tokens * head_dim;
  if (kind == QG_KV_Q8) {
    out->v_off = (int32_t)td;
    out->ks_off = (int32_t)(2 * td);
    out->vs_off = (int32_t)(2 * td + td / 16);
    out->head_bytes = 2 * td + td / 8;
  } else {
    out->v_off = (int32_t)(2 * td);
    out->ks_off = out->vs_off = 0;
    out->head_bytes = 4 * td;
  }
  out->page_bytes = kv_heads * out->head_bytes;
  return QG_OK;
}

// Checks a pool's description and returns its layout.
inline int kv_pool_layout(const qg_kv_pool *pool, KvLayout *out) {
  if (!pool) return QG_ERR_NULL;
  if (int st = kv_layout(pool->kind, pool->kv_heads, pool->head_dim, pool->page_tokens, out)) return st;
  if (pool->num_pages < 1 || pool->num_pages > 0x7FFFFFFF || pool->layers < 1 || pool->layers > 65535) return QG_ERR_SHAPE;
  if (pool->layers > 1 && pool->layer_stride < pool->num_pages * out->page_bytes) return QG_ERR_SHAPE;
  if (!pool->pages) return QG_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(pool->pages) & 15) || (pool->layers > 1 && (pool->layer_stride & 15))) return QG_ERR_ALIGN;
  return QG_OK;
}

// Checks a page table of `rows` sequences of up to `pages` pages.
inline int kv_table_check(const int32_t *table, int64_t ld, int64_t rows, int64_t pages) {
  if (rows < 0 || rows > 0x7FFFFFFF || pages < 0 || pages > 0x7FFFFFFF || (rows > 1 && ld < pages)) return QG_ERR_SHAPE;
  if (rows > 0 && pages > 0 && !table) return QG_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(table) & 3) return QG_ERR_ALIGN;
  return QG_OK;
}

}  // namespace qg
