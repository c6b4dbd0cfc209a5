// Where the rows of a paged-cache call lie (paged_kv.hip and rope.hip): a token's page by the table, and 8
// consecutive elements of its K and V in that page.
#pragma once
#include <hip/hip_runtime.h>

#include "kv_codec.h"

namespace qg {

struct RowsArgs {
  uint8_t *pool;                 // the layer's first page
  int64_t page_bytes, head_bytes;
  int32_t v_off, ks_off, vs_off;
  int32_t num_pages;
  const int32_t *table;
  int64_t ld_table;
  int32_t table_rows, table_pages;
  uint16_t *x[2];                // K and V rows
  int64_t ldx[2];
  const int32_t *seqs, *positions;
  uint32_t lanes, per_row;       // count * per_row lanes, per_row = kv_heads * head_dim / 8
  int32_t lane_shift, tok_shift; // log2 of head_dim / 8 and of page_tokens
};

// The place of one row's token: the page's first byte and the place in the page, or nullptr.
__device__ __forceinline__ uint8_t *row_page(const RowsArgs &a, uint32_t row, int32_t &at) {
  const int32_t s = a.seqs ? a.seqs[row] : (int32_t)row;
  const int32_t pos = a.positions[row];
  at = pos & ((1 << a.tok_shift) - 1);
  const int32_t slot = pos >> a.tok_shift;
  if (s < 0 || s >= a.table_rows || pos < 0 || slot >= a.table_pages) return nullptr;
  const int32_t page = a.table[(int64_t)s * a.ld_table + slot];
  if (page < 0 || page >= a.num_pages) return nullptr;
  return a.pool + (int64_t)page * a.page_bytes;
}

// Where 8 elements of a row lie in its page: the lane's elements are in one head and one group of
// 32, and the 4 lanes of a group are neighbours in a wave (head_dim / 8 lanes a head, a multiple of 4).
template <bool Q8>
struct RowPlace {
  uint8_t *part;                 // the head's part of the page; nullptr: no place
  int64_t off[2], scale_off[2];  // of K and V
};
template <bool Q8>
__device__ __forceinline__ RowPlace<Q8> place_in(const RowsArgs &a, uint8_t *page, int32_t at, uint32_t c) {
  RowPlace<Q8> p;
  const uint32_t head = c >> a.lane_shift, e = 8 * (c & ((1u << a.lane_shift) - 1));   // element within the head
  const int32_t dim = 8 << a.lane_shift, group = e / kKvGroup;
  const int64_t elem = (int64_t)at * dim + e;
  p.part = page ? page + (int64_t)head * a.head_bytes : nullptr;
  p.off[0] = Q8 ? elem : 2 * elem;
  p.off[1] = a.v_off + p.off[0];
  p.scale_off[0] = a.ks_off + 2 * ((int64_t)at * (dim / kKvGroup) + group);
  p.scale_off[1] = a.vs_off + 2 * (((int64_t)group << a.tok_shift) + at);
  return p;
}
template <bool Q8>
__device__ __forceinline__ RowPlace<Q8> row_place(const RowsArgs &a, uint32_t row, uint32_t c) {
  int32_t at;
  uint8_t *page = row_page(a, row, at);
  return place_in<Q8>(a, page, at, c);
}

}  // namespace qg
