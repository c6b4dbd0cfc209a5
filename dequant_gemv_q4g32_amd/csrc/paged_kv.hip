// Paged KV cache, gfx950: append and gather of token rows, and the page operations (copy, fork,
// free, compact). The attention that reads the pages is in paged_attn.hip.
//
// Every kernel here moves bytes and is bound by HBM, or by a launch's latency when there is
// little to move. A lane handles 16 bytes of a page, or 8 elements of a row (one 16-byte fp16
// access, one 8-byte code access), as in the dense codec (kvcache.hip).
#include <hip/hip_runtime.h>

#include "../../include/qgemv.h"
#include "device_common.h"
#include "kv_codec.h"
#include "kv_pages.h"
#include "kv_rows.h"
#include "launch.h"

namespace qg {

constexpr int kPageThreads = 256;

// ---- append and gather ---------------------------------------------------------------------

// A lane takes 8 elements of K and the same 8 of V: both share the look-up of the place, and are on
// their way while it runs. 2048 int8 rows of 8 heads of 128: 5.7 us; a decode step's 64 rows: 3.3 us,
// a launch and the look-up's latency.
template <bool Q8>
__global__ __launch_bounds__(kPageThreads) void kv_append_kernel(RowsArgs a) {
  const uint32_t i = blockIdx.x * kPageThreads + threadIdx.x;
  const bool live = i < a.lanes;
  const uint32_t row = live ? i / a.per_row : 0, c = live ? i - row * a.per_row : 0;
  u32x4 v[2] = {u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}};
#pragma unroll
  for (int w = 0; w < 2; ++w)
    if (live) v[w] = *reinterpret_cast<const u32x4 *>(a.x[w] + (int64_t)row * a.ldx[w] + 8 * c);
  const RowPlace<Q8> p = row_place<Q8>(a, row, c);
  uint16_t d[2];
  u32x2 codes[2];
  if constexpr (Q8) {
#pragma unroll
    for (int w = 0; w < 2; ++w) codes[w] = kv_encode8(v[w], d[w]);   // every lane: the quad's maximum needs all four
  }
  if (!live || !p.part) return;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if constexpr (Q8) {
      *reinterpret_cast<u32x2 *>(p.part + p.off[w]) = codes[w];
      if ((c & 3) == 0) *reinterpret_cast<uint16_t *>(p.part + p.scale_off[w]) = d[w];
    } else {
      *reinterpret_cast<u32x4 *>(p.part + p.off[w]) = v[w];
    }
  }
}

// The way back. 8192 int8 rows of 8 heads of 128 (51 MB read and written) take 12.2 us: a launch
// and the three dependent loads before the data's own, then the data at the streaming rate. Two
// rows a lane gained 5% there and lost 25% of a decode step's 64 rows (2.7 us).
template <bool Q8>
__global__ __launch_bounds__(kPageThreads) void kv_gather_kernel(RowsArgs a) {
  const uint32_t i = blockIdx.x * kPageThreads + threadIdx.x;
  if (i >= a.lanes) return;
  const uint32_t row = i / a.per_row, c = i - row * a.per_row;
  const RowPlace<Q8> p = row_place<Q8>(a, row, c);
  u32x4 v[2] = {u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}};
  if (p.part) {
    if constexpr (Q8) {
      u32x2 codes[2];
      uint16_t d[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        codes[w] = *reinterpret_cast<const u32x2 *>(p.part + p.off[w]);
        d[w] = *reinterpret_cast<const uint16_t *>(p.part + p.scale_off[w]);
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) v[w] = kv_decode8(codes[w], half_bits(d[w]));
    } else {
#pragma unroll
      for (int w = 0; w < 2; ++w) v[w] = *reinterpret_cast<const u32x4 *>(p.part + p.off[w]);
    }
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) *reinterpret_cast<u32x4 *>(a.x[w] + (int64_t)row * a.ldx[w] + 8 * c) = v[w];
}

// ---- page copies ----------------------------------------------------------------------------

struct PoolArgs {
  uint8_t *pages;
  int64_t layer_stride, page_bytes;
  int32_t layers, num_pages;
  int32_t chunks;                // copies of a page are split into chunks of kChunk bytes
};

constexpr int64_t kChunk = 16384;                  // 4 loads of 16 bytes in flight a lane

// One workgroup copies chunk `c` of a page, past the caches (every byte is touched once): 268 MB
// copied in 100 us = 5.4 TB/s read and written, cached loads and stores 107 us; chunks of 8 KB the
// same, of 32 KB 133 us.
__device__ __forceinline__ void copy_chunk(const PoolArgs &p, int32_t layer, int32_t src, int32_t dst, int32_t c) {
  const int64_t base = (int64_t)layer * p.layer_stride;
  const int64_t first = (int64_t)c * kChunk;
  const uint8_t *s = p.pages + base + (int64_t)src * p.page_bytes + first;
  uint8_t *d = p.pages + base + (int64_t)dst * p.page_bytes + first;
  const int32_t n = (int32_t)(p.page_bytes - first < kChunk ? p.page_bytes - first : kChunk);   // a multiple of 128
  u32x4 v[4];
  constexpr int kStep = 16 * kPageThreads;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int32_t o = u * kStep + 16 * (int)threadIdx.x;
    if (o < n) v[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(s + o));
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int32_t o = u * kStep + 16 * (int)threadIdx.x;
    if (o < n) __builtin_nontemporal_store(v[u], reinterpret_cast<u32x4 *>(d + o));
  }
}

// Grid (pairs, chunks, layers).
__global__ __launch_bounds__(kPageThreads) void kv_copy_kernel(PoolArgs p, const int32_t *src, const int32_t *dst) {
  const int32_t s = src[blockIdx.x], d = dst[blockIdx.x];
  if (s < 0 || d < 0 || s >= p.num_pages || d >= p.num_pages || s == d) return;
  copy_chunk(p, blockIdx.z, s, d, blockIdx.y);
}

// ---- fork and free -----------------------------------------------------------------------------

struct TableArgs {
  int32_t *table;
  int64_t ld;
  int32_t rows, pages;
  int32_t tok_shift;
  int32_t *lens, *refs;
};

__device__ __forceinline__ int32_t row_len(const TableArgs &t, int32_t row) {
  const int64_t n = t.lens[row], most = (int64_t)t.pages << t.tok_shift;
  return (int32_t)(n < 0 ? 0 : n < most ? n : most);
}

// Grid (forks, chunks + 1, layers): blockIdx.y == 0 of layer 0 writes the table row, the others
// copy a chunk of the last page. No workgroup reads what another writes: a destination row that
// is also a source row or an earlier destination, or a new page named before, drops the fork,
// and source rows are never written.
__global__ __launch_bounds__(kPageThreads) void kv_fork_kernel(PoolArgs p, TableArgs t, const int32_t *src_rows,
                                                              const int32_t *dst_rows, const int32_t *new_pages,
                                                              int32_t count) {
  const bool table_part = blockIdx.y == 0;
  if (table_part && blockIdx.z != 0) return;
  const int32_t i = blockIdx.x;
  const int32_t s = src_rows[i], d = dst_rows[i];
  if (s < 0 || d < 0 || s >= t.rows || d >= t.rows) return;
  const int32_t n = row_len(t, s);
  const int32_t whole = n >> t.tok_shift;
  const bool rest = (n & ((1 << t.tok_shift) - 1)) != 0;
  const int32_t *from = t.table + (int64_t)s * t.ld;
  // a partly filled last page is copied; where the source's entry is no page, so is the new row's
  const int32_t tail = rest ? from[whole] : -1;
  const bool copy = tail >= 0 && tail < p.num_pages;
  if (!copy && !table_part) return;
  const int32_t fresh = new_pages[i];
  bool drop = copy && (fresh < 0 || fresh >= p.num_pages);
  for (int32_t k = threadIdx.x; k < count; k += kPageThreads)
    drop |= src_rows[k] == d || (k < i && (dst_rows[k] == d || (copy && new_pages[k] == fresh)));
  if (__syncthreads_or(drop)) return;
  if (!table_part) {
    if (tail != fresh) copy_chunk(p, blockIdx.z, tail, fresh, blockIdx.y - 1);
    return;
  }
  const int32_t taken = whole + (rest && !copy ? 1 : 0);    // entries that are the source's own
  int32_t *to = t.table + (int64_t)d * t.ld;
  for (int32_t j = threadIdx.x; j < t.pages; j += kPageThreads) {
    int32_t e = -1;
    if (j < taken) {
      e = from[j];
      if (e >= 0 && e < p.num_pages) atomicAdd(t.refs + e, 1);
    } else if (j == whole && copy) {
      e = fresh;
    }
    to[j] = e;
  }
  if (threadIdx.x == 0) {
    t.lens[d] = n;
    if (copy) t.refs[fresh] = 1;
  }
}

// Grid (rows). The workgroup that takes the row's length out of lens gives up its pages, so a
// row named twice is released once.
__global__ __launch_bounds__(kPageThreads) void kv_free_kernel(TableArgs t, int32_t num_pages, const int32_t *rows) {
  __shared__ int32_t taken;
  const int32_t r = rows[blockIdx.x];
  if (r < 0 || r >= t.rows) return;
  if (threadIdx.x == 0) taken = t.lens[r] > 0 ? atomicExch(t.lens + r, 0) : 0;
  __syncthreads();
  if (taken <= 0) return;
  const int32_t pages = (int32_t)(((int64_t)taken + (1 << t.tok_shift) - 1) >> t.tok_shift);
  int32_t *row = t.table + (int64_t)r * t.ld;
  for (int32_t j = threadIdx.x; j < t.pages; j += kPageThreads) {
    const int32_t e = row[j];
    if (j < pages && e >= 0 && e < num_pages) atomicSub(t.refs + e, 1);
    row[j] = -1;
  }
}

// ---- compaction ----------------------------------------------------------------------------------
//
// With lp(p) the number of held pages before p and L = lp(num_pages), a held page p >= L is the
// (lp(p) - lp(L))-th that moves, and a free page p < L the (p - lp(p))-th that receives one; there
// are as many of the one as of the other. Three launches: counts of held pages by block (left out
// for small pools, where every workgroup of the second counts for itself); the ranks, as lists of
// sources and destinations; the copies, with the table and the counts.

constexpr int kScanPages = 4 * kPageThreads;       // pages a workgroup of the first two launches covers

struct CompactArgs {
  const int32_t *refs;
  int32_t *refs_out, *remap, *live;
  int32_t *blocks;                                   // held pages of each block
  int32_t *src, *dst, *moves;                        // lists of up to num_pages / 2 pages, and their length
  int32_t num_pages, num_blocks;
  int32_t direct;                                    // the second launch counts for itself
};

// Sum over the workgroup, in every thread; red: 4 ints of LDS.
__device__ __forceinline__ int32_t block_sum(int32_t v, int32_t *red) {
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

__global__ __launch_bounds__(kPageThreads) void kv_count_kernel(CompactArgs c) {
  __shared__ int32_t red[4];
  int32_t held = 0;
  for (int u = 0; u < 4; ++u) {
    const int64_t p = (int64_t)blockIdx.x * kScanPages + u * kPageThreads + threadIdx.x;
    if (p < c.num_pages) held += c.refs[p] > 0;
  }
  held = block_sum(held, red);
  if (threadIdx.x == 0) c.blocks[blockIdx.x] = held;
}

__global__ __launch_bounds__(kPageThreads) void kv_rank_kernel(CompactArgs c) {
  __shared__ int32_t red[4];
  __shared__ int32_t waves[4];
  const int32_t b = blockIdx.x;
  // held pages in all blocks, and in the blocks before this one
  int32_t all = 0, before = 0;
  if (c.direct) {
    for (int32_t p = threadIdx.x; p < c.num_pages; p += kPageThreads) {
      const int32_t held = c.refs[p] > 0;
      all += held;
      before += p < b * kScanPages ? held : 0;
    }
  } else {
    for (int32_t k = threadIdx.x; k < c.num_blocks; k += kPageThreads) {
      const int32_t n = c.blocks[k];
      all += n;
      before += k < b ? n : 0;
    }
  }
  const int32_t live = block_sum(all, red);
  before = block_sum(before, red);
  // held pages before page `live`: whole blocks, and the part of its own block
  const int32_t lb = c.direct ? 0 : live / kScanPages;
  int32_t low = 0;
  for (int32_t k = threadIdx.x; k < lb; k += kPageThreads) low += c.blocks[k];
  for (int32_t p = lb * kScanPages + threadIdx.x; p < live; p += kPageThreads) low += c.refs[p] > 0;
  low = block_sum(low, red);
  if (b == 0 && threadIdx.x == 0) {
    *c.live = live;
    *c.moves = live - low;
  }
  // this block's pages, four neighbours a thread
  const int64_t p0 = (int64_t)b * kScanPages + 4 * (int)threadIdx.x;
  int32_t r[4], mine = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    r[u] = p0 + u < c.num_pages ? c.refs[p0 + u] : 0;
    mine += r[u] > 0;
  }
  int32_t scan = mine;
  for (int o = 1; o < 64; o <<= 1) {
    const int32_t up = __shfl_up(scan, o);
    scan += (int)(threadIdx.x & 63) >= o ? up : 0;
  }
  if ((threadIdx.x & 63) == 63) waves[threadIdx.x >> 6] = scan;
  __syncthreads();
  int32_t lp = before + scan - mine;
  for (int w = 0; w < (int)(threadIdx.x >> 6); ++w) lp += waves[w];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t p = p0 + u;
    if (p >= c.num_pages) break;
    const bool held = r[u] > 0;
    if (held && p >= live) {
      const int32_t rank = lp - low;
      c.src[rank] = (int32_t)p;
      c.remap[p] = -2 - rank;                       // replaced by dst[rank] in the last launch
    } else {
      if (!held && p < live) c.dst[p - lp] = (int32_t)p;
      c.remap[p] = held ? (int32_t)p : -1;
      if (held || p >= live) c.refs_out[p] = held ? r[u] : 0;   // the others: with the move
    }
    lp += held;
  }
}

// Workgroups below table_groups replace the table's entries, the others share the copies.
__global__ __launch_bounds__(kPageThreads) void kv_move_kernel(PoolArgs p, CompactArgs c, const int32_t *table, int64_t ld,
                                                              int32_t *table_out, int64_t ld_out, int64_t entries,
                                                              int32_t per_row, int32_t table_groups) {
  if ((int32_t)blockIdx.x < table_groups) {
    for (int64_t i = (int64_t)blockIdx.x * kPageThreads + threadIdx.x; i < entries;
         i += (int64_t)table_groups * kPageThreads) {
      const int64_t r = i / per_row, j = i - r * per_row;
      int32_t e = table[r * ld + j];
      if (e >= 0 && e < p.num_pages) {
        // the rank of a moved page, or its new index if a copying workgroup came first
        e = __hip_atomic_load(c.remap + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (e <= -2) e = c.dst[-2 - e];
      } else {
        e = -1;
      }
      table_out[r * ld_out + j] = e;
    }
    return;
  }
  const int32_t moves = *c.moves;
  const int64_t items = (int64_t)moves * p.layers * p.chunks;
  const int64_t per_move = (int64_t)p.layers * p.chunks;
  for (int64_t it = (int64_t)blockIdx.x - table_groups; it < items; it += (int64_t)gridDim.x - table_groups) {
    const int32_t m = (int32_t)(it / per_move), rest = (int32_t)(it - m * per_move);
    const int32_t layer = rest / p.chunks, chunk = rest - layer * p.chunks;
    const int32_t src = c.src[m], dst = c.dst[m];
    copy_chunk(p, layer, src, dst, chunk);
    if (rest == 0 && threadIdx.x == 0) {
      const int32_t n = c.refs[src];
      c.refs_out[dst] = n;
      c.refs_out[src] = 0;
      __hip_atomic_store(c.remap + src, dst, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
}

namespace {

bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int log2_of(int64_t v) {
  int s = 0;
  while ((int64_t(1) << s) < v) ++s;
  return s;
}

PoolArgs pool_args(const qg_kv_pool *pool, const KvLayout &L) {
  PoolArgs p;
  p.pages = static_cast<uint8_t *>(pool->pages);
  p.layer_stride = pool->layers > 1 ? pool->layer_stride : 0;
  p.page_bytes = L.page_bytes;
  p.layers = (int32_t)pool->layers;
  p.num_pages = (int32_t)pool->num_pages;
  p.chunks = (int32_t)((L.page_bytes + kChunk - 1) / kChunk);
  return p;
}

int kv_rows(bool append, const qg_kv_pool *pool, int64_t layer, const int32_t *table, int64_t ld_table, int64_t table_rows,
            int64_t table_pages, uint16_t *k, int64_t ldk, uint16_t *v, int64_t ldv, const int32_t *seqs,
            const int32_t *positions, int64_t count, void *stream) {
  KvLayout L;
  if (int st = kv_pool_layout(pool, &L)) return st;
  if (int st = kv_table_check(table, ld_table, table_rows, table_pages)) return st;
  if (layer < 0 || layer >= pool->layers || count < 0) return QG_ERR_SHAPE;
  const int64_t cols = (int64_t)pool->kv_heads * pool->head_dim, per_row = cols / 8;
  if (count > 0x7FFFFFFF / per_row || (count > 1 && (ldk < cols || ldv < cols))) return QG_ERR_SHAPE;
  if (count == 0) return QG_OK;
  if (!k || !v || !positions) return QG_ERR_NULL;
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(seqs, 4) || misaligned(positions, 4) ||
      (count > 1 && (ldk % 8 || ldv % 8)))
    return QG_ERR_ALIGN;
  RowsArgs a;
  a.pool = static_cast<uint8_t *>(pool->pages) + (layer ? layer * pool->layer_stride : 0);
  a.page_bytes = L.page_bytes;
  a.head_bytes = L.head_bytes;
  a.v_off = L.v_off;
  a.ks_off = L.ks_off;
  a.vs_off = L.vs_off;
  a.num_pages = (int32_t)pool->num_pages;
  a.table = table;
  a.ld_table = ld_table;
  a.table_rows = (int32_t)table_rows;
  a.table_pages = (int32_t)table_pages;
  a.x[0] = k;
  a.x[1] = v;
  a.ldx[0] = count > 1 ? ldk : cols;
  a.ldx[1] = count > 1 ? ldv : cols;
  a.seqs = seqs;
  a.positions = positions;
  a.lanes = (uint32_t)(count * per_row);
  a.per_row = (uint32_t)per_row;
  a.lane_shift = log2_of(pool->head_dim / 8);
  a.tok_shift = log2_of(pool->page_tokens);
  const bool q8 = pool->kind == QG_KV_Q8;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 block(kPageThreads), grid((a.lanes + kPageThreads - 1) / kPageThreads);
  if (append)
    return q8 ? launch(kv_append_kernel<true>, grid, block, 0, s, a) : launch(kv_append_kernel<false>, grid, block, 0, s, a);
  return q8 ? launch(kv_gather_kernel<true>, grid, block, 0, s, a) : launch(kv_gather_kernel<false>, grid, block, 0, s, a);
}

// Workspace of a compaction: block counts, the two lists and their length.
int64_t compact_ints(int64_t num_pages) { return (num_pages + kScanPages - 1) / kScanPages + 2 * (num_pages / 2 + 1) + 1; }

constexpr int64_t kCompactPages = int64_t(1) << 24;
constexpr int64_t kDirectPages = 4096;          // 301 pages: 8.6 us in three launches, 7.0 in two
constexpr int64_t kMaxForks = 4096;                  // every workgroup of a fork looks through all of them
constexpr int64_t kMaxCount = int64_t(1) << 23;     // workgroups of 256 threads in a grid's x axis

}  // namespace

}  // namespace qg

using namespace qg;

extern "C" {

int qg_kv_append(const qg_kv_pool *pool, int64_t layer, const int32_t *table, int64_t ld_table, int64_t table_rows,
                 int64_t table_pages, const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv, const int32_t *seqs,
                 const int32_t *positions, int64_t count, void *stream) {
  return kv_rows(true, pool, layer, table, ld_table, table_rows, table_pages, const_cast<uint16_t *>(k), ldk,
                 const_cast<uint16_t *>(v), ldv, seqs, positions, count, stream);
}

int qg_kv_gather(const qg_kv_pool *pool, int64_t layer, const int32_t *table, int64_t ld_table, int64_t table_rows,
                 int64_t table_pages, uint16_t *k, int64_t ldk, uint16_t *v, int64_t ldv, const int32_t *seqs,
                 const int32_t *positions, int64_t count, void *stream) {
  return kv_rows(false, pool, layer, table, ld_table, table_rows, table_pages, k, ldk, v, ldv, seqs, positions, count,
                 stream);
}

int qg_kv_copy_pages(const qg_kv_pool *pool, const int32_t *src, const int32_t *dst, int64_t count, void *stream) {
  KvLayout L;
  if (int st = kv_pool_layout(pool, &L)) return st;
  if (count < 0 || count > kMaxCount) return QG_ERR_SHAPE;
  if (count == 0) return QG_OK;
  if (!src || !dst) return QG_ERR_NULL;
  if (misaligned(src, 4) || misaligned(dst, 4)) return QG_ERR_ALIGN;
  const PoolArgs p = pool_args(pool, L);
  return launch(kv_copy_kernel, dim3((unsigned)count, (unsigned)p.chunks, (unsigned)p.layers), dim3(kPageThreads), 0,
                static_cast<hipStream_t>(stream), p, src, dst);
}

int qg_kv_fork(const qg_kv_pool *pool, int32_t *table, int64_t ld_table, int64_t table_rows, int64_t table_pages,
               int32_t *lens, int32_t *refs, const int32_t *src_rows, const int32_t *dst_rows, const int32_t *new_pages,
               int64_t count, void *stream) {
  KvLayout L;
  if (int st = kv_pool_layout(pool, &L)) return st;
  if (int st = kv_table_check(table, ld_table, table_rows, table_pages)) return st;
  if (count < 0 || count > kMaxForks) return QG_ERR_SHAPE;
  if (count == 0 || table_rows == 0) return QG_OK;
  if (!lens || !refs || !src_rows || !dst_rows || !new_pages) return QG_ERR_NULL;
  if (misaligned(lens, 4) || misaligned(refs, 4) || misaligned(src_rows, 4) || misaligned(dst_rows, 4) ||
      misaligned(new_pages, 4))
    return QG_ERR_ALIGN;
  const PoolArgs p = pool_args(pool, L);
  const TableArgs t{table, ld_table, (int32_t)table_rows, (int32_t)table_pages, log2_of(pool->page_tokens), lens, refs};
  return launch(kv_fork_kernel, dim3((unsigned)count, (unsigned)p.chunks + 1, (unsigned)p.layers), dim3(kPageThreads), 0,
                static_cast<hipStream_t>(stream), p, t, src_rows, dst_rows, new_pages, (int32_t)count);
}

int qg_kv_free(const qg_kv_pool *pool, int32_t *table, int64_t ld_table, int64_t table_rows, int64_t table_pages,
               int32_t *lens, int32_t *refs, const int32_t *rows, int64_t count, void *stream) {
  KvLayout L;
  if (int st = kv_pool_layout(pool, &L)) return st;
  if (int st = kv_table_check(table, ld_table, table_rows, table_pages)) return st;
  if (count < 0 || count > kMaxCount) return QG_ERR_SHAPE;
  if (count == 0 || table_rows == 0) return QG_OK;
  if (!lens || !refs || !rows) return QG_ERR_NULL;
  if (misaligned(lens, 4) || misaligned(refs, 4) || misaligned(rows, 4)) return QG_ERR_ALIGN;
  const TableArgs t{table, ld_table, (int32_t)table_rows, (int32_t)table_pages, log2_of(pool->page_tokens), lens, refs};
  return launch(kv_free_kernel, dim3((unsigned)count), dim3(kPageThreads), 0, static_cast<hipStream_t>(stream), t,
                (int32_t)pool->num_pages, rows);
}

int qg_kv_compact_bytes(const qg_kv_pool *pool, int64_t *bytes) {
  if (!bytes) return QG_ERR_NULL;
  KvLayout L;
  if (int st = kv_pool_layout(pool, &L)) return st;
  if (pool->num_pages > kCompactPages) return QG_ERR_SHAPE;
  *bytes = 4 * compact_ints(pool->num_pages);
  return QG_OK;
}

int qg_kv_compact(const qg_kv_pool *pool, const int32_t *table, int64_t ld_table, int32_t *table_out, int64_t ld_out,
                  int64_t table_rows, int64_t table_pages, const int32_t *refs, int32_t *refs_out, int32_t *remap,
                  int32_t *live, void *workspace, int64_t workspace_bytes, void *stream) {
  KvLayout L;
  if (int st = kv_pool_layout(pool, &L)) return st;
  if (int st = kv_table_check(table, ld_table, table_rows, table_pages)) return st;
  if (int st = kv_table_check(table_out, ld_out, table_rows, table_pages)) return st;
  if (pool->num_pages > kCompactPages) return QG_ERR_SHAPE;
  if (!refs || !refs_out || !remap || !live || !workspace) return QG_ERR_NULL;
  if (misaligned(refs, 4) || misaligned(refs_out, 4) || misaligned(remap, 4) || misaligned(live, 4) ||
      misaligned(workspace, 4))
    return QG_ERR_ALIGN;
  const int64_t n = pool->num_pages;
  if (workspace_bytes < 4 * compact_ints(n)) return QG_ERR_WORKSPACE;
  const PoolArgs p = pool_args(pool, L);
  CompactArgs c;
  c.refs = refs;
  c.refs_out = refs_out;
  c.remap = remap;
  c.live = live;
  c.num_pages = (int32_t)n;
  c.num_blocks = (int32_t)((n + kScanPages - 1) / kScanPages);
  c.blocks = static_cast<int32_t *>(workspace);
  c.src = c.blocks + c.num_blocks;
  c.dst = c.src + n / 2 + 1;
  c.moves = c.dst + n / 2 + 1;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 block(kPageThreads);
  c.direct = n <= kDirectPages;
  if (!c.direct)
    if (int st = launch(kv_count_kernel, dim3(c.num_blocks), block, 0, s, c)) return st;
  if (int st = launch(kv_rank_kernel, dim3(c.num_blocks), block, 0, s, c)) return st;
  const int64_t entries = table_rows * table_pages;
  const int64_t groups = (entries + 4 * kPageThreads - 1) / (4 * kPageThreads);
  const int32_t table_groups = (int32_t)(groups < 256 ? groups : 256);
  const int64_t most = n / 2 * p.layers * p.chunks;
  const int64_t copies = most < 2048 ? most : 2048;
  if (table_groups + copies == 0) return QG_OK;
  return launch(kv_move_kernel, dim3((unsigned)(table_groups + copies)), block, 0, s, p, c, table, ld_table, table_out, ld_out,
                entries, (int32_t)(table_pages > 0 ? table_pages : 1), table_groups);
}

}  // extern "C"
