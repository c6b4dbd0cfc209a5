// Places for a step's tokens, gfx950: page tables grow (extend) and shrink (trim) by lengths that lie
// on the device, and the slot maps that append takes come with them.
//
// Little is moved here; every launch is a chain of dependent loads (lengths, the last page's entry and
// its count, the counts of all pages) and prefix sums. extend reads refs once and writes what changes. So the time is
// latency: trim 3 us, extend's launches 4.4 and 7.4 us with 64 rows and 4096 pages, 4.8 and 9 with 1000 and 262144.
#include <hip/hip_runtime.h>

#include "../../include/qgemv.h"
#include "kv_pages.h"
#include "launch.h"

namespace qg {

constexpr int kRowThreads = 256;

// ---- trim ------------------------------------------------------------------------------------

// A wave for each row: the entries past the kept tokens' pages give up their page. A row is one
// wave's, and the counts are atomic sums, so the order of the rows changes nothing.
__global__ __launch_bounds__(kRowThreads) void kv_trim_kernel(int32_t *table, int64_t ld, int32_t rows, int64_t capacity,
                                                             int32_t tok_shift, int32_t *lens, int32_t *refs,
                                                             int32_t num_pages, const int32_t *to) {
  const int32_t r = (int32_t)(blockIdx.x * (kRowThreads / 64) + (threadIdx.x >> 6)), lane = threadIdx.x & 63;
  if (r >= rows) return;
  const int32_t keep = to[r], raw = lens[r];
  const int64_t len = raw < capacity ? raw : capacity;
  if (keep < 0 || keep >= len) return;
  const int32_t t1 = (1 << tok_shift) - 1;
  const int64_t last = (len + t1) >> tok_shift;
  int32_t *row = table + (int64_t)r * ld;
  for (int64_t j = (((int64_t)keep + t1) >> tok_shift) + lane; j < last; j += 64) {
    const int32_t e = row[j];
    if (e >= 0 && e < num_pages) atomicSub(refs + e, 1);
    row[j] = -1;
  }
  if (lane == 0) lens[r] = keep;
}

// ---- extend ------------------------------------------------------------------------------------
//
// With n_r tokens asked for row r, N_r = n_0 + .. + n_r, the pages that row r lacks (0 for a row that
// is refused for itself) and their sum P_r up to r, row r is served if N_r <= slots and, where it
// lacks pages, P_r <= the number of free pages; its pages are the free ones of rank P_(r-1) to P_r - 1.
// The sums are kept saturated (at slots + 1, and at num_pages + 1): a sum past its limit decides the
// same whatever it is, and a saturated sum is still associative.
//
// Two launches. The first counts the free pages of each block of kBlockPages and makes the rows' sums in one
// workgroup. In the second, workgroups find the row of each free page's rank, the row of each slot,
// and write the rows' results; they read only what the first launch wrote, and refs of their own block.

constexpr int kScanThreads = 1024;
constexpr int kBlockPages = 4 * kScanThreads;
constexpr int32_t kSamples = 4096;                  // entries of a sum that a search holds in LDS

struct ExtendArgs {
  int32_t *table;
  int64_t ld;
  int32_t rows, tok_shift;
  int64_t capacity;              // tokens of a row
  int32_t *lens, *refs;
  int32_t num_pages, blocks;
  const int32_t *add;
  int32_t *granted, *starts, *seqs, *positions;
  int32_t slots;
  int32_t *free_blocks;          // workspace: free pages of each block,
  uint32_t *ends, *upto;         // N_r and P_r,
  int32_t *len, *state;          // the rows' lengths, and kOk and kNeeds of each
};
constexpr int32_t kOk = 1, kNeeds = 2;

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b, uint32_t cap) { return min(a + b, cap); }

// Sum over this thread and those before it, saturated at cap; total: over all. lds: 16 values.
__device__ __forceinline__ uint32_t block_scan_sat(uint32_t v, uint32_t cap, uint32_t *lds, uint32_t &total) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t up = (uint32_t)__shfl_up((int)v, o);
    if ((int)(threadIdx.x & 63) >= o) v = sat_add(v, up, cap);
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 63) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t before = 0, all = 0;
  for (int w = 0; w < kScanThreads / 64; ++w) {
    const uint32_t x = lds[w];
    if (w < (int)(threadIdx.x >> 6)) before = sat_add(before, x, cap);
    all = sat_add(all, x, cap);
  }
  total = all;
  return sat_add(before, v, cap);
}

// Row r's request: tokens (saturated), pages that it lacks, and whether anything of its own refuses it.
struct Request {
  uint32_t tokens, pages;
  int32_t len;
  bool ok;
};
__device__ __forceinline__ Request request_of(const ExtendArgs &a, int32_t r) {
  Request q{0, 0, 0, false};
  if (r >= a.rows) return q;
  const int32_t n = max(a.add[r], 0), raw = max(a.lens[r], 0);
  q.len = (int32_t)(raw < a.capacity ? raw : a.capacity);
  q.tokens = min((uint32_t)n, (uint32_t)a.slots + 1);
  const int32_t t1 = (1 << a.tok_shift) - 1;
  const int64_t end = (int64_t)q.len + n;
  q.ok = n > 0 && end <= a.capacity;
  if (!q.ok) return q;
  if (q.len & t1) {              // the page that takes the first new token holds others of this row: no other row may hold it
    const int32_t e = a.table[(int64_t)r * a.ld + (q.len >> a.tok_shift)];
    q.ok = e >= 0 && e < a.num_pages && a.refs[e] == 1;
    if (!q.ok) return q;
  }
  q.pages = (uint32_t)(((end + t1) >> a.tok_shift) - (((int64_t)q.len + t1) >> a.tok_shift));
  return q;
}

__global__ __launch_bounds__(kScanThreads) void kv_extend_count_kernel(ExtendArgs a) {
  __shared__ uint32_t lds[kScanThreads / 64];
  if ((int32_t)blockIdx.x < a.blocks) {
    uint32_t n = 0, total;
    for (int u = 0; u < 4; ++u) {
      const int64_t p = (int64_t)blockIdx.x * kBlockPages + u * kScanThreads + threadIdx.x;
      if (p < a.num_pages) n += a.refs[p] <= 0;
    }
    block_scan_sat(n, kBlockPages, lds, total);
    if (threadIdx.x == 0) a.free_blocks[blockIdx.x] = (int32_t)total;
    return;
  }
  const uint32_t cap_n = (uint32_t)a.slots + 1, cap_p = (uint32_t)a.num_pages + 1;
  uint32_t sum_n = 0, sum_p = 0;
  for (int32_t r0 = 0; r0 < a.rows; r0 += kScanThreads) {
    const int32_t r = r0 + (int32_t)threadIdx.x;
    Request q = request_of(a, r);
    uint32_t all_n, all_p;
    const uint32_t n = sat_add(sum_n, block_scan_sat(q.tokens, cap_n, lds, all_n), cap_n);
    q.ok = q.ok && n <= (uint32_t)a.slots;
    if (!q.ok) q.pages = 0;
    const uint32_t p = sat_add(sum_p, block_scan_sat(min(q.pages, cap_p), cap_p, lds, all_p), cap_p);
    sum_n = sat_add(sum_n, all_n, cap_n);
    sum_p = sat_add(sum_p, all_p, cap_p);
    if (r < a.rows) {
      a.ends[r] = n;
      a.upto[r] = p;
      a.len[r] = q.len;
      a.state[r] = (q.ok ? kOk : 0) | (q.pages ? kNeeds : 0);
    }
  }
}

// The first r with sums[r] > x (rows: none). samples: every stride-th entry in LDS, count of them.
__device__ __forceinline__ int32_t find_row(const uint32_t *samples, int32_t count, int32_t stride, const uint32_t *sums,
                                           int32_t rows, uint32_t x) {
  int32_t lo = 0, hi = count;                        // samples[i] = sums[min((i + 1) * stride, rows) - 1]
  while (lo < hi) {
    const int32_t mid = (lo + hi) >> 1;
    if (samples[mid] > x) hi = mid; else lo = mid + 1;
  }
  if (stride == 1 || lo == count) return min(lo * stride, rows);
  int32_t a = lo * stride, b = min(a + stride, rows) - 1;   // sums[b] > x
  while (a < b) {
    const int32_t mid = (a + b) >> 1;
    if (sums[mid] > x) b = mid; else a = mid + 1;
  }
  return a;
}

__global__ __launch_bounds__(kScanThreads) void kv_extend_kernel(ExtendArgs a, int32_t row_blocks) {
  __shared__ uint32_t lds[kScanThreads / 64];
  __shared__ uint32_t samples[kSamples];
  const int32_t b = blockIdx.x, tid = threadIdx.x;
  const bool page_part = b < a.blocks, row_part = !page_part && b < a.blocks + row_blocks;
  // free pages before this block, and in all
  uint32_t mine = 0, all = 0;
  for (int32_t k = tid; k < a.blocks; k += kScanThreads) {
    const uint32_t n = (uint32_t)a.free_blocks[k];
    all += n;
    mine += k < b ? n : 0;
  }
  uint32_t total, before;
  block_scan_sat(all, 0x7FFFFFFF, lds, total);
  block_scan_sat(mine, 0x7FFFFFFF, lds, before);
  auto served = [&](int32_t r) { return (a.state[r] & kOk) && (!(a.state[r] & kNeeds) || a.upto[r] <= total); };
  if (row_part) {
    const int32_t r = (b - a.blocks) * kScanThreads + tid;
    if (a.starts && r <= a.rows) a.starts[r] = r ? (int32_t)min(a.ends[r - 1], (uint32_t)a.slots) : 0;
    if (r >= a.rows) return;
    const int32_t n = served(r) ? a.add[r] : 0;
    a.granted[r] = n;
    if (n) a.lens[r] = a.len[r] + n;
    return;
  }
  const uint32_t *sums = page_part ? a.upto : a.ends;
  const int32_t stride = (a.rows + kSamples - 1) / kSamples, count = stride ? (a.rows + stride - 1) / stride : 0;
  for (int32_t i = tid; i < count; i += kScanThreads) samples[i] = sums[min((i + 1) * stride, a.rows) - 1];
  __syncthreads();
  if (page_part) {
    if (count == 0 || before >= samples[count - 1]) return;
    const int64_t p0 = (int64_t)b * kBlockPages + 4 * tid;   // four neighbours a thread
    bool is_free[4];
    uint32_t n = 0, unused;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      is_free[u] = p0 + u < a.num_pages && a.refs[p0 + u] <= 0;
      n += is_free[u];
    }
    uint32_t rank = before + block_scan_sat(n, kBlockPages, lds, unused) - n;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (!is_free[u]) continue;
      const int32_t r = find_row(samples, count, stride, a.upto, a.rows, rank);
      if (r < a.rows && a.upto[r] <= total) {
        const uint32_t first = r ? a.upto[r - 1] : 0;
        const int64_t held = ((int64_t)a.len[r] + (1 << a.tok_shift) - 1) >> a.tok_shift;
        a.table[(int64_t)r * a.ld + held + (rank - first)] = (int32_t)(p0 + u);
        a.refs[p0 + u] = 1;
      }
      ++rank;
    }
    return;
  }
  const int64_t i = (int64_t)(b - a.blocks - row_blocks) * kScanThreads + tid;
  if (i >= a.slots) return;
  const int32_t r = find_row(samples, count, stride, a.ends, a.rows, (uint32_t)i);
  int32_t s = -1, pos = -1;
  if (r < a.rows && served(r)) {
    s = r;
    pos = a.len[r] + (int32_t)(i - (r ? a.ends[r - 1] : 0));
  }
  a.seqs[i] = s;
  a.positions[i] = pos;
}

namespace {

// Tokens of a table's row: lengths are int32.
int64_t row_capacity(const qg_kv_pool *pool, int64_t table_pages) {
  const int64_t n = table_pages * pool->page_tokens;
  return n < 0x7FFFFFFF ? n : 0x7FFFFFFF;
}

bool misaligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) != 0; }

constexpr int64_t kExtendPages = int64_t(1) << 24;
constexpr int64_t kExtendRows = 65536;
constexpr int64_t kExtendSlots = int64_t(1) << 26;

int64_t extend_blocks(int64_t num_pages) { return (num_pages + kBlockPages - 1) / kBlockPages; }

}  // namespace

}  // namespace qg

using namespace qg;

extern "C" {

int qg_kv_trim(const qg_kv_pool *pool, int32_t *table, int64_t ld_table, int64_t table_rows, int64_t table_pages,
               int32_t *lens, int32_t *refs, const int32_t *to, void *stream) {
  KvLayout L;
  if (int st = kv_pool_layout(pool, &L)) return st;
  if (int st = kv_table_check(table, ld_table, table_rows, table_pages)) return st;
  if (table_rows > kExtendRows) return QG_ERR_SHAPE;
  if (table_rows == 0) return QG_OK;
  if (!lens || !refs || !to) return QG_ERR_NULL;
  if (misaligned4(lens) || misaligned4(refs) || misaligned4(to)) return QG_ERR_ALIGN;
  const int64_t capacity = row_capacity(pool, table_pages);
  constexpr int64_t kRows = kRowThreads / 64;
  return launch(kv_trim_kernel, dim3((unsigned)((table_rows + kRows - 1) / kRows)), dim3(kRowThreads), 0,
                static_cast<hipStream_t>(stream), table, ld_table, (int32_t)table_rows, capacity,
                (int32_t)__builtin_ctz(pool->page_tokens), lens, refs, (int32_t)pool->num_pages, to);
}

int qg_kv_extend_bytes(const qg_kv_pool *pool, int64_t table_rows, int64_t *bytes) {
  if (!bytes) return QG_ERR_NULL;
  KvLayout L;
  if (int st = kv_pool_layout(pool, &L)) return st;
  if (table_rows < 0 || table_rows > kExtendRows || pool->num_pages > kExtendPages) return QG_ERR_SHAPE;
  *bytes = 4 * (extend_blocks(pool->num_pages) + 4 * table_rows);
  return QG_OK;
}

int qg_kv_extend(const qg_kv_pool *pool, int32_t *table, int64_t ld_table, int64_t table_rows, int64_t table_pages,
                 int32_t *lens, int32_t *refs, const int32_t *add, int32_t *granted, int32_t *starts, int32_t *seqs,
                 int32_t *positions, int64_t slots, void *workspace, int64_t workspace_bytes, void *stream) {
  KvLayout L;
  if (int st = kv_pool_layout(pool, &L)) return st;
  if (int st = kv_table_check(table, ld_table, table_rows, table_pages)) return st;
  if (slots < 0 || slots > kExtendSlots) return QG_ERR_SHAPE;
  int64_t need = 0;
  if (int st = qg_kv_extend_bytes(pool, table_rows, &need)) return st;
  if (!refs || !workspace || (table_rows && (!lens || !add || !granted)) || (slots && (!seqs || !positions))) return QG_ERR_NULL;
  if (misaligned4(lens) || misaligned4(refs) || misaligned4(add) || misaligned4(granted) || misaligned4(starts) ||
      misaligned4(seqs) || misaligned4(positions) || misaligned4(workspace))
    return QG_ERR_ALIGN;
  if (workspace_bytes < need) return QG_ERR_WORKSPACE;
  ExtendArgs a;
  a.table = table;
  a.ld = ld_table;
  a.rows = (int32_t)table_rows;
  a.tok_shift = __builtin_ctz(pool->page_tokens);
  a.capacity = row_capacity(pool, table_pages);
  a.lens = lens;
  a.refs = refs;
  a.num_pages = (int32_t)pool->num_pages;
  a.blocks = (int32_t)extend_blocks(pool->num_pages);
  a.add = add;
  a.granted = granted;
  a.starts = starts;
  a.seqs = seqs;
  a.positions = positions;
  a.slots = (int32_t)slots;
  a.free_blocks = static_cast<int32_t *>(workspace);
  a.ends = reinterpret_cast<uint32_t *>(a.free_blocks + a.blocks);
  a.upto = a.ends + table_rows;
  a.len = reinterpret_cast<int32_t *>(a.upto + table_rows);
  a.state = a.len + table_rows;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 block(kScanThreads);
  if (int st = launch(kv_extend_count_kernel, dim3((unsigned)a.blocks + 1), block, 0, s, a)) return st;
  const int32_t row_blocks = (int32_t)(table_rows / kScanThreads + 1);
  const int64_t slot_blocks = (slots + kScanThreads - 1) / kScanThreads;
  return launch(kv_extend_kernel, dim3((unsigned)(a.blocks + row_blocks + slot_blocks)), block, 0, s, a, row_blocks);
}

}  // extern "C"
