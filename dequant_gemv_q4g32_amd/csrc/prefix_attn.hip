// Attention of one new token a sequence where neighbouring sequences share their first tokens, gfx950.
//
// A group's rows with the heads of a KV head are one block of queries against the shared tokens: unlike a single
// sequence's few heads, enough of them to keep the matrix cores busy. One launch does both kinds of work, each on its
// share of the workgroups: the shared tokens, once a group, in one pass with a running reference, up to 256 query rows
// a workgroup, and the tokens that a row has for itself, as paged_attn.hip does them, a wave for up to 16 heads. The
// second kind also takes groups of few rows, 16 query rows (rows by heads) in place of a row's heads, or
// their rows one by one. A second launch joins the parts.
//
// Measured: 128 rows of 32 heads on 8 of 128 after 16384 shared int8 tokens, up to 1024 of their own, take 90 and 8 us; a
// pass over the shared tokens for each row would read 4.6 GB, 670 us at HBM's rate. Shared work reaches 530 to 650
// TFLOP/s on its workgroups, the weights' second halves not counted; a large library product 1150 on all. Of a tile's 3.3 us
// the matrix instructions are busy for 1.5, the vector instructions about as long, LDS for 0.9, and the two waves of a SIMD do
// not overlap them all. Own work runs at 28 to 38 KB a us and workgroup: instruction issue for int8, loads in flight for
// fp16. Short calls are latency: 3 us for the plan, 5 to the first scores (page, K, LDS), 2 to 3 to
// store the parts, 4 to 9 for the join (8 rows after 1000 tokens: 12 and 4).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "../../include/qgemv.h"
#include "attn_common.h"
#include "device_common.h"
#include "kv_pages.h"
#include "launch.h"

namespace qg {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Waves of a workgroup, each with 32 query rows of the shared tokens: two on every SIMD, so that one's vector
// instructions run beside the other's matrix instructions. Heads of 256 take the registers of two.
__host__ __device__ constexpr int prefix_waves(int dim) { return dim == 256 ? 4 : 8; }
// Shared tokens of a tile: 8192 elements of K, and of V.
__host__ __device__ constexpr int tile_tokens(int dim) { return 8192 / dim; }
// Heads of a KV head that a wave takes against a row's own tokens.
constexpr int kHeads = 16;
constexpr int kMaxGroups = 1023;
// Scores (s times the scale, units of log2) from which on a weight takes its exponent from the rounded product, as own
// work's do and as the reference is placed; below, from s by one fused operation. The two differ by half a
// last place of the score: here 2^-13 at most, but 16 for a score of 2^28, which would carry weights out of fp16.
constexpr float kFused = 4096.0f;

// Both kinds of work lie on a line each, segment after segment, and every worker (a workgroup of shared work, a wave of
// own work) gets an equal part of its line. A segment's first units are a lead, which stands for what its start costs a
// worker that comes from another one.
constexpr int32_t kLead = 4;
// The same for own work, about 3 us; a step takes what its bytes do, of which the waves of a workgroup together
// get 38 KB a us, or 28 where they are decoded. (64 rows after 8192 fp16 tokens take 62 us at 30 and 38 and 64 at 46, 128
// after 16384 int8 ones 102 at 28 and 103 at 24 and 36, 48 rows of 16 heads of 256 41 at 24 and 28 and 43 at 36.)
__host__ __device__ constexpr double own_step_us(int dim, bool q8) {
  return prefix_waves(dim) * 32 * dim * (q8 ? 2.125 / 28e3 : 4.0 / 38e3);
}
__host__ __device__ constexpr int32_t own_lead(int dim, bool q8) { return (int32_t)(3.0 / own_step_us(dim, q8) + 0.5); }
// What the workgroups find out of a group (of at least two rows). Its query rows are rows * (heads of a KV head), in
// tiles a KV head; its tokens, whole pages, are tiles too. On the line of shared work its segments (KV head, row tile)
// follow each other, `units` each.
struct GroupPlan {
  int32_t row0, rows, tokens, row_tiles, units;
  uint32_t unit0;                // units of the groups before
};
// A group of few query rows goes to the line of own work instead (row_tiles 0), before its first row: 16 query rows are a
// pack, and a KV head's packs have `units` each as if they were heads of a row.
//
// Of a row: its group (-1: it shares nothing), and its place on the line of own work: the packs that it is the first row
// of, then for each head tile in turn `units`, a lead and steps of 32 tokens, or none.
struct RowPlan {
  int32_t group;
  uint32_t unit0, units;
};
// Of the call: both lines, and their workers.
struct Split {
  uint32_t shared, workers, own, waves;
};

// Partial results: query rows' sums, and their references and denominators. From one part to the next on a line the
// worker or the segment goes up, or both: a worker's rows of a segment lie behind as many as a part has at most for each
// worker before it, and the rows of all segments before (part_row, own_part).
struct Parts {
  float *o, *ml;                 // [rows][D], [rows][2]
};

struct PrefixArgs {
  const uint8_t *pool;           // the layer's first page
  int64_t page_bytes, head_bytes;
  int32_t v_off, ks_off, vs_off;
  int32_t num_pages, tok_shift;
  const uint16_t *q;
  int64_t ldq;
  const int32_t *table;
  int64_t ld_table;
  const int32_t *lens, *starts, *prefix;
  int32_t groups, batch, heads, group, kv_heads;   // group = heads / kv_heads
  int32_t tiles_per_kv, head_tiles;   // own work: head tiles of a KV head, and of all of them
  int32_t max_len;
  int32_t part_rows, own_rows;   // the most query rows of a part of shared work, and of own work
  int32_t own_lead;              // of own work's segments
  uint32_t own_most;             // waves that own work may have: the parts' room
  float shared_cost, tile_steps; // of a tile of shared work for a workgroup, in steps of own work of a wave: of each of
                                 // its waves, and of all where they all do such work
  float scale_log2;              // |scale| * log2(e), or 1 where that is not a normal number;
  uint32_t keep, flip;           // for these, q is taken as zero, or as its negative: masks of two fp16 numbers
  void *out;
  int64_t ldo;
  int32_t out_f32;
  float *lse;
  Split *split;                  // workspace: what the join has to know,
  GroupPlan *plan;
  RowPlan *rows;
  Parts parts, packs, own_parts; // and the partial results
};

// ---- the plan ------------------------------------------------------------------------------------
//
// Every workgroup makes the whole plan by itself: it is a chain of three loads and some sums, and a launch of its
// own took 5 us.

__device__ __forceinline__ uint32_t scan_max(uint32_t v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t up = (uint32_t)__shfl_up((int)v, o);
    if ((int)(threadIdx.x & 63) >= o) v = max(v, up);
  }
  return v;
}

struct Plan {
  int32_t lead[kMaxGroups + 1];  // the groups' first rows, made to ascend, and the last one's end
  GroupPlan g[kMaxGroups];
  uint32_t red[8];
  uint32_t found[2][8];

  // the group of row b, -1: none
  __device__ __forceinline__ int32_t group_of(int32_t b, int32_t groups) const {
    int32_t lo = 0, hi = groups + 1;                 // the last lead <= b is lo - 1
    while (lo < hi) {
      const int32_t mid = (lo + hi) >> 1;
      if (lead[mid] <= b) lo = mid + 1; else hi = mid;
    }
    return lo > groups || lo == 0 || g[lo - 1].tokens == 0 ? -1 : lo - 1;
  }
};

// The sum over the threads before this one, and in all.
template <int W>
__device__ __forceinline__ uint32_t scan_sum(uint32_t x, uint32_t &all, Plan &p) {
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, sum = wave_scan(x);
  __syncthreads();
  if (lane == 63) p.red[wave] = sum;
  __syncthreads();
  uint32_t before = 0, total = 0;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    const uint32_t r = p.red[k];
    before += k < (int)wave ? r : 0;
    total += r;
  }
  all = uniform(total);
  return before + sum - x;
}

// Where worker w puts query row m of a KV head of a group.
__device__ __forceinline__ int64_t part_row(const PrefixArgs &a, const GroupPlan &p, uint32_t w, int32_t kvh, int32_t m) {
  return (int64_t)w * a.part_rows + (int64_t)p.row0 * a.heads + (int64_t)kvh * p.rows * a.group + m;
}

// The same for a pack's and wave w.
__device__ __forceinline__ int64_t pack_row(const PrefixArgs &a, const GroupPlan &p, uint32_t w, int32_t kvh, int32_t m) {
  return (int64_t)w * kHeads + (int64_t)p.row0 * a.heads + (int64_t)kvh * p.rows * a.group + m;
}
__device__ __forceinline__ int32_t packs_of(const PrefixArgs &a, const GroupPlan &p) { return (p.rows * a.group + kHeads - 1) / kHeads; }
// What the packs before row b's own tokens have on the line.
__device__ __forceinline__ uint32_t pack_units(const PrefixArgs &a, const GroupPlan &p, int32_t b) {
  return p.row0 == b && p.tokens && !p.row_tiles ? (uint32_t)(packs_of(a, p) * a.kv_heads) * (uint32_t)p.units : 0;
}

// And wave v the first row of its part of a head tile of row b.
__device__ __forceinline__ int64_t own_part(const PrefixArgs &a, uint32_t v, int32_t b, int32_t ht) {
  return ((int64_t)v + (int64_t)b * a.head_tiles + ht) * a.own_rows;
}

// What of a row's tokens is its own: [first, len), in steps of 32 from base = first rounded down, and the units
// that a head tile of it has on the line.
struct Own {
  int32_t first, len, base;
  uint32_t units;
};
__device__ __forceinline__ Own own_of(const PrefixArgs &a, int32_t raw, int32_t shared) {
  Own o;
  o.len = min(max(raw, 0), a.max_len);
  o.first = min(shared, o.len);
  o.base = o.first & ~(kTile - 1);
  o.units = o.first < o.len ? (uint32_t)(o.len - o.base + kTile - 1) / kTile + a.own_lead : 0;
  return o;
}

// ---- the shared tokens ---------------------------------------------------------------------------

// What a tile is to a workgroup. K is fetched 16 bytes a thread and load, V in pieces of four tokens by four
// elements, so that the 64 lanes of a load lie in one block of 16 tokens: its page is scalar. In LDS K is [T][D], V^T
// [D][T] with each 16 bytes the eight tokens of a lane's operand (16 s + 4 h + {0..3, 8..11} for step s, lane half h:
// place 2 s + h). 16 neighbouring lanes read the same place of neighbouring rows at once, which shall lie in different
// banks, and all places of a lane are constants away from one address. So a row of K has 16 bytes more than
// it needs; V^T, which a lane writes four rows apart from its neighbour, has rows of 4 places mod 16 and one more after
// every four rows: both ways all 16 differ. (With one more place a row the writes met 4 to a bank: 4 us more for 128 rows
// after 16384 int8 tokens.)
template <int D, bool Q8>
struct Shape {
  static constexpr int NT = 64 * prefix_waves(D);
  static constexpr int T = tile_tokens(D);
  static constexpr int TB = T / 32;                 // blocks of 32 tokens
  static constexpr int KS = D / 16;                 // matrix steps along the head
  static constexpr int DB = D / 32;                 // blocks of 32 elements of the head
  static constexpr int KBytes = Q8 ? D : 2 * D;     // bytes of a token's K
  static constexpr int KPer = KBytes / 16;          // loads of a token's K
  static constexpr int KL = T * KPer / NT;          // such loads a thread
  static constexpr int VPer = D / 4;                // pieces of four tokens' V
  static constexpr int VL = T / 4 * VPer / NT;      // pieces a thread
  static constexpr uint32_t KRow = D / 8 + 1;       // 16-byte places of a row of K in LDS,
  static constexpr uint32_t VRow = T / 8 == 4 ? 4 : T / 8 + 4, VFour = 4 * VRow + 1;   // of one of V^T, and of four
  static constexpr uint32_t KTile = T * KRow, VTile = D / 4 * VFour;   // and of a tile
  static constexpr uint32_t kLds = 16 * 3 * (KTile + VTile);      // bytes of three tiles
};

// K and V of a tile on its way, and their way into LDS. A page that is none has an empty range, whose loads
// give zeros.
template <int D, bool Q8>
struct StagedK {
  using S = Shape<D, Q8>;
  u32x4 k[S::KL];
  uint32_t s[S::KL];
  __device__ __forceinline__ void write(u32x4 *lds) const {
    const uint32_t at = threadIdx.x / S::KPer * S::KRow + threadIdx.x % S::KPer * (Q8 ? 2 : 1);
#pragma unroll
    for (int i = 0; i < S::KL; ++i) {
      u32x4 *to = lds + at + i * (S::NT / S::KPer) * S::KRow;
      if constexpr (Q8) {
        const uint32_t d = s[i] * 0x00010001u;
        u32x4 w[2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x = k[i][j] ^ 0x80808080u;
          w[j >> 1][2 * (j & 1)] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, x, kSelLow), d);
          w[j >> 1][2 * (j & 1) + 1] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, x, kSelHigh), d);
        }
        to[0] = w[0];
        to[1] = w[1];
      } else {
        to[0] = k[i];
      }
    }
  }
};

template <int D, bool Q8>
struct StagedV {
  using S = Shape<D, Q8>;
  u32x2 v[S::VL][4];                               // int8: one dword each
  u32x2 s[S::VL];
  __device__ __forceinline__ void write(u32x4 *lds) const {
    const uint32_t d0 = 4 * (threadIdx.x % S::VPer), run = threadIdx.x / S::VPer;   // of four tokens
    const uint32_t at = d0 / 4 * S::VFour + 2 * (run >> 2) + (run & 1), half = (run >> 1) & 1;
#pragma unroll
    for (int i = 0; i < S::VL; ++i) {
      u32x2 e[4];                                   // elements d0 .. d0 + 3, four tokens each
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if constexpr (Q8) {
          const uint32_t x0 = v[i][2 * p].x ^ 0x80808080u, x1 = v[i][2 * p + 1].x ^ 0x80808080u, d = s[i][p];
          const uint32_t a = __builtin_amdgcn_perm(x1, x0, 0x05010400u), b = __builtin_amdgcn_perm(x1, x0, 0x07030602u);
          e[0][p] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, a, kSelLow), d);
          e[1][p] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, a, kSelHigh), d);
          e[2][p] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, b, kSelLow), d);
          e[3][p] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, b, kSelHigh), d);
        } else {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            e[2 * w][p] = __builtin_amdgcn_perm(v[i][2 * p + 1][w], v[i][2 * p][w], 0x05040100u);
            e[2 * w + 1][p] = __builtin_amdgcn_perm(v[i][2 * p + 1][w], v[i][2 * p][w], 0x07060302u);
          }
        }
      }
      constexpr uint32_t kStep = S::NT / S::VPer / 2;   // places between a thread's pieces: their runs are a multiple of 4 apart
      static_assert(S::VL == 1 || S::NT / S::VPer % 4 == 0, "the pieces' halves agree");
#pragma unroll
      for (int j = 0; j < 4; ++j) *(reinterpret_cast<u32x2 *>(lds + at + j * S::VRow + i * kStep) + half) = e[j];
    }
  }
};

// A worker's part [at, end) of the line of shared work, segment by segment. The weights are hi + lo fp16 pairs (22
// bits), for fp16 results too: as one fp16 number they would add as much to such a result's error as its own rounding, and
// where the values all but cancel 30 times what pairs do. (A tile would take 2.3 to 2.7 us in place of 3.3, the call for 128 rows
// after 16384 int8 tokens 88 in place of 102.)
//
// The work is in steps of 32 tokens, three of which are under way at once, each independent of the others: the
// scores of the next, the softmax of this one, the products with V of the one before. So matrix and vector
// instructions alternate throughout. K and V lie in three buffers of a tile each: a tile's writing, its scores'
// reading and its products' reading go on between the same two barriers.
//
// S^T = K Q^T and O^T += V^T P^T on v_mfma_f32_32x32x16_f16: a lane of S^T holds one query row and 16 of 32
// tokens, which is the operand that P^T has to be, so the softmax stays in the registers.
template <int D, bool Q8>
__device__ __forceinline__ void shared_work(const PrefixArgs &a, const Plan &plan, u32x4 *tiles, uint32_t w, uint32_t at, uint32_t end) {
  using S = Shape<D, Q8>;
  constexpr int T = S::T, TB = S::TB, KS = S::KS, DB = S::DB, kBlocks = T / 16, kRows = S::NT / 2, NT = S::NT;
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), n = lane & 31, h = lane >> 5;
  u32x4 *const lds_k = tiles, *const lds_v = tiles + 3 * S::KTile;
  const uint32_t k_at = n * S::KRow + h, v_at = n / 4 * S::VFour + n % 4 * S::VRow + h;   // a lane's places of K and V
  // a lane's part of an address of K and V, beside the wave's first rows
  const uint32_t k_lane = (lane / S::KPer) * S::KBytes + 16 * (lane % S::KPer);
  const uint32_t ks_lane = Q8 ? (lane / S::KPer) * (D / 16) + 2 * (lane % S::KPer / 2) : 0;
  const uint32_t v_run = lane / S::VPer, v_lane = 4 * v_run * S::KBytes + (Q8 ? 4 : 8) * (tid % S::VPer);
  const uint32_t vs_lane = 2 * (((4 * (tid % S::VPer) / 32) << a.tok_shift) + 4 * v_run);
  int32_t g = 0;
  {                                                  // the last group with unit0 <= at
    int32_t lo = 0, hi = a.groups;
    while (lo < hi) {
      const int32_t mid = (lo + hi) >> 1;
      if (uniform(plan.g[mid].unit0) <= at) lo = mid + 1; else hi = mid;
    }
    g = lo - 1;
  }
  while (at < end) {
    const GroupPlan p{uniform(plan.g[g].row0), uniform(plan.g[g].rows), uniform(plan.g[g].tokens), uniform(plan.g[g].row_tiles),
                      uniform(plan.g[g].units), uniform(plan.g[g].unit0)};
    const int32_t rows = p.rows * a.group;
    const uint32_t segs = (uint32_t)(p.row_tiles * a.kv_heads);
    if (p.units == 0 || at - p.unit0 >= segs * (uint32_t)p.units) {
      ++g;
      continue;
    }
    const uint32_t seg = (at - p.unit0) / (uint32_t)p.units, u = at - p.unit0 - seg * (uint32_t)p.units;
    const uint32_t until = min(u + (end - at), (uint32_t)p.units);
    at += until - u;
    if (until <= kLead) continue;
    const uint32_t first = max(u, (uint32_t)kLead) - kLead, last = until - kLead;   // tiles of the group's tokens
    const int32_t kvh = (int32_t)(seg / (uint32_t)p.row_tiles), rt = (int32_t)seg - kvh * p.row_tiles;
    const int32_t *row = a.table + (int64_t)p.row0 * a.ld_table;
    const uint8_t *kv = a.pool + kvh * a.head_bytes;

    // The pages of 64 blocks of 16 tokens, a block a lane (-1: none, or not this worker's); those of the next 64
    // on their way.
    const uint32_t blocks = min(last * kBlocks, (uint32_t)p.tokens / 16);
    auto pages_at = [&](uint32_t blk) { return blk + lane < blocks ? row[(int64_t)(blk + lane) * 16 >> a.tok_shift] : -1; };
    auto in_pool = [&](int32_t page) { return page < a.num_pages ? max(page, -1) : -1; };
    uint32_t base = first * kBlocks;                 // of the blocks in ids
    int32_t ids = in_pool(pages_at(base)), ids_next = pages_at(base + 64);
    auto block = [&](int32_t page) {
      return make_rsrc(kv + (uint64_t)(uint32_t)max(page, 0) * (uint64_t)a.page_bytes, page < 0 ? 0u : (uint32_t)a.head_bytes);
    };
    const uint32_t mask = (1u << a.tok_shift) - 1;
    int32_t v_page[S::VL];                           // of the tile whose K was fetched last: for its V
    uint32_t fine = 0;                               // that tile's blocks that are in a page
    auto fetch_k = [&](uint32_t tile, StagedK<D, Q8> &t) {
      if (tile * kBlocks >= base + 64) {
        base += 64;
        ids = in_pool(ids_next);
        ids_next = pages_at(base + 64);
      }
      const uint32_t b0 = tile * kBlocks - base;
      fine = (uint32_t)(__ballot(ids >= 0) >> b0) & ((1u << kBlocks) - 1);
#pragma unroll
      for (int i = 0; i < S::KL; ++i) {
        const uint32_t r = (64 * wave + NT * i) / S::KPer;   // the load's first token, a lane's others in k_lane
        const rsrc_t rs = block(__builtin_amdgcn_readlane(ids, b0 + r / 16));
        const uint32_t place = (tile * T + r) & mask;
        t.k[i] = bldx4<0>(rs, k_lane, place * S::KBytes);
        if constexpr (Q8) t.s[i] = bldh(rs, ks_lane, a.ks_off + place * (D / 16));
      }
#pragma unroll
      for (int i = 0; i < S::VL; ++i) v_page[i] = __builtin_amdgcn_readlane(ids, b0 + (64 * wave + NT * i) / S::VPer / 4);
    };
    auto fetch_v = [&](uint32_t tile, const int32_t *pages, StagedV<D, Q8> &t) {
#pragma unroll
      for (int i = 0; i < S::VL; ++i) {
        const uint32_t r = 4 * ((64 * wave + NT * i) / S::VPer);
        const rsrc_t rs = block(pages[i]);
        const uint32_t place = (tile * T + r) & mask;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (Q8) t.v[i][j].x = bldx1<0>(rs, v_lane + j * S::KBytes, a.v_off + place * S::KBytes);
          else t.v[i][j] = bldx2<0>(rs, v_lane + j * S::KBytes, a.v_off + place * S::KBytes);
        }
        if constexpr (Q8) t.s[i] = bldx2<0>(rs, vs_lane, a.vs_off + 2 * place);
      }
    };

    StagedK<D, Q8> kt, kt1;
    StagedV<D, Q8> vt;
    int32_t pages[S::VL];                            // of V of the tile after the one in vt
    fetch_k(first, kt);
    uint32_t cur = fine;
#pragma unroll
    for (int i = 0; i < S::VL; ++i) pages[i] = v_page[i];
    fetch_v(first, pages, vt);
    fetch_k(first + 1, kt1);
    uint32_t next_fine = fine;
#pragma unroll
    for (int i = 0; i < S::VL; ++i) pages[i] = v_page[i];
    // the lane's query row; one that is not finite is taken as zeros, and marked
    const int32_t m = rt * kRows + (int32_t)(32 * wave + n);
    const bool active = rt * kRows + (int32_t)(32 * wave) < rows;
    const int32_t b = p.row0 + min(m, rows - 1) / a.group, hd = kvh * a.group + min(m, rows - 1) % a.group;
    half8_t q[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i)
      q[i] = *reinterpret_cast<const half8_t *>(a.q + b * a.ldq + (int64_t)hd * D + 16 * i + 8 * h);
    const int32_t limit = min(max(a.lens[b], 0), p.tokens);   // the tokens that the row sees
    const bool whole = !__any(limit < p.tokens);
    bool bad = nonfinite<KS>(q);
    bad = __shfl_xor((int)bad, 32) || bad;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      u32x4 x = __builtin_bit_cast(u32x4, q[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = m < rows && !bad ? (x[j] & a.keep) ^ a.flip : 0u;
      q[i] = __builtin_bit_cast(half8_t, x);
    }
    f32x16 o[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
    float ref = -INFINITY, l = 0.f;
    bool rounded = false;                            // whether a reference of the wave is past kFused

    __syncthreads();                                 // the segment before is done with LDS
    kt.write(lds_k);
    vt.write(lds_v);
    kt1.write(lds_k + S::KTile);
    fetch_k(first + 2, kt);
    fetch_v(first + 1, pages, vt);
#pragma unroll
    for (int i = 0; i < S::VL; ++i) pages[i] = v_page[i];
    uint32_t after = fine;
    __syncthreads();

    // Between two steps: the scores of the step to come, and the weights of the one done (none before the first).
    f32x16 s;
    half8_t hi[2], lo[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) hi[k][j] = lo[k][j] = (_Float16)0.f;
    constexpr int kSlots = KS + 2 * DB, kRing = 4;
    // The buffers of tiles t - 1, t, t + 1 and t + 2 (that of t + 2 is that of t - 1). Before the first tile there are no
    // weights, and any finite V will do.
    uint32_t past = 0, now = 0, ahead = 1, spare = 2;
    if (active) {
#pragma unroll
      for (int j = 0; j < 16; ++j) s[j] = 0.f;
#pragma unroll
      for (int i = 0; i < KS; ++i)
        s = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, lds_k[k_at + 2 * i]), q[i], s, 0, 0, 0);
    }
    // The way of the next tiles: half of the waves, one on each SIMD, go it before their steps and the others after
    // them, so that the matrix cores have work meanwhile.
    auto stage = [&](uint32_t tile) {
      kt.write(lds_k + spare * S::KTile);
      vt.write(lds_v + ahead * S::VTile);
      fetch_k(tile + 3, kt);
      fetch_v(tile + 2, pages, vt);
#pragma unroll
      for (int i = 0; i < S::VL; ++i) pages[i] = v_page[i];
    };
    for (uint32_t tile = first; tile < last; ++tile) {
      if (wave < NT / 128) stage(tile);
      if (active) {
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
          if (!(whole && cur == (1u << kBlocks) - 1)) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int32_t tok = 32 * tb + 8 * (j >> 2) + 4 * (int)h + (j & 3);
              const bool seen = (cur >> (2 * tb + (j >> 3)) & 1) && (int32_t)(tile * T) + tok < limit;
              s[j] = seen ? s[j] : -INFINITY;
            }
          }
          float top = s[0];
#pragma unroll
          for (int j = 1; j < 16; ++j) top = fmaxf(top, s[j]);
          top *= a.scale_log2;
          const bool moves = __any(top - ref > kHigh);   // ref -inf: moves for any score, not for none (NaN)
          float keep = 1.0f;
          if (moves) {
            top = fmaxf(top, __shfl_xor(top, 32));
            const float to = fmaxf(ref, top - kLow);
            keep = to == ref ? 1.0f : __builtin_amdgcn_exp2f(ref - to);
            ref = to;
            l *= keep;
          }
          const float off = ref == -INFINITY ? 0.f : -ref;   // no token so far: all weights are 2^-inf
          if (moves) rounded = __any(fabsf(off) >= kFused);
          if (rounded) {
#pragma unroll
            for (int j = 0; j < 16; ++j) s[j] *= a.scale_log2;
          }
          const float times = rounded ? 1.0f : a.scale_log2;
          // One step in slots, in the order written: a matrix instruction, the read of the operand of the one four
          // slots on, a part of the softmax. Past the last tile the scores are of what is there, and nobody reads them.
          const u32x4 *ks = lds_k + (tb + 1 < TB ? now : ahead) * S::KTile + k_at + 32 * ((tb + 1) % TB) * S::KRow;
          const u32x4 *vs = lds_v + (tb > 0 ? now : past) * S::VTile + v_at + 4 * ((tb + TB - 1) % TB);
          auto read = [&](int i) { return i < KS ? ks[2 * i] : vs[2 * ((i - KS) / DB) + 8 * ((i - KS) % DB) * S::VFour]; };
          u32x4 ring[kRing];
          f32x16 next;
#pragma unroll
          for (int j = 0; j < 16; ++j) next[j] = 0.f;
          u32x4 hi_now[2], lo_now[2];                // pairs of weights
          float y0 = 0.f;
#pragma unroll
          for (int i = 0; i < kRing; ++i) ring[i] = read(i);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < kSlots; ++i) {
            const half8_t x = __builtin_bit_cast(half8_t, ring[i % kRing]);
            if (i < KS) {
              next = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, q[i < KS ? i : 0], next, 0, 0, 0);
            } else {
              f32x16 &to = o[(i - KS) % DB];
              to = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, hi[(i - KS) / DB], to, 0, 0, 0);
              to = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, lo[(i - KS) / DB], to, 0, 0, 0);
            }
            if (i + kRing < kSlots) ring[i % kRing] = read(i + kRing);
#pragma unroll
            for (int j = 16 * i / kSlots; j < 16 * (i + 1) / kSlots; ++j) {
              float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j], times, off));
              asm volatile("" : "+v"(y));            // here and not where it is used
              l += y;
              asm volatile("" : "+v"(l));
              if ((j & 1) == 0) {
                y0 = y;
                continue;
              }
              const h2_t x2 = h2_t{(_Float16)y0, (_Float16)y};
              uint32_t bits = __builtin_bit_cast(uint32_t, x2);
              asm volatile("" : "+v"(bits));
              hi_now[j >> 3][(j & 7) >> 1] = bits;
              bits = __builtin_bit_cast(uint32_t, h2_t{(_Float16)(y0 - (float)x2[0]), (_Float16)(y - (float)x2[1])});
              asm volatile("" : "+v"(bits));
              lo_now[j >> 3][(j & 7) >> 1] = bits;
            }
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            hi[k] = __builtin_bit_cast(half8_t, hi_now[k]);
            lo[k] = __builtin_bit_cast(half8_t, lo_now[k]);
          }
          s = next;
          if (moves) {                               // the products so far belong to the reference of before
#pragma unroll
            for (int i = 0; i < DB; ++i) o[i] *= keep;
          }
        }
      }
      if (wave >= NT / 128) stage(tile);
      cur = next_fine;
      next_fine = after;
      after = fine;
      past = now;
      now = ahead;
      ahead = spare;
      spare = past;
      __syncthreads();
    }
    if (active) {                                    // the products of the last block
      const u32x4 *vs = lds_v + past * S::VTile + v_at + 4 * (TB - 1);
#pragma unroll
      for (int i = 0; i < 2 * DB; ++i) {
        const half8_t x = __builtin_bit_cast(half8_t, vs[2 * (i / DB) + 8 * (i % DB) * S::VFour]);
        o[i % DB] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, hi[i / DB], o[i % DB], 0, 0, 0);
        o[i % DB] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, lo[i / DB], o[i % DB], 0, 0, 0);
      }
    }
    l += __shfl_xor(l, 32);
    if (m < rows) {
      const int64_t r = part_row(a, p, w, kvh, m);
      if (bad && ref > -INFINITY) l = __builtin_nanf("");
#pragma unroll
      for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<f32x4 *>(a.parts.o + r * D + 32 * i + 8 * j + 4 * h) =
              f32x4{o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]};
      if (h == 0) *reinterpret_cast<f32x2 *>(a.parts.ml + 2 * r) = f32x2{ref, l};
    }
  }
}

// ---- the rows' own tokens ------------------------------------------------------------------------

// A wave's part of one head tile of one row's own tokens, or of a pack.
struct OwnSegment {
  uint32_t row_at, u0;       // where row b, and the segment, begin on the line
  uint32_t at, end;          // the wave's part of it; at in the lead: a step before the first, all masked
  int32_t b;
  Own seen;
  int32_t h0, rows;          // its first head, query rows
  int32_t m0;                // of a pack: its first query row
  bool pack;
  int64_t part;              // its first row of wave 0's partial results
  const uint8_t *kv;         // its KV head's part of page 0
  const int32_t *row;        // the row's entries
};

// The segment at unit `at` < end, at or after row b, which starts at row_at on the line.
__device__ __forceinline__ OwnSegment own_segment(const PrefixArgs &a, const Plan &plan, uint32_t at, uint32_t end, int32_t b,
                                                  uint32_t row_at) {
  OwnSegment s;
  GroupPlan p;
  uint32_t before;
  for (;;) {
    const int32_t g = uniform(plan.group_of(b, a.groups));
    p = GroupPlan{-1, 0, 0, 0, 0, 0};
    if (g >= 0)
      p = GroupPlan{uniform(plan.g[g].row0), uniform(plan.g[g].rows), uniform(plan.g[g].tokens), uniform(plan.g[g].row_tiles),
                    uniform(plan.g[g].units), 0};
    before = pack_units(a, p, b);
    s.seen = own_of(a, scalar_load(a.lens + b), p.tokens);
    const uint32_t n = before + s.seen.units * (uint32_t)a.head_tiles;
    if (at - row_at < n) break;
    row_at += n;
    ++b;
  }
  s.b = b;
  s.row_at = row_at;
  s.pack = at - row_at < before;
  int32_t kvh;
  if (s.pack) {
    s.seen = Own{0, p.tokens, 0, (uint32_t)p.units};
    const int32_t i = (int32_t)((at - row_at) / s.seen.units), n = packs_of(a, p);
    kvh = i / n;
    s.u0 = row_at + (uint32_t)i * s.seen.units;
    s.m0 = (i - kvh * n) * kHeads;
    s.h0 = kvh * a.group;
    s.rows = min(kHeads, p.rows * a.group - s.m0);
    s.part = pack_row(a, p, 0, kvh, s.m0);
  } else {
    const int32_t ht = (int32_t)((at - row_at - before) / s.seen.units);
    s.u0 = row_at + before + (uint32_t)ht * s.seen.units;
    kvh = ht / a.tiles_per_kv;
    const int32_t first_head = (ht - kvh * a.tiles_per_kv) * kHeads;
    s.m0 = 0;
    s.h0 = kvh * a.group + first_head;
    s.rows = min(kHeads, a.group - first_head);
    s.part = own_part(a, 0, b, ht);
  }
  s.end = min(end, s.u0 + s.seen.units);
  s.at = at < s.u0 + a.own_lead && s.u0 + a.own_lead < s.end ? s.u0 + a.own_lead : at;
  s.kv = a.pool + kvh * a.head_bytes;
  s.row = a.table + b * a.ld_table;
  return s;
}

// Wave v's part [at, end) of the line of own work, as the waves of paged_attn.hip take theirs: the loads are issued in
// one order everywhere, the next step's K while this one's softmax and products run, its V from then on.
template <int D, bool Q8>
__device__ __forceinline__ void own_work(const PrefixArgs &a, const Plan &plan, uint32_t v, uint32_t at, uint32_t end, int32_t from_b,
                                         uint32_t from_at) {
  using T = Tile<D, Q8>;
  constexpr int VJ = T::VJ;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const uint32_t vs_lane = 2 * ((((VJ * (uint32_t)c) / 32) << a.tok_shift) + 4 * g);   // the lane's V scales
  T t;
  half8_t q[1][T::KD];
  Block blk[2];
  int32_t page[2];                                   // of the step in t; below 0: none
  OwnSegment cur = own_segment(a, plan, at, end, from_b, from_at), fetch = cur;   // fetch: of the step in t, fetch.at that step
  auto token = [&](int st) { return fetch.seen.base + ((int32_t)(fetch.at - fetch.u0) - a.own_lead) * kTile + 16 * st; };
  auto look_up = [&]() {
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const int32_t tok = token(st);
      page[st] = fetch.at < end && tok >= 0 && tok < fetch.seen.len ? scalar_load(fetch.row + (tok >> a.tok_shift)) : -1;
    }
  };
  auto locate = [&]() {
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      if (page[st] >= a.num_pages) page[st] = -1;
      const uint32_t p = (uint32_t)max(page[st], 0);
      blk[st].r = make_rsrc(fetch.kv + (uint64_t)p * (uint64_t)a.page_bytes, page[st] < 0 ? 0u : (uint32_t)a.head_bytes);
      blk[st].place = (uint32_t)token(st) & ((1u << a.tok_shift) - 1);
    }
  };
  int32_t limit = 0;                                 // the tokens that the lane's query row sees; of the segment in q
  auto load_q = [&]() {                              // query rows past the segment's are its last: nobody reads their results
    int32_t m = fetch.m0 + min(c, fetch.rows - 1), b = fetch.b;
    if (fetch.pack) {
      const int32_t down = m / a.group;
      b += down;
      m -= down * a.group;
    }
    const uint16_t *from = a.q + b * a.ldq + (int64_t)(fetch.h0 + m) * D + 16 * g;
    limit = a.lens[b];
#pragma unroll
    for (int i = 0; i < T::KD; ++i) q[0][i] = *reinterpret_cast<const half8_t *>(from + 64 * (i >> 1) + 8 * (i & 1));
  };
  look_up();
  locate();
  load_q();
  __builtin_amdgcn_sched_barrier(0);
  load_k<D, Q8>(a, blk, t);
  __builtin_amdgcn_sched_barrier(0);
  load_v<D, Q8>(a, blk, vs_lane, t);
  __builtin_amdgcn_sched_barrier(0);
  bool more = true;
  while (more) {
    f32x4 o[1][VJ];
#pragma unroll
    for (int j = 0; j < VJ; ++j) o[0][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    float ref = -INFINITY, l = 0.f;
    bool inside = true, fresh = true, bad = false;   // the step in t is of segment cur, and its first; q is not finite
    const bool even = !cur.pack || !__any(limit < cur.seen.len);   // all see the same tokens
    const int32_t seen = limit;
    while (inside) {
      const int32_t t0 = token(0);
      const bool full = even && t0 >= cur.seen.first && t0 + kTile <= cur.seen.len && page[0] >= 0 && page[1] >= 0;
      uint32_t valid = 0xFF, sees = 0xFF;            // of the lane's eight tokens: those that are there, those its query row sees
      if (!full) {
        valid = sees = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int32_t tok = t0 + 16 * (i >> 2) + 4 * g + (i & 3);
          valid |= (uint32_t)(tok >= cur.seen.first && tok < cur.seen.len && page[i >> 2] >= 0) << i;
          sees |= (uint32_t)(tok < seen) << i;
        }
        sees &= valid;
      }
      more = fetch.at + 1 < end;
      if (++fetch.at == fetch.end) {
        inside = false;
        if (more) fetch = own_segment(a, plan, fetch.at, end, fetch.b, fetch.row_at);
      }
      look_up();
      if (fresh) {                                   // a head that is not finite is taken as zeros, and marked
        bad = nonfinite<T::KD>(q[0]);
        bad = __shfl_xor((int)bad, 16) || bad;
        bad = __shfl_xor((int)bad, 32) || bad;
#pragma unroll
        for (int i = 0; i < T::KD; ++i) {
          u32x4 x = __builtin_bit_cast(u32x4, q[0][i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = bad ? 0u : (x[j] & a.keep) ^ a.flip;
          q[0][i] = __builtin_bit_cast(half8_t, x);
        }
        fresh = false;
      }
      f32x4 x[2][1];
#pragma unroll
      for (int st = 0; st < 2; ++st) scores<D, Q8, 1>(t, st, q, x[st]);
      locate();
      if (more && !inside) load_q();
      load_k<D, Q8>(a, blk, t);
      float y[8], top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i >> 2][0][i & 3] * a.scale_log2;
      if (!full) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = (sees >> i & 1) ? y[i] : -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, y[i]);
      if (__any(top - ref > kHigh)) {                // ref -inf: moves for any score, not for none (NaN)
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float to = fmaxf(ref, top - kLow);
        const float keep = to == ref ? 1.0f : __builtin_amdgcn_exp2f(ref - to);
        ref = to;
        l *= keep;
#pragma unroll
        for (int j = 0; j < VJ; ++j) o[0][j] *= keep;
      }
      half8_t hi[1], lo[1];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_exp2f(y[i] - ref);
      if (!full) {                                   // masked places may hold anything: zero times NaN is NaN
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = (sees >> i & 1) ? y[i] : 0.f;
        if constexpr (Q8) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t m = (valid >> i & 1) ? 0u : (i & 1) ? 0xFFFF0000u : 0x0000FFFFu;
            t.vs[i >> 2][(i & 3) >> 1] &= ~m;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < T::VW; ++k) t.v[i][k] = (valid >> i & 1) ? t.v[i][k] : 0u;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        l += y[i];
        hi[0][i] = (_Float16)y[i];
        lo[0][i] = (_Float16)(y[i] - (float)hi[0][i]);
      }
      accumulate<D, Q8, 1>(t, hi, lo, o);
      load_v<D, Q8>(a, blk, vs_lane, t);
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (bad && ref > -INFINITY) l = __builtin_nanf("");
    if (c < cur.rows) {
      const int64_t r = cur.part + (int64_t)v * (cur.pack ? kHeads : a.own_rows) + c;
      const Parts &to = cur.pack ? a.packs : a.own_parts;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < VJ; j += 4)
          *reinterpret_cast<f32x4 *>(to.o + r * D + VJ * (4 * g + i) + j) = f32x4{o[0][j][i], o[0][j + 1][i], o[0][j + 2][i], o[0][j + 3][i]};
      if (g == 0) *reinterpret_cast<f32x2 *>(to.ml + 2 * r) = f32x2{ref, l};
    }
    cur = fetch;
  }
}

// ---- the launch ----------------------------------------------------------------------------------

template <int D, bool Q8>
__global__ __launch_bounds__(64 * prefix_waves(D), D == 256 ? 1 : 2) void prefix_kernel(PrefixArgs a) {
  constexpr int W = prefix_waves(D), NT = 64 * W, kRows = NT / 2, kPer = (kMaxGroups + 1) / NT;
  extern __shared__ __align__(16) u32x4 tiles[];
  __shared__ Plan plan;
  const int32_t tid = threadIdx.x, wave = uniform(tid >> 6);
  if constexpr (Q8) __builtin_amdgcn_s_setreg(1 | (23 << 6) | (0 << 11), 1);   // hwreg(MODE, 23, 1): FP16_OVFL

  // the groups' first rows: a thread's in order, then the largest of the threads before
  uint32_t lead[kPer], most = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int32_t g = kPer * tid + i, s = g <= a.groups ? a.starts[g] : 0;
    most = max(most, (uint32_t)min(max(s, 0), a.batch));
    lead[i] = most;
  }
  const uint32_t upto = scan_max(most);
  if ((tid & 63) == 63) plan.red[wave] = upto;
  __syncthreads();
  const uint32_t left = (uint32_t)__shfl_up((int)upto, 1);
  uint32_t before = (tid & 63) ? left : 0;
  for (int k = 0; k < wave; ++k) before = max(before, plan.red[k]);
#pragma unroll
  for (int i = 0; i < kPer; ++i) plan.lead[kPer * tid + i] = (int32_t)max(lead[i], before);
  __syncthreads();
  uint32_t units = 0, shared;
  GroupPlan mine[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int32_t g = kPer * tid + i;
    mine[i] = GroupPlan{0, 0, 0, 0, 0, units};
    if (g >= a.groups) continue;
    GroupPlan &p = mine[i];
    p.row0 = plan.lead[g];
    p.rows = plan.lead[g + 1] - p.row0;
    if (p.rows > 1) {
      const int32_t len = min(max(a.lens[p.row0], 0), a.max_len);
      p.tokens = min(max(a.prefix[g], 0), len) >> a.tok_shift << a.tok_shift;   // whole pages
    }
    const int32_t tiles = (p.tokens + tile_tokens(D) - 1) / tile_tokens(D);
    p.row_tiles = (int32_t)(((int64_t)p.rows * a.group + kRows - 1) / kRows);
    // Three ways, by what a KV head's tokens cost in steps of own work: once for up to 256 query rows, once for each
    // pack, or for each row apart, behind whose own tokens they lie. us with 24 groups of 2, 4 and 8 rows of 32 heads on
    // 8, 1600 tokens: together 66, 76, 78 (int8) and 69, 73, 77 (fp16), in packs 33, 36, 49 and 44, 46, 70, apart
    // 40, 65, 103 and 57, 98, 153; with 43 groups of 2 rows of 128 heads on 8, whose packs are a row each, 353 int8 tokens, 77,
    // 39 and 34. With few tiles for each workgroup in all, latency counts, which is least together: one group of
    // 2, 4, 8 and 16 rows of 32 heads after 1000 int8 tokens 15, 15, 16, 18, in packs 16, 17, 19, 22, apart 15, 18, 20, 21; after
    // 4000 tokens 19, 22, 23, 25 against 24, 26, 31, 30 and 22, 23, 25, 32.
    const int32_t steps = (p.tokens + kTile - 1) / kTile;
    const float together = a.tile_steps * p.row_tiles * (tiles + kLead), packs = (float)packs_of(a, p) * (steps + a.own_lead),
                apart = (float)p.rows * a.tiles_per_kv * steps;
    const bool few = (float)a.groups * a.kv_heads * (tiles + kLead) <= 2.5f * gridDim.x;
    p.units = p.tokens ? tiles + kLead : 0;
    if (!few && apart <= min(packs, together)) {
      p.tokens = 0;
      p.units = 0;
      p.row_tiles = 0;
    } else if (!few && packs <= together) {
      p.row_tiles = 0;
      p.units = p.tokens ? steps + a.own_lead : 0;
    }
    units += (uint32_t)(p.row_tiles * a.kv_heads) * (uint32_t)p.units;
  }
  units = scan_sum<W>(units, shared, plan);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int32_t g = kPer * tid + i;
    if (g >= a.groups) continue;
    mine[i].unit0 += units;
    plan.g[g] = mine[i];
    if (blockIdx.x == 0) a.plan[g] = mine[i];
  }
  __syncthreads();
  // the packs and the rows' own tokens, a run of rows for each thread
  const int32_t per = (a.batch + NT - 1) / NT, my_b = tid * per;
  uint32_t my_units = 0, own;
  for (int32_t b = my_b; b < min(my_b + per, a.batch); ++b) {
    const int32_t g = plan.group_of(b, a.groups);
    my_units += own_of(a, a.lens[b], g < 0 ? 0 : plan.g[g].tokens).units * (uint32_t)a.head_tiles + (g < 0 ? 0 : pack_units(a, plan.g[g], b));
  }
  uint32_t my_at = my_units;
  my_at = scan_sum<W>(my_at, own, plan);

  // Both kinds of work get workgroups by their cost.
  uint32_t workers = 0;
  if (shared) {
    const float x = (float)shared * a.shared_cost * W, y = (float)own;
    workers = (uint32_t)((float)gridDim.x * (x / (x + y)) + 0.5f);
    workers = min(max(workers, 1u), gridDim.x - (own ? 1u : 0u));
  }
  // A wave a unit is soonest done, but the join then has a part of each: 48 parts of a segment, more where a
  // wave gets four units. One row of two heads of 256 and 14394 tokens takes 11 and 41 us with 450 parts, 17 and 11 with
  // 112; four rows of 32 heads and 830 tokens, 27 units a segment, 11 and 5, and 16 and 4 with four units a wave.
  const uint32_t most_waves = min(a.own_most, max(own / 4, 48u * (uint32_t)(a.batch * a.head_tiles)));
  const Split split{shared, workers, own, min((gridDim.x - workers) * W, most_waves)};
  if (blockIdx.x == gridDim.x - 1) {
    if (tid == 0) *a.split = split;
    uint32_t u = my_at;
    for (int32_t b = my_b; b < min(my_b + per, a.batch); ++b) {
      const int32_t g = plan.group_of(b, a.groups);
      const uint32_t n = own_of(a, a.lens[b], g < 0 ? 0 : plan.g[g].tokens).units;
      a.rows[b] = RowPlan{g, u, n};
      u += n * (uint32_t)a.head_tiles + (g < 0 ? 0 : pack_units(a, plan.g[g], b));
    }
  }
  if (blockIdx.x < workers) {
    const Line line = make_line(shared, workers);
    if (blockIdx.x >= line.waves) return;
    shared_work<D, Q8>(a, plan, tiles, blockIdx.x, line.start(blockIdx.x), line.start(blockIdx.x + 1));
    return;
  }
  if (own == 0) return;
  const Line line = make_line(own, split.waves);
  const uint32_t v0 = (blockIdx.x - workers) * W;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    const uint32_t at = line.start(v0 + k);
    if (at >= my_at && at - my_at < my_units) {
      plan.found[0][k] = (uint32_t)my_b;
      plan.found[1][k] = my_at;
    }
  }
  __syncthreads();
  const uint32_t v = v0 + wave;
  if (v >= line.waves) return;
  own_work<D, Q8>(a, plan, v, line.start(v), line.start(v + 1), (int32_t)uniform(plan.found[0][wave]), uniform(plan.found[1][wave]));
}

// ---- the join ------------------------------------------------------------------------------------

// With few rows (query heads of the batch) the parts are many: most workgroups hold one of each row. The whole call then
// takes less with a workgroup a row than with a team of it; with many rows there are few parts, and it takes
// more. 256, 512, 768, 1024, 1280, 1536 and 2048 rows of 128 after 6000 int8 tokens: 33, 32, 31, 32, 35, 37, 42 us with a
// workgroup a row, 48, 37, 33, 35, 38, 38, 41 with a team.
constexpr int64_t kFewRows = 1024;

// D / 4 threads, a team, take every TEAMS-th part of a row's shared tokens and of its own; the teams of a row meet in LDS.
template <int D, int TEAMS>
__global__ __launch_bounds__(256) void prefix_join_kernel(PrefixArgs a) {
  constexpr uint32_t kLanes = D / 4, kAll = 256 / kLanes;
  static_assert(kAll % TEAMS == 0);
  __shared__ f32x4 team_o[256];
  __shared__ f32x2 team_ml[kAll];
  const uint32_t team = threadIdx.x / kLanes, turn = team % TEAMS, d = 4 * (threadIdx.x % kLanes);
  const int64_t all = (int64_t)a.batch * a.heads, at_row = (int64_t)blockIdx.x * (kAll / TEAMS) + team / TEAMS;
  const int64_t row = min(at_row, all - 1);
  const int32_t b = (int32_t)(row / a.heads), hd = (int32_t)(row - (int64_t)b * a.heads), kvh = hd / a.group;
  const Split split = *a.split;
  const RowPlan rp = a.rows[b];
  f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;
  auto add = [&](const f32x4 &x, const f32x2 &y) {
    const float now = fmaxf(m, y[0]);
    const float keep = m == now ? 1.0f : __builtin_amdgcn_exp2f(m - now);
    const float f = y[0] == now ? 1.0f : __builtin_amdgcn_exp2f(y[0] - now);
    o = o * keep + x * f;
    l = l * keep + y[1] * f;
    m = now;
  };
  auto join = [&](const Parts &parts, uint32_t first, uint32_t last, int64_t r, int32_t step) {   // at r + w * step
#pragma unroll 4
    for (uint32_t w = first + turn; w <= last; w += TEAMS) {
      const int64_t at = r + (int64_t)w * step;
      const f32x4 x = *reinterpret_cast<const f32x4 *>(parts.o + at * D + d);
      const f32x2 y = *reinterpret_cast<const f32x2 *>(parts.ml + 2 * at);
      add(x, y);
    }
  };
  const Line own = make_line(max(split.own, 1u), max(split.waves, 1u));
  uint32_t own_at = rp.unit0;
  if (rp.group >= 0) {
    constexpr int32_t kRows = 32 * prefix_waves(D);
    const GroupPlan p = a.plan[rp.group];
    const int32_t q = (b - p.row0) * a.group + hd - kvh * a.group;
    own_at += pack_units(a, p, b);
    if (p.row_tiles) {
      const Line line = make_line(split.shared, split.workers);
      const uint32_t u0 = p.unit0 + (uint32_t)(kvh * p.row_tiles + q / kRows) * (uint32_t)p.units;
      join(a.parts, line.holder(u0 + kLead), line.holder(u0 + (uint32_t)p.units - 1), part_row(a, p, 0, kvh, q), a.part_rows);
    } else {
      const uint32_t u0 = a.rows[p.row0].unit0 + (uint32_t)(kvh * packs_of(a, p) + q / kHeads) * (uint32_t)p.units;
      join(a.packs, own.holder(u0), own.holder(u0 + (uint32_t)p.units - 1), pack_row(a, p, 0, kvh, q), kHeads);
    }
  }
  if (rp.units) {
    const int32_t head = hd - kvh * a.group, ht = kvh * a.tiles_per_kv + head / kHeads;
    const uint32_t u0 = own_at + (uint32_t)ht * rp.units;
    join(a.own_parts, own.holder(u0), own.holder(u0 + rp.units - 1), own_part(a, 0, b, ht) + head % kHeads, a.own_rows);
  }
  if constexpr (TEAMS > 1) {
    team_o[threadIdx.x] = o;
    team_ml[team] = f32x2{m, l};                     // the same from all of a team
    __syncthreads();
    if (turn) return;
#pragma unroll
    for (int i = 1; i < TEAMS; ++i) add(team_o[threadIdx.x + i * kLanes], team_ml[team + i]);
  }
  if (at_row >= all) return;
  o *= l > 0.f ? 1.0f / l : l;                       // no token: 0; NaN sums stay NaN
  const int64_t to = b * a.ldo + (int64_t)hd * D + d;
  if (a.out_f32) {
    *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + to) = o;
  } else {
    half4_t y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = (_Float16)o[i];
    *reinterpret_cast<half4_t *>(static_cast<uint16_t *>(a.out) + to) = y;
  }
  if (d == 0 && a.lse) a.lse[row] = (m + __log2f(l)) * kLn2;
}

namespace {

bool prefix_misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

constexpr int64_t kResident = 256;                 // workgroups that are resident at once

// Where things lie in the workspace, in bytes, and the rows of the parts. A group's query rows of a KV head fill
// all their tiles but one, so there are at most `segments` segments of shared work. Their rows are batch * heads at most.
struct PrefixSpace {
  int64_t plan, rows, parts, parts_ml, packs, packs_ml, own_parts, own_ml, bytes;
  int32_t part_rows, own_rows, own_waves;
};

int prefix_space(const qg_kv_pool *pool, int64_t batch, int64_t heads, int64_t groups, int64_t max_len, int64_t max_tail,
                 PrefixSpace *s) {
  const int64_t dim = pool->head_dim, group = heads / pool->kv_heads, waves = prefix_waves((int)dim), rows = 32 * waves;
  const int64_t whole = batch * group / rows;        // rows are at most batch * group in all, a group has two rows or more
  const int64_t segments = pool->kv_heads * (whole + (groups < batch / 2 ? groups : batch / 2));
  const int64_t units = max_len ? segments * ((max_len + tile_tokens((int)dim) - 1) / tile_tokens((int)dim) + kLead) : 0;
  const int64_t head_tiles = pool->kv_heads * ((group + kHeads - 1) / kHeads);
  const int64_t lead = own_lead((int)dim, pool->kind == QG_KV_Q8);
  const auto steps = [lead](int64_t n) { return (n + kTile - 1) / kTile + 1 + lead; };   // from the middle of one on: one more
  const int64_t packs = pool->kv_heads * (batch * group / kHeads + (groups < batch / 2 ? groups : batch / 2));
  const int64_t pack_units = groups ? packs * steps(max_len) : 0;
  if (units > 0x7FFFFFFF || batch * head_tiles * steps(max_len) + pack_units > 0x7FFFFFFF) return QG_ERR_SHAPE;
  // what is past the prefix's last whole page is a row's own, too
  const int64_t tail = max_tail + pool->page_tokens < max_len ? max_tail + pool->page_tokens : max_len;
  // room for max_tail tokens of every row and for the packs, and for one row that shares nothing
  const int64_t own = std::max(batch * steps(tail), steps(max_len)) * head_tiles + pack_units, workers = units < kResident ? units : kResident;
  s->own_waves = (int32_t)(own < kResident * waves ? own : kResident * waves);
  s->part_rows = (int32_t)(batch * group < rows ? batch * group : rows);
  s->own_rows = (int32_t)(group < kHeads ? group : kHeads);
  const auto up = [](int64_t n) { return (n + 15) / 16 * 16; };
  s->plan = up(sizeof(Split));
  s->rows = s->plan + up(groups * (int64_t)sizeof(GroupPlan));
  s->parts = s->rows + up(batch * (int64_t)sizeof(RowPlan));
  const int64_t all = workers ? workers * s->part_rows + batch * heads : 0;
  const int64_t all_own = batch ? s->own_rows * (s->own_waves + batch * head_tiles) : 0;
  s->parts_ml = s->parts + 4 * dim * all;
  const int64_t all_packs = groups ? (int64_t)s->own_waves * kHeads + batch * heads : 0;
  s->packs = s->parts_ml + up(8 * all);
  s->packs_ml = s->packs + 4 * dim * all_packs;
  s->own_parts = s->packs_ml + up(8 * all_packs);
  s->own_ml = s->own_parts + 4 * dim * all_own;
  s->bytes = s->own_ml + up(8 * all_own);
  return QG_OK;
}

int prefix_shape(const qg_kv_pool *pool, int64_t batch, int64_t heads, int64_t groups, int64_t max_len, int64_t max_tail) {
  KvLayout L;
  if (int st = kv_pool_layout(pool, &L)) return st;
  if (batch < 0 || heads < 1 || heads % pool->kv_heads || heads > (1 << 22) || batch > (1 << 22) / heads) return QG_ERR_SHAPE;
  if (max_len < 0 || max_len > (1 << 30)) return QG_ERR_SHAPE;
  if (groups < 0 || groups > kMaxGroups || groups > batch || max_tail < 0 || max_tail > (1 << 30)) return QG_ERR_SHAPE;
  return QG_OK;
}

template <int D, bool Q8>
int launch_prefix(const PrefixArgs &a, hipStream_t s) {
  const dim3 grid(kResident), block(64 * prefix_waves(D));
  return launch(prefix_kernel<D, Q8>, grid, block, Shape<D, Q8>::kLds, s, a);
}

template <int D>
int launch_dim(const PrefixArgs &a, bool q8, hipStream_t s) {
  if (int st = q8 ? launch_prefix<D, true>(a, s) : launch_prefix<D, false>(a, s)) return st;
  constexpr int64_t kAll = 256 / (D / 4);
  const int64_t rows = (int64_t)a.batch * a.heads;
  if (rows <= kFewRows) return launch(prefix_join_kernel<D, kAll>, dim3((unsigned)rows), dim3(256), 0, s, a);
  return launch(prefix_join_kernel<D, 1>, dim3((unsigned)((rows + kAll - 1) / kAll)), dim3(256), 0, s, a);
}

}  // namespace

}  // namespace qg

using namespace qg;

extern "C" {

int qg_prefix_attention_bytes(const qg_kv_pool *pool, int64_t batch, int64_t heads, int64_t groups, int64_t max_len,
                              int64_t max_tail, int64_t *bytes) {
  if (!bytes) return QG_ERR_NULL;
  if (int st = prefix_shape(pool, batch, heads, groups, max_len, max_tail)) return st;
  PrefixSpace w;
  if (int st = prefix_space(pool, batch, heads, groups, max_len, max_tail, &w)) return st;
  *bytes = w.bytes;
  return QG_OK;
}

int qg_prefix_attention(const qg_kv_pool *pool, int64_t layer, const uint16_t *q, int64_t ldq, const int32_t *table,
                        int64_t ld_table, const int32_t *lens, const int32_t *starts, const int32_t *prefix, int64_t groups,
                        int64_t batch, int64_t heads, int64_t max_len, int64_t max_tail, float scale, void *out, int64_t ldo,
                        int out_f32, float *lse, void *workspace, int64_t workspace_bytes, void *stream) {
  if (int st = prefix_shape(pool, batch, heads, groups, max_len, max_tail)) return st;
  KvLayout L;
  if (int st = kv_pool_layout(pool, &L)) return st;
  const int64_t cols = heads * pool->head_dim;
  if (int st = kv_table_check(table, ld_table, batch, (max_len + pool->page_tokens - 1) / pool->page_tokens)) return st;
  if (layer < 0 || layer >= pool->layers || (batch > 1 && (ldq < cols || ldo < cols))) return QG_ERR_SHAPE;
  if (!std::isfinite(scale * kLog2e)) return QG_ERR_RANGE;   // scores are kept in units of log2
  if (batch == 0) return QG_OK;
  PrefixSpace w;
  if (int st = prefix_space(pool, batch, heads, groups, max_len, max_tail, &w)) return st;
  if (!q || !lens || !out || !workspace || !starts || (groups && !prefix)) return QG_ERR_NULL;
  if (prefix_misaligned(q, 16) || prefix_misaligned(out, 16) || prefix_misaligned(lens, 4) || prefix_misaligned(lse, 4) ||
      prefix_misaligned(starts, 4) || prefix_misaligned(prefix, 4) || prefix_misaligned(workspace, 16) ||
      (batch > 1 && (ldq % 8 || ldo % (out_f32 ? 4 : 8))))
    return QG_ERR_ALIGN;
  if (workspace_bytes < w.bytes) return QG_ERR_WORKSPACE;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  PrefixArgs a;
  a.pool = static_cast<const uint8_t *>(pool->pages) + (layer ? layer * pool->layer_stride : 0);
  a.page_bytes = L.page_bytes;
  a.head_bytes = L.head_bytes;
  a.v_off = L.v_off;
  a.ks_off = L.ks_off;
  a.vs_off = L.vs_off;
  a.num_pages = (int32_t)pool->num_pages;
  a.tok_shift = __builtin_ctz(pool->page_tokens);
  a.q = q;
  a.ldq = batch > 1 ? ldq : cols;
  a.table = table;
  a.ld_table = ld_table;
  a.lens = lens;
  a.starts = starts;
  a.prefix = prefix;
  a.groups = (int32_t)groups;
  a.batch = (int32_t)batch;
  a.heads = (int32_t)heads;
  a.kv_heads = pool->kv_heads;
  a.group = (int32_t)(heads / pool->kv_heads);
  a.tiles_per_kv = (a.group + kHeads - 1) / kHeads;
  a.head_tiles = a.tiles_per_kv * pool->kv_heads;
  a.max_len = (int32_t)max_len;
  a.part_rows = w.part_rows;
  a.own_rows = w.own_rows;
  a.own_most = (uint32_t)w.own_waves;
  a.own_lead = own_lead(pool->head_dim, pool->kind == QG_KV_Q8);
  // A tile of shared work takes 3.3 us (4.0 with heads of 64), with heads of 256, half the rows, 1.9. 128 rows of 32 heads of
  // 128 after 16384 int8 tokens: 102 us with 2.6 and 3.0 here, 103 to 104 with 2.3 and 3.5. Heads of 256, 79 rows of 48 on 4 in 3
  // groups after up to 6127 tokens: 70 with 2.1, 71 with 2.4, 82 with 2.8.
  const double tile_us = pool->head_dim == 256 ? 2.2 : 3.0;
  a.shared_cost = (float)(tile_us / own_step_us(pool->head_dim, pool->kind == QG_KV_Q8));
  // on all of the card: int8 at 30 KB a us for each workgroup, fp16 at HBM's 6 TB/s, which are 23
  a.tile_steps = (float)(tile_us / (32 * pool->head_dim * (pool->kind == QG_KV_Q8 ? 2.125 / 30e3 : 4.0 / 23e3)));
  const float size = std::fabs(scale * kLog2e);
  a.scale_log2 = size < FLT_MIN ? 1.0f : size;
  a.keep = size < FLT_MIN ? 0 : 0xFFFFFFFFu;
  a.flip = scale < 0 ? 0x80008000u : 0;
  a.out = out;
  a.ldo = batch > 1 ? ldo : cols;
  a.out_f32 = out_f32 != 0;
  a.lse = lse;
  a.split = reinterpret_cast<Split *>(ws);
  a.plan = reinterpret_cast<GroupPlan *>(ws + w.plan);
  a.rows = reinterpret_cast<RowPlan *>(ws + w.rows);
  a.parts = Parts{reinterpret_cast<float *>(ws + w.parts), reinterpret_cast<float *>(ws + w.parts_ml)};
  a.packs = Parts{reinterpret_cast<float *>(ws + w.packs), reinterpret_cast<float *>(ws + w.packs_ml)};
  a.own_parts = Parts{reinterpret_cast<float *>(ws + w.own_parts), reinterpret_cast<float *>(ws + w.own_ml)};
  const bool q8 = pool->kind == QG_KV_Q8;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  switch (pool->head_dim) {
    case 64: return launch_dim<64>(a, q8, s);
    case 128: return launch_dim<128>(a, q8, s);
    default: return launch_dim<256>(a, q8, s);
  }
}

}  // extern "C"
