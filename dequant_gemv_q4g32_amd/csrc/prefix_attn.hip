// Attention of one new token a sequence where neighbouring sequences share their first tokens, gfx950.
//
// A group's rows with the heads of a KV head are one block of queries against the shared tokens: unlike a
// single sequence's few heads, enough of them to keep the matrix cores busy. Three steps: the shared tokens,
// once a group, as a flash attention of up to 128 query rows a workgroup; what the rows do not share, by the
// one-token kernel (paged_attn.hip); the join of both.
//
// Shared tokens: S^T = K Q^T and O^T += V^T P^T on v_mfma_f32_32x32x16_f16. A wave takes 32 query rows, and
// a lane of S^T holds one row and 16 of 32 tokens, which is the operand that P^T has to be: the softmax stays in the
// registers. K and V go through LDS as fp16, decoded and V turned once for the four waves, in two buffers: while
// one tile is multiplied the next one is written and the one after that is on its way from memory.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/qgemv.h"
#include "attn_common.h"
#include "device_common.h"
#include "kv_pages.h"
#include "launch.h"

namespace qg {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kPrefixThreads = 256;
constexpr int kRows = 128;                         // query rows of a workgroup, 32 a wave
constexpr int kElems = 8192;                       // elements of K (and of V) a tile: 128 tokens of 64, 64 of 128, 32 of 256

// What the plan says of a group. Its query rows are rows * (heads of a KV head), in tiles of kRows a KV head; its
// tokens are `units` tiles. On the line its segments (KV head, row tile) follow each other, `units` each.
struct GroupPlan {
  int32_t row0, rows, tokens;
  int32_t row_tiles, units;
  uint32_t unit0, seg0;          // units and segments of the groups before
  int32_t pad;
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
  int32_t max_len, tile_tokens;
  float scale_log2;              // |scale| * log2(e)
  uint32_t flip;                 // sign bits of two fp16 numbers where scale is negative: turned in q
  void *out;
  int64_t ldo;
  int32_t out_f32;
  float *lse;
  uint32_t *total;               // workspace: units in all;
  GroupPlan *plan;
  int32_t *from, *group_of;      // of each row: the tokens that it shares, its group (-1: shares none)
  float *parts;                  // partial results: part w + s is worker w's of segment s
  float *tail, *tail_ml;         // what launch_attn_tail gives
};

// A part: [kRows][D] sums, then each row's reference and denominator.
__host__ __device__ __forceinline__ int64_t part_floats(int32_t dim) { return (int64_t)kRows * dim + 2 * kRows; }

constexpr int kPlanThreads = 1024;
constexpr int kPlanGroups = 4;                     // groups a thread
constexpr int64_t kMaxGroups = kPlanThreads * kPlanGroups - 1;

// Sum (or maximum) over the threads up to this one. lds: a value for each wave.
template <bool MAX>
__device__ __forceinline__ uint32_t plan_scan(uint32_t v, uint32_t *lds) {
  auto join = [](uint32_t a, uint32_t b) { return MAX ? max(a, b) : a + b; };
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t up = (uint32_t)__shfl_up((int)v, o);
    if ((int)(threadIdx.x & 63) >= o) v = join(v, up);
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 63) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  for (int w = 0; w < (int)(threadIdx.x >> 6); ++w) v = join(v, lds[w]);
  return v;
}

// One workgroup: the groups' rows and shared tokens, their places on the line, and each row's group.
__global__ __launch_bounds__(kPlanThreads) void prefix_plan_kernel(PrefixArgs a) {
  __shared__ uint32_t lds[kPlanThreads / 64];
  __shared__ int32_t lead[kPlanThreads * kPlanGroups];   // the groups' first rows, made to ascend, and the last one's end
  __shared__ int32_t shared[kPlanThreads * kPlanGroups];
  const int32_t g0 = kPlanGroups * (int32_t)threadIdx.x;
  uint32_t at[kPlanGroups], most = 0;
#pragma unroll
  for (int i = 0; i < kPlanGroups; ++i) {
    const int32_t s = g0 + i <= a.groups ? a.starts[g0 + i] : 0;
    most = max(most, (uint32_t)min(max(s, 0), a.batch));
    at[i] = most;
  }
  const uint32_t upto = plan_scan<true>(most, lds);
  // what is before this thread: the scan's value of the thread before
  __shared__ uint32_t edge[kPlanThreads];
  edge[threadIdx.x] = upto;
  __syncthreads();
  const uint32_t before = threadIdx.x ? edge[threadIdx.x - 1] : 0;
#pragma unroll
  for (int i = 0; i < kPlanGroups; ++i) lead[g0 + i] = (int32_t)max(at[i], before);
  __syncthreads();
  GroupPlan p[kPlanGroups];
  uint32_t units = 0, segs = 0;
#pragma unroll
  for (int i = 0; i < kPlanGroups; ++i) {
    const int32_t g = g0 + i;
    p[i] = GroupPlan{0, 0, 0, 0, 0, 0, 0, 0};
    if (g >= a.groups) continue;
    p[i].row0 = lead[g];
    p[i].rows = lead[g + 1] - lead[g];
    if (p[i].rows > 1) {
      const int32_t len = min(max(a.lens[p[i].row0], 0), a.max_len);
      p[i].tokens = min(max(a.prefix[g], 0), len) >> a.tok_shift << a.tok_shift;   // whole pages
    }
    p[i].units = (p[i].tokens + a.tile_tokens - 1) / a.tile_tokens;
    p[i].row_tiles = p[i].units ? (int32_t)(((int64_t)p[i].rows * a.group + kRows - 1) / kRows) : 0;
    p[i].unit0 = units;
    p[i].seg0 = segs;
    segs += (uint32_t)(p[i].row_tiles * a.kv_heads);
    units += (uint32_t)(p[i].row_tiles * a.kv_heads) * (uint32_t)p[i].units;
    shared[g] = p[i].tokens;
  }
  const uint32_t all_units = plan_scan<false>(units, lds), all_segs = plan_scan<false>(segs, lds);
#pragma unroll
  for (int i = 0; i < kPlanGroups; ++i) {
    if (g0 + i >= a.groups) continue;
    p[i].unit0 += all_units - units;
    p[i].seg0 += all_segs - segs;
    a.plan[g0 + i] = p[i];
  }
  if (threadIdx.x == kPlanThreads - 1) *a.total = all_units;
  __syncthreads();
  for (int32_t b = threadIdx.x; b < a.batch; b += kPlanThreads) {
    int32_t lo = 0, hi = a.groups + 1;               // the last g with lead[g] <= b is lo - 1
    while (lo < hi) {
      const int32_t mid = (lo + hi) >> 1;
      if (lead[mid] <= b) lo = mid + 1; else hi = mid;
    }
    const int32_t g = lo - 1;
    const int32_t n = g >= 0 && g < a.groups ? shared[g] : 0;
    a.from[b] = n;
    a.group_of[b] = n ? g : -1;
  }
}

// ---- the shared tokens ---------------------------------------------------------------------------

template <int D, bool Q8>
struct Shape {
  static constexpr int T = kElems / D;              // tokens of a tile
  static constexpr int TB = T / 32;                 // blocks of 32 of them
  static constexpr int KS = D / 16;                 // matrix steps along the head
  static constexpr int DB = D / 32;                 // blocks of 32 elements of the head
  static constexpr int KL = Q8 ? 2 : 4;             // 16-byte loads of K a thread
  static constexpr int KPer = Q8 ? D / 16 : D / 8;  // such loads a token
  static constexpr int VPer = D / 4;                // threads that share eight tokens of V, four elements each
};

// Places in LDS, in units of 16 bytes: neighbouring lanes read the same place of neighbouring rows, so a row's
// places are exchanged by its number to spread them over the banks. K is [T][D], V^T [D][T] with each
// place eight tokens of a lane's operand (16 s + 4 h + {0..3, 8..11} for step s, lane half h: place 2 s + h).
template <int D>
__device__ __forceinline__ uint32_t k_place(uint32_t tok, uint32_t c) { return tok * (D / 8) + (c ^ (tok & 7)); }
template <int D>
__device__ __forceinline__ uint32_t v_place(uint32_t d, uint32_t c) {
  constexpr uint32_t kPer = kElems / D / 8;          // places of a row: 16, 8, 4
  return d * kPer + (c ^ (kPer >= 8 ? (d ^ (d >> 3)) & 7 : ((d >> 1) ^ (d >> 3)) & 3));
}

// What a thread holds of the tile on its way.
template <int D, bool Q8>
struct Staged {
  u32x4 k[Shape<D, Q8>::KL];
  uint16_t ks[Shape<D, Q8>::KL];
  u32x2 v[8];                                        // int8: one dword each
  u32x2 vs[2];
  bool fine;                                         // the thread's tokens of V are in a page
};

template <int D, bool Q8>
__device__ __forceinline__ void write_tile(const Staged<D, Q8> &t, u32x4 *lds) {
  using S = Shape<D, Q8>;
  const uint32_t tid = threadIdx.x;
#pragma unroll
  for (int i = 0; i < S::KL; ++i) {
    const uint32_t id = tid + kPrefixThreads * i, tok = id / S::KPer, c = id % S::KPer;
    if constexpr (Q8) {
      const uint32_t d = t.ks[i] * 0x00010001u;
      u32x4 w[2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = t.k[i][j] ^ 0x80808080u;
        w[j >> 1][2 * (j & 1)] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, x, kSelLow), d);
        w[j >> 1][2 * (j & 1) + 1] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, x, kSelHigh), d);
      }
      lds[k_place<D>(tok, 2 * c)] = w[0];
      lds[k_place<D>(tok, 2 * c + 1)] = w[1];
    } else {
      lds[k_place<D>(tok, c)] = t.k[i];
    }
  }
  const uint32_t c = tid / S::VPer, d0 = 4 * (tid % S::VPer);
  u32x4 e[4];                                        // elements d0 .. d0 + 3, eight tokens each
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    if constexpr (Q8) {
      const uint32_t x0 = t.v[2 * p].x ^ 0x80808080u, x1 = t.v[2 * p + 1].x ^ 0x80808080u, d = t.vs[p >> 1][p & 1];
      const uint32_t a = __builtin_amdgcn_perm(x1, x0, 0x05010400u), b = __builtin_amdgcn_perm(x1, x0, 0x07030602u);
      e[0][p] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, a, kSelLow), d);
      e[1][p] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, a, kSelHigh), d);
      e[2][p] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, b, kSelLow), d);
      e[3][p] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, b, kSelHigh), d);
    } else {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        e[2 * w][p] = __builtin_amdgcn_perm(t.v[2 * p + 1][w], t.v[2 * p][w], 0x05040100u);
        e[2 * w + 1][p] = __builtin_amdgcn_perm(t.v[2 * p + 1][w], t.v[2 * p][w], 0x07060302u);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)                        // what is in no page may be anything, and zero times NaN is NaN
    lds[kElems / 8 + v_place<D>(d0 + i, c)] = t.fine ? e[i] : u32x4{0, 0, 0, 0};
}

// Workgroup `bid` takes its part of the line, segment by segment. PAIRS: weights as hi + lo fp16 pairs (22
// bits), for fp32 results; else as one fp16 number, whose rounding, 2^-12 of a weight on average and
// independent from token to token, is of the size of an fp16 result's own.
template <int D, bool Q8, bool PAIRS>
__global__ __launch_bounds__(kPrefixThreads, D == 256 ? 1 : 2) void prefix_kernel(PrefixArgs a) {
  using S = Shape<D, Q8>;
  constexpr int T = S::T, TB = S::TB, KS = S::KS, DB = S::DB, kBlocks = T / 16;
  extern __shared__ __align__(16) u32x4 tiles[];     // [2][K, V^T]
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), n = lane & 31, h = lane >> 5;
  if constexpr (Q8) __builtin_amdgcn_s_setreg(1 | (23 << 6) | (0 << 11), 1);   // hwreg(MODE, 23, 1): FP16_OVFL
  const uint32_t total = (uint32_t)scalar_load(reinterpret_cast<const int32_t *>(a.total));
  if (total == 0) return;
  const Line line = make_line(total, gridDim.x);
  const uint32_t w = blockIdx.x;
  if (w >= line.waves) return;
  const uint32_t end = line.start(w + 1);
  uint32_t at = line.start(w);
  int32_t g = 0;
  {                                                  // the last group with unit0 <= at that has units
    int32_t lo = 0, hi = a.groups;
    while (lo < hi) {
      const int32_t mid = (lo + hi) >> 1;
      if ((uint32_t)scalar_load(reinterpret_cast<const int32_t *>(&a.plan[mid].unit0)) <= at) lo = mid + 1; else hi = mid;
    }
    g = lo - 1;
  }
  while (at < end) {
    const int32_t *said = reinterpret_cast<const int32_t *>(a.plan + g);
    const GroupPlan p{scalar_load(said), scalar_load(said + 1), scalar_load(said + 2), scalar_load(said + 3), scalar_load(said + 4),
                      (uint32_t)scalar_load(said + 5), (uint32_t)scalar_load(said + 6), 0};
    const uint32_t segs = (uint32_t)(p.row_tiles * a.kv_heads);
    if (p.units == 0 || at - p.unit0 >= segs * (uint32_t)p.units) {
      ++g;
      continue;
    }
    const uint32_t seg = (at - p.unit0) / (uint32_t)p.units, first = at - p.unit0 - seg * (uint32_t)p.units;
    const uint32_t last = min(first + (end - at), (uint32_t)p.units);   // tiles [first, last) of the group's tokens
    const int32_t kvh = (int32_t)(seg / (uint32_t)p.row_tiles), rt = (int32_t)seg - kvh * p.row_tiles;
    const int32_t *row = a.table + (int64_t)p.row0 * a.ld_table;
    const uint8_t *kv = a.pool + kvh * a.head_bytes;
    // the lane's query row
    const int32_t m = rt * kRows + (int32_t)(32 * wave + n), rows = p.rows * a.group;
    const bool active = rt * kRows + (int32_t)(32 * wave) < rows;
    const int32_t b = p.row0 + min(m, rows - 1) / a.group, hd = kvh * a.group + min(m, rows - 1) % a.group;
    half8_t q[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      u32x4 x = *reinterpret_cast<const u32x4 *>(a.q + b * a.ldq + (int64_t)hd * D + 16 * i + 8 * h);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = m < rows ? x[j] ^ a.flip : 0u;
      q[i] = __builtin_bit_cast(half8_t, x);
    }
    const int32_t limit = min(max(a.lens[b], 0), p.tokens);   // the tokens that the row sees
    bool whole = !__any(limit < p.tokens);
    const bool bad = Q8 && nonfinite<KS>(q);
    f32x16 o[DB];
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
    float ref = -INFINITY, l = 0.f;

    // The pages of 64 blocks of 16 tokens, a block a lane; those of the next 64 on their way.
    auto pages_at = [&](uint32_t blk) {
      const int64_t tok = (int64_t)(blk + lane) * 16;
      int32_t page = -1;
      if (tok < p.tokens) page = row[tok >> a.tok_shift];
      return page;
    };
    uint32_t base = first * kBlocks;                 // of the blocks in ids
    int32_t ids = pages_at(base), ids_next = pages_at(base + 64);
    Staged<D, Q8> t;
    uint32_t fine = 0;                               // blocks of the tile in t that are in a page
    auto fetch = [&](uint32_t tile) {
      if (tile * kBlocks >= base + 64) {
        base += 64;
        ids = ids_next;
        ids_next = pages_at(base + 64);
      }
      const uint32_t b0 = tile * kBlocks - base;
      const bool ok = ids >= 0 && ids < a.num_pages;
      fine = (uint32_t)(__ballot(ok) >> b0) & ((1u << kBlocks) - 1);
      const int32_t safe = ok ? ids : 0;
      const uint32_t mask = (1u << a.tok_shift) - 1;
#pragma unroll
      for (int i = 0; i < S::KL; ++i) {
        const uint32_t id = tid + kPrefixThreads * i, r = id / S::KPer, c = id % S::KPer;
        const uint32_t place = (tile * T + r) & mask;
        const uint8_t *at = kv + (uint64_t)(uint32_t)__shfl(safe, (int)(b0 + r / 16)) * (uint64_t)a.page_bytes;
        t.k[i] = *reinterpret_cast<const u32x4 *>(at + place * (Q8 ? D : 2 * D) + 16 * c);
        if constexpr (Q8) t.ks[i] = *reinterpret_cast<const uint16_t *>(at + a.ks_off + 2 * (place * (D / 32) + c / 2));
      }
      const uint32_t c = tid / S::VPer, d0 = 4 * (tid % S::VPer), r = 16 * (c >> 1) + 4 * (c & 1);
      const uint32_t place = (tile * T + r) & mask;
      const uint8_t *at = kv + (uint64_t)(uint32_t)__shfl(safe, (int)(b0 + c / 2)) * (uint64_t)a.page_bytes;
      t.fine = (fine >> (c / 2)) & 1;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t tok = place + (j & 3) + 8 * (j >> 2);
        if constexpr (Q8) t.v[j].x = *reinterpret_cast<const uint32_t *>(at + a.v_off + tok * D + d0);
        else t.v[j] = *reinterpret_cast<const u32x2 *>(at + a.v_off + tok * (2 * D) + 2 * d0);
      }
      if constexpr (Q8) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          t.vs[j] = *reinterpret_cast<const u32x2 *>(at + a.vs_off + 2 * (((d0 / 32) << a.tok_shift) + place + 8 * j));
      }
    };

    fetch(first);
    __syncthreads();                                 // the segment before is done with LDS
    write_tile<D, Q8>(t, tiles);
    uint32_t cur = fine;
    if (first + 1 < last) fetch(first + 1);
    __syncthreads();
    for (uint32_t tile = first; tile < last; ++tile) {
      const u32x4 *lds = tiles + ((tile - first) & 1) * (kElems / 4);
      uint32_t next = 0;
      if (tile + 1 < last) {
        write_tile<D, Q8>(t, tiles + ((tile - first + 1) & 1) * (kElems / 4));
        next = fine;
        if (tile + 2 < last) fetch(tile + 2);
      }
      if (active) {
        f32x16 s[TB];
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
#pragma unroll
          for (int j = 0; j < 16; ++j) s[tb][j] = 0.f;
#pragma unroll
          for (int i = 0; i < KS; ++i)
            s[tb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, lds[k_place<D>(32 * tb + n, 2 * i + h)]), q[i],
                                                           s[tb], 0, 0, 0);
        }
        const bool full = whole && cur == (1u << kBlocks) - 1;
        auto seen = [&](int tb, int j) {             // the token of the lane's score j of block tb is seen by its row
          const int32_t tok = 32 * tb + 8 * (j >> 2) + 4 * (int)h + (j & 3);
          return (cur >> (2 * tb + (j >> 3)) & 1) && (int32_t)(tile * T) + tok < limit;
        };
        if (!full) {
#pragma unroll
          for (int tb = 0; tb < TB; ++tb)
#pragma unroll
            for (int j = 0; j < 16; ++j) s[tb][j] = seen(tb, j) ? s[tb][j] : -INFINITY;
        }
        float top = s[0][0];
#pragma unroll
        for (int tb = 0; tb < TB; ++tb)
#pragma unroll
          for (int j = 0; j < 16; ++j) top = fmaxf(top, s[tb][j]);
        top = top > -INFINITY ? top * a.scale_log2 : top;
        if (__any(top - ref > kHigh)) {              // ref -inf: moves for any score, not for none (NaN)
          top = fmaxf(top, __shfl_xor(top, 32));
          const float now = fmaxf(ref, top - kLow);
          const float keep = now == ref ? 1.0f : __builtin_amdgcn_exp2f(ref - now);
          ref = now;
          l *= keep;
#pragma unroll
          for (int i = 0; i < DB; ++i) o[i] *= keep;
        }
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
          float y[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            y[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[tb][j], a.scale_log2, -ref));
            if (!full) y[j] = seen(tb, j) ? y[j] : 0.f;
            l += y[j];
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            half8_t hi, lo;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              hi[j] = (_Float16)y[8 * k + j];
              if constexpr (PAIRS) lo[j] = (_Float16)(y[8 * k + j] - (float)hi[j]);
            }
#pragma unroll
            for (int i = 0; i < DB; ++i) {
              const half8_t v = __builtin_bit_cast(half8_t, lds[kElems / 8 + v_place<D>(32 * i + n, 2 * (2 * tb + k) + h)]);
              o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, hi, o[i], 0, 0, 0);
              if constexpr (PAIRS) o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, lo, o[i], 0, 0, 0);
            }
          }
        }
      }
      cur = next;
      __syncthreads();
    }
    if (active && m < rows) {
      float *part = a.parts + (int64_t)(w + p.seg0 + seg) * part_floats(D);
      const int r = 32 * (int)wave + (int)n;
      if (bad && ref > -INFINITY) l = __builtin_nanf("");
#pragma unroll
      for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<f32x4 *>(part + r * D + 32 * i + 8 * j + 4 * h) = f32x4{o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]};
    }
    l += __shfl_xor(l, 32);
    if (active && m < rows && h == 0) {
      float *part = a.parts + (int64_t)(w + p.seg0 + seg) * part_floats(D);
      *reinterpret_cast<f32x2 *>(part + kRows * D + 2 * (32 * wave + n)) = f32x2{ref, l};
    }
    at += last - first;
  }
}

// ---- the join ------------------------------------------------------------------------------------

// D / 4 threads a row of the output: its tail's sums and the parts of its shared tokens.
template <int D>
__global__ __launch_bounds__(256) void prefix_join_kernel(PrefixArgs a, uint32_t workers) {
  constexpr uint32_t kLanes = D / 4;
  const int64_t row = (int64_t)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
  const uint32_t d = 4 * (threadIdx.x % kLanes);
  if (row >= (int64_t)a.batch * a.heads) return;
  const int32_t b = (int32_t)(row / a.heads), hd = (int32_t)(row - (int64_t)b * a.heads);
  f32x4 o = *reinterpret_cast<const f32x4 *>(a.tail + row * D + d);
  const f32x2 ml = *reinterpret_cast<const f32x2 *>(a.tail_ml + 2 * row);
  float m = ml[0], l = ml[1];
  const int32_t g = a.group_of[b];
  if (g >= 0) {
    const GroupPlan p = a.plan[g];
    const Line line = make_line(*a.total, workers);
    const int32_t kvh = hd / a.group, q = (b - p.row0) * a.group + hd - kvh * a.group, rt = q / kRows, r = q - rt * kRows;
    const uint32_t seg = (uint32_t)(kvh * p.row_tiles + rt), u0 = p.unit0 + seg * (uint32_t)p.units;
    const uint32_t w0 = line.holder(u0), w1 = line.holder(u0 + (uint32_t)p.units - 1);
#pragma unroll 4
    for (uint32_t w = w0; w <= w1; ++w) {
      const float *part = a.parts + (int64_t)(w + p.seg0 + seg) * part_floats(D);
      const f32x4 x = *reinterpret_cast<const f32x4 *>(part + r * D + d);
      const f32x2 y = *reinterpret_cast<const f32x2 *>(part + kRows * D + 2 * r);
      const float now = fmaxf(m, y[0]);
      const float keep = m == now ? 1.0f : __builtin_amdgcn_exp2f(m - now);
      const float f = y[0] == now ? 1.0f : __builtin_amdgcn_exp2f(y[0] - now);
      o = o * keep + x * f;
      l = l * keep + y[1] * f;
      m = now;
    }
  }
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

// Workgroups that are resident at once.
int64_t prefix_resident(int64_t dim) { return dim == 256 ? 256 : 512; }

// Where things lie in the workspace, in bytes, and what the host can say of the line: at most `segments` segments
// (a group's query rows of a KV head fill all their tiles but one) of at most `units` in all.
struct PrefixSpace {
  int64_t plan, from, group_of, tail, tail_ml, tail_ws, parts, bytes;
  int64_t segments, units, workers;
};

int prefix_space(const qg_kv_pool *pool, int64_t batch, int64_t heads, int64_t groups, int64_t max_len, int64_t max_tail,
                 PrefixSpace *s) {
  const int64_t dim = pool->head_dim, group = heads / pool->kv_heads, tile = kElems / dim;
  const int64_t whole = batch * group / kRows;       // rows are at most batch * group in all, a group has two rows or more
  s->segments = pool->kv_heads * (whole + (groups < batch / 2 ? groups : batch / 2));
  s->units = s->segments * ((max_len + tile - 1) / tile);
  if (s->units > 0x7FFFFFFF) return QG_ERR_SHAPE;
  const int64_t most = prefix_resident(dim);
  s->workers = s->units < most ? s->units : most;
  const auto up = [](int64_t n) { return (n + 15) / 16 * 16; };
  s->plan = 16;
  s->from = s->plan + groups * (int64_t)sizeof(GroupPlan);
  s->group_of = s->from + up(4 * batch);
  s->tail = s->group_of + up(4 * batch);
  s->tail_ml = s->tail + 4 * batch * heads * dim;
  s->tail_ws = s->tail_ml + up(8 * batch * heads);
  s->parts = s->tail_ws + up(attn_tail_bytes(pool, batch, heads, max_tail));
  s->bytes = s->parts + 4 * part_floats((int32_t)dim) * (s->workers ? s->workers + s->segments - 1 : 0);
  return QG_OK;
}

// The tail's likely length: what is past the prefix's last whole page too.
int64_t prefix_tail(const qg_kv_pool *pool, int64_t max_len, int64_t max_tail) {
  const int64_t n = max_tail + pool->page_tokens;
  return n < max_len ? n : max_len;
}

int prefix_shape(const qg_kv_pool *pool, int64_t batch, int64_t heads, int64_t groups, int64_t max_len, int64_t max_tail) {
  if (int st = attn_shape_check(pool, batch, heads, max_len)) return st;
  if (groups < 0 || groups > kMaxGroups || groups > batch || max_tail < 0 || max_tail > (1 << 30)) return QG_ERR_SHAPE;
  return QG_OK;
}

template <int D, bool Q8>
int launch_prefix(const PrefixArgs &a, int64_t workers, hipStream_t s) {
  constexpr size_t kLds = 2 * 2 * kElems * sizeof(uint16_t);
  const dim3 grid((unsigned)workers), block(kPrefixThreads);
  if (a.out_f32) return launch(prefix_kernel<D, Q8, true>, grid, block, kLds, s, a);
  return launch(prefix_kernel<D, Q8, false>, grid, block, kLds, s, a);
}

template <int D>
int launch_join(const PrefixArgs &a, int64_t workers, hipStream_t s) {
  constexpr int64_t kPer = 256 / (D / 4);
  const int64_t rows = (int64_t)a.batch * a.heads;
  return launch(prefix_join_kernel<D>, dim3((unsigned)((rows + kPer - 1) / kPer)), dim3(256), 0, s, a, (uint32_t)workers);
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
  if (int st = prefix_space(pool, batch, heads, groups, max_len, prefix_tail(pool, max_len, max_tail), &w)) return st;
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
  const int64_t tail = prefix_tail(pool, max_len, max_tail);
  PrefixSpace w;
  if (int st = prefix_space(pool, batch, heads, groups, max_len, tail, &w)) return st;
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
  a.max_len = (int32_t)max_len;
  a.tile_tokens = kElems / pool->head_dim;
  a.scale_log2 = std::fabs(scale * kLog2e);
  a.flip = std::signbit(scale) ? 0x80008000u : 0;
  a.out = out;
  a.ldo = batch > 1 ? ldo : cols;
  a.out_f32 = out_f32 != 0;
  a.lse = lse;
  a.total = reinterpret_cast<uint32_t *>(ws);
  a.plan = reinterpret_cast<GroupPlan *>(ws + w.plan);
  a.from = reinterpret_cast<int32_t *>(ws + w.from);
  a.group_of = reinterpret_cast<int32_t *>(ws + w.group_of);
  a.tail = reinterpret_cast<float *>(ws + w.tail);
  a.tail_ml = reinterpret_cast<float *>(ws + w.tail_ml);
  a.parts = reinterpret_cast<float *>(ws + w.parts);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (int st = launch(prefix_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a)) return st;
  const bool q8 = pool->kind == QG_KV_Q8;
  if (w.workers) {
    int st;
    switch (pool->head_dim) {
      case 64: st = q8 ? launch_prefix<64, true>(a, w.workers, s) : launch_prefix<64, false>(a, w.workers, s); break;
      case 128: st = q8 ? launch_prefix<128, true>(a, w.workers, s) : launch_prefix<128, false>(a, w.workers, s); break;
      default: st = q8 ? launch_prefix<256, true>(a, w.workers, s) : launch_prefix<256, false>(a, w.workers, s);
    }
    if (st) return st;
  }
  if (int st = launch_attn_tail(pool, L, layer, q, ldq, table, ld_table, lens, a.from, batch, heads, max_len, tail,
                                scale * kLog2e, a.tail, a.tail_ml, ws + w.tail_ws, stream))
    return st;
  switch (pool->head_dim) {
    case 64: return launch_join<64>(a, w.workers, s);
    case 128: return launch_join<128>(a, w.workers, s);
    default: return launch_join<256>(a, w.workers, s);
  }
}

}  // extern "C"
