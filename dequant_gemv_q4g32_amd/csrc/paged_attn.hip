// Attention of one new token a sequence over a paged KV cache, gfx950.
//
// For a sequence b, a head h of KV head g and its cached tokens j:
//   s_j = scale <q, K_j>,  out = sum_j e^(s_j) V_j / sum_j e^(s_j)
// in one pass over K and V. With powers of two (s in units of log2) and a running reference `ref`
// per head, a wave keeps o = sum 2^(s_j - ref) V_j and l = sum 2^(s_j - ref); moving ref scales both
// by 2^(old - new), and two such results join by scaling to the larger ref.
//
// Work of a wave: up to 16 or 32 heads of one KV head (a head tile) against 32 tokens a step, two
// blocks of 16. S^T = K Q^T and O^T += V^T P^T run on v_mfma_f32_16x16x32_f16 with fp32 sums. S^T's lanes
// hold one head and four tokens each, which is the layout the weights P^T need as the next
// product's operand, so the softmax never leaves the registers: no shuffle but the largest score's,
// and that only when ref moves. int8 K and V are decoded to fp16 in registers; the row-major V is
// turned by byte permutes on the way (8 tokens of one element are an operand). The weights meet V
// as hi + lo fp16 pairs, 22 bits.
//
// What bounds it: each cached byte is read once, so HBM, and for int8 also instruction issue (about
// 372 vector and 130 scalar instructions a step of 8.7 KB; a wave alone needs 1.3 us for it). The
// next step's K is on its way while the softmax and the products with V run, its V from then on.
// Measured (GPU time; a plain stream of reads reaches 6.8 TB/s here): 64 sequences of 8192 tokens,
// 64 heads on 8 of 128: fp16 320 us = 6.7 TB/s, int8 186 us = 6.1 TB/s; one of 131072 tokens, int8,
// 54 us = 5.3 TB/s; 32 of up to 8192, int8, 47 us = 4.9 TB/s; 48 of up to 6007 with one KV head of
// 256, int8, 27 us; one of 1000 tokens 9.5 us, of 100 tokens 6 us (a launch and four dependent
// memory latencies: length, page, K, and the first step). HBM reads are the algorithm's bytes.
// The scalar registers do not hold all of a wave's places: 34 to 61 spill to vector lanes, none in the
// blocks with matrix instructions.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/qgemv.h"
#include "attn_common.h"
#include "device_common.h"
#include "kv_pages.h"
#include "launch.h"

namespace qg {

struct AttnArgs {
  const uint8_t *pool;           // the layer's first page
  int64_t page_bytes, head_bytes;
  int32_t v_off, ks_off, vs_off;
  int32_t num_pages, tok_shift;
  const uint16_t *q;
  int64_t ldq;
  const int32_t *table;
  int64_t ld_table;
  const int32_t *lens;
  int32_t batch, heads, group;   // group = heads / kv_heads
  int32_t tile_heads;            // heads of a head tile: 16, or 32 where a KV head has more than 16
  int32_t tiles_per_kv, head_tiles;   // head tiles of a KV head, and of all of them
  int32_t rows;                  // heads of a tile that a partial result has room for
  int32_t max_len, window;
  float scale_log2;              // scale * log2(e)
  void *out;
  int64_t ldo;
  int32_t out_f32;
  float *lse;
  uint32_t *starts;              // workspace: where each sequence starts on the line, and its end;
  const int32_t *starts_in;      // the same for reading
  float *slots;                  // workspace: two parts a wave
};

constexpr int kWaves = 4;                          // waves of a workgroup
constexpr int kThreads = 64 * kWaves;

// What of sequence b is seen: tokens [first, len), in tiles from base = first rounded down.
// On the line (below) a head tile of few tiles counts one unit more: its start costs a wave about as
// much as half a tile, which a wave with many short sequences would be late by (32 sequences of up to
// 8192 tokens, some of none or one: 56 us without the unit, 51 with it).
struct Seen {
  int32_t first, len, base, tiles;
  uint32_t lead, units;
};
constexpr int32_t kShort = 16;                       // tiles below which a head tile has that unit
template <bool WHOLE>
__device__ __forceinline__ Seen seen_of(const AttnArgs &a, int32_t raw) {
  Seen s;
  s.len = min(max(raw, 0), a.max_len);
  s.first = a.window ? max(0, s.len - a.window) : 0;
  s.base = s.first & ~(kTile - 1);
  s.tiles = max(1, (s.len - s.base + kTile - 1) / kTile);      // an empty sequence still gets its zeros written
  s.lead = !WHOLE && s.tiles < kShort ? 1 : 0;
  s.units = (uint32_t)s.tiles + s.lead;
  return s;
}

// The split. The units of all sequences and head tiles, sequence by sequence and head tile by head
// tile, are one line of `total` units (below 2^31), of which wave v of `waves` takes the v-th part:
// quota units, and one more if v < extra. Every wave finds its place on the line from lens alone.
// A head tile [u0, u1) of the line is thus covered by neighbouring waves. A wave that goes on
// past u1 (its range ends beyond) has left the head tile behind as a part of its own; the waves whose
// range ends within the head tile end on it, and those of one workgroup join their parts. So the
// parts of a head tile are: one for each workgroup with such waves (named by the first of them,
// the leader), and one for a wave that goes on past u1. A workgroup for each head tile instead would
// put one long sequence on as many CUs as it has KV heads, and wait for the longest of ragged ones.

// Sum of `v` over the threads before this one; total: over all. lds: a value for each wave.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *lds, uint32_t &total) {
  const uint32_t scan = wave_scan(v);
  if ((threadIdx.x & 63) == 63) lds[threadIdx.x >> 6] = scan;
  __syncthreads();
  uint32_t before = 0, all = 0;
  for (int w = 0; w < kWaves; ++w) {
    const uint32_t t = lds[w];
    before += w < (int)(threadIdx.x >> 6) ? t : 0;
    all += t;
  }
  total = uniform(all);
  return before + scan - v;
}

// A part in the workspace: [rows][D] sums, then each row's reference and denominator, in whole 16
// bytes. Slot 2 v: what wave v left behind; slot 2 v + 1: what the waves of its workgroup from v on
// ended on.
__host__ __device__ __forceinline__ int32_t slot_floats(int32_t rows, int32_t dim) {
  return rows * dim + (2 * rows + 3) / 4 * 4;
}
__device__ __forceinline__ float *slot_of(const AttnArgs &a, uint32_t slot, int D) {
  return a.slots + (int64_t)slot * slot_floats(a.rows, D);
}

// A wave's part of one head tile of one sequence.
struct Segment {
  uint32_t u0, u1;           // the head tile on the line
  uint32_t tile0;            // where its tiles start
  uint32_t at, end;          // the wave's part of it; at < tile0: a tile before the first, all masked
  bool from_start;           // the wave's part starts with the head tile
  int32_t b;
  int32_t first, len, base;  // what of the sequence is seen
  int32_t ht, h0, rows;      // head tile of the sequence, its first head, heads
  const uint8_t *kv;         // its KV head's part of page 0
  const int32_t *row;        // the sequence's row of the table
};

// The segment at unit `at` < end of the line, at or after sequence b of `len` tokens, which starts
// at seq_at.
template <bool WHOLE>
__device__ __forceinline__ Segment segment_at(const AttnArgs &a, uint32_t at, uint32_t end, int32_t b, uint32_t seq_at,
                                              int32_t len) {
  Segment g;
  Seen s = seen_of<WHOLE>(a, len);
  while (at - seq_at >= s.units * a.head_tiles) {
    seq_at += s.units * a.head_tiles;
    ++b;
    s = seen_of<WHOLE>(a, scalar_load(a.lens + b));
  }
  g.ht = (int32_t)((at - seq_at) / s.units);
  g.u0 = seq_at + (uint32_t)g.ht * s.units;
  g.u1 = g.u0 + s.units;
  g.tile0 = g.u0 + s.lead;
  g.end = min(end, g.u1);
  g.from_start = at == g.u0;
  g.at = at < g.tile0 && g.tile0 < g.end ? g.tile0 : at;
  g.b = b;
  g.first = s.first;
  g.len = s.len;
  g.base = s.base;
  const int32_t kvh = g.ht / a.tiles_per_kv, first_head = (g.ht - kvh * a.tiles_per_kv) * a.tile_heads;
  g.h0 = kvh * a.group + first_head;
  g.rows = min(a.tile_heads, a.group - first_head);
  g.kv = a.pool + kvh * a.head_bytes;
  g.row = a.table + b * a.ld_table;
  return g;
}

// Output rows of a whole head tile, or a part of one: 4 elements at d of row r.
template <int D>
__device__ __forceinline__ void store_result(const AttnArgs &a, int32_t b, int32_t h0, float *slot, int r, int d, f32x4 o,
                                             float m, float l) {
  if (slot) {
    *reinterpret_cast<f32x4 *>(slot + r * D + d) = o;
    if (d == 0) *reinterpret_cast<f32x2 *>(slot + a.rows * D + 2 * r) = f32x2{m, l};
    return;
  }
  const int32_t h = h0 + r;
  const int64_t at = b * a.ldo + (int64_t)h * D + d;
  const float inv = l > 0.f ? 1.0f / l : l;          // no token: 0; NaN sums stay NaN
  o *= inv;
  if (a.out_f32) {
    *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + at) = o;
  } else {
    half4_t y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = (_Float16)o[i];
    *reinterpret_cast<half4_t *>(static_cast<uint16_t *>(a.out) + at) = y;
  }
  if (d == 0 && a.lse) a.lse[(int64_t)b * a.heads + h] = (m + __log2f(l)) * kLn2;
}

// WHOLE: workgroup (sequence, head tile) of one to four waves takes that head tile, its waves a share
// each, and there is nothing to join afterwards. Else the workgroups' waves take the parts of the line.
template <int D, bool Q8, bool WHOLE, int HT>
__global__ __launch_bounds__(kThreads, D == 64 ? (HT == 1 ? 4 : 3) : D == 128 ? 2 : 1) void attn_kernel(AttnArgs a) {
  using T = Tile<D, Q8>;
  constexpr int VJ = T::VJ;
  constexpr int kPad = D + 4;                        // LDS rows of neighbouring heads start in other banks
  extern __shared__ __align__(16) float sums[];      // [kWaves][rows][kPad], rows = heads of a tile; in 16-byte accesses
  __shared__ uint32_t scan[kWaves], found[3][kWaves];
  __shared__ float wave_m[kWaves][16 * HT], wave_l[kWaves][16 * HT], run_m[kWaves][16 * HT];
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), c = lane & 15, g = lane >> 4;
  if constexpr (Q8) __builtin_amdgcn_s_setreg(1 | (23 << 6) | (0 << 11), 1);   // hwreg(MODE, 23, 1): FP16_OVFL
  const uint32_t vs_lane = 2 * ((((VJ * (uint32_t)c) / 32) << a.tok_shift) + 4 * g);   // the lane's V scales

  // this workgroup's waves on the line
  Line line;
  uint32_t v0, from_b, from_at;                      // first wave; a sequence at or before this wave's part, its start
  int32_t from_len;                                  // and its length
  if constexpr (WHOLE) {
    from_b = blockIdx.x / a.head_tiles;
    from_len = scalar_load(a.lens + from_b);
    const uint32_t tiles = seen_of<true>(a, from_len).units;
    line = make_line(tiles, blockDim.x / 64);
    line.first = (blockIdx.x - from_b * a.head_tiles) * tiles;
    from_at = 0;
    v0 = 0;
  } else {
    // Every wave for itself where the batch fits its lanes (no LDS and no barrier in the way of the
    // first loads), else a share of the batch for each thread of the workgroup.
    const bool one = a.batch <= 64;
    const int32_t per = one ? 1 : (a.batch + kThreads - 1) / kThreads, my_b = (one ? lane : (int32_t)threadIdx.x) * per;
    uint32_t mine = 0;
    int32_t my_len = 0;                              // of sequence my_b
    for (int32_t i = 0; i < per; ++i)
      if (my_b + i < a.batch) {
        const int32_t len = a.lens[my_b + i];
        if (i == 0) my_len = len;
        mine += seen_of<false>(a, len).units * a.head_tiles;
      }
    uint32_t total, before;
    if (one) {
      const uint32_t scan = wave_scan(mine);
      before = scan - mine;
      total = __builtin_amdgcn_readlane(scan, 63);
    } else {
      before = block_scan(mine, scan, total);
    }
    if (blockIdx.x == 0) {                           // for the join
      uint32_t at = before;
      for (int32_t i = 0; i < per; ++i)
        if (my_b + i < a.batch) {
          a.starts[my_b + i] = at;
          at += seen_of<false>(a, a.lens[my_b + i]).units * a.head_tiles;
        }
      if (threadIdx.x == 0) a.starts[a.batch] = total;
    }
    line = make_line(total, gridDim.x * kWaves);
    v0 = blockIdx.x * kWaves;
    if (v0 >= line.waves) return;
    if (one) {
      const uint32_t at = line.start(v0 + wave);
      const uint64_t here = __ballot(at >= before && at - before < mine);
      const int32_t i = here ? __builtin_ctzll(here) : 0;    // none: a wave without a part
      from_b = i;
      from_at = __builtin_amdgcn_readlane(before, i);
      from_len = __builtin_amdgcn_readlane(my_len, i);
    } else {
#pragma unroll
      for (int k = 0; k < kWaves; ++k) {
        const uint32_t at = line.start(v0 + k);
        if (at >= before && at - before < mine) {
          found[0][k] = (uint32_t)my_b;
          found[1][k] = before;
          found[2][k] = (uint32_t)my_len;
        }
      }
      __syncthreads();
      from_b = uniform(found[0][wave]);
      from_at = uniform(found[1][wave]);
      from_len = (int32_t)uniform(found[2][wave]);
    }
  }
  const uint32_t v = v0 + wave, live = min((uint32_t)kWaves, line.waves - v0);   // waves with a part of the line

  f32x4 o[HT][VJ];
  float ref[HT], l[HT];
  Segment cur;
  if ((uint32_t)wave < live) {
    const uint32_t end = line.start(v + 1);
    T t;
    half8_t q[HT][T::KD];
    Block blk[2];
    int32_t page[2];                                 // of the tile in t; below 0: none
    cur = segment_at<WHOLE>(a, line.start(v), end, (int32_t)from_b, from_at, from_len);
    Segment fetch = cur;                             // the segment of the tile in t, fetch.at that tile
    auto token = [&](int st) { return fetch.base + (int32_t)(fetch.at - fetch.tile0) * kTile + 16 * st; };
    auto look_up = [&]() {
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const int32_t tok = token(st);
        page[st] = fetch.at < end && tok >= 0 && tok < fetch.len ? scalar_load(fetch.row + (tok >> a.tok_shift)) : -1;
      }
    };
    auto locate = [&]() {
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        if (page[st] >= a.num_pages) page[st] = -1;
        const uint32_t p = (uint32_t)max(page[st], 0);
        blk[st].r = make_rsrc(fetch.kv + (uint64_t)p * (uint32_t)a.page_bytes, page[st] < 0 ? 0u : (uint32_t)a.head_bytes);
        blk[st].place = (uint32_t)token(st) & ((1u << a.tok_shift) - 1);
      }
    };
    auto load_q = [&]() {                            // heads past the tile's read as zeros: their lanes' own offsets are out of range
      const uint16_t *at = a.q + uniform(fetch.b) * a.ldq + (int64_t)uniform(fetch.h0) * D;
      const rsrc_t r = make_rsrc(at, (uint32_t)uniform(fetch.rows) * D * 2);
#pragma unroll
      for (int u = 0; u < HT; ++u)
#pragma unroll
        for (int i = 0; i < T::KD; ++i)
          q[u][i] = __builtin_bit_cast(half8_t, bldx4<0>(r, (16 * u + c) * (2 * D) + 32 * g, 128 * (i >> 1) + 16 * (i & 1)));
    };
    // The loads are issued in one order everywhere (q where it changes, K, V), and after the last tile
    // from empty ranges instead of not at all: only so the wait for a tile's K or V leaves the
    // younger loads in flight.
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
      bool bad[HT];                                  // the lane's part of q is not finite
#pragma unroll
      for (int u = 0; u < HT; ++u) {
#pragma unroll
        for (int j = 0; j < VJ; ++j) o[u][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        ref[u] = -INFINITY;
        l[u] = 0.f;
        bad[u] = false;
      }
      bool inside = true, fresh = true;              // the tile in t is of segment cur, and its first
      while (inside) {
        const int32_t t0 = token(0);
        const bool full = t0 >= cur.first && t0 + kTile <= cur.len && page[0] >= 0 && page[1] >= 0;
        uint32_t valid = 0xFF;                       // of the lane's eight tokens
        if (!full) {
          valid = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int32_t tok = t0 + 16 * (i >> 2) + 4 * g + (i & 3);
            valid |= (uint32_t)(tok >= cur.first && tok < cur.len && page[i >> 2] >= 0) << i;
          }
        }
        // the next tile's pages are on their way while this one's scores are made, its K while the
        // softmax and the products with V are, its V from then on: also across segments
        more = fetch.at + 1 < end;
        if (++fetch.at == fetch.end) {
          inside = false;
          if (more) fetch = segment_at<WHOLE>(a, fetch.at, end, fetch.b, fetch.u0 - (fetch.u1 - fetch.u0) * fetch.ht, fetch.len);
        }
        look_up();
        f32x4 x[2][HT];
#pragma unroll
        for (int st = 0; st < 2; ++st) scores<D, Q8, HT>(t, st, q, x[st]);
        if (Q8 && fresh) {
#pragma unroll
          for (int u = 0; u < HT; ++u) bad[u] = nonfinite<T::KD>(q[u]);
          fresh = false;
        }
        locate();
        if (more && !inside) load_q();
        load_k<D, Q8>(a, blk, t);
        half8_t hi[HT], lo[HT];
#pragma unroll
        for (int u = 0; u < HT; ++u) {
          float y[8], top = -INFINITY;
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = x[i >> 2][u][i & 3] * a.scale_log2;
          if (!full) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = (valid >> i & 1) ? y[i] : -INFINITY;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, y[i]);
          if (__any(top - ref[u] > kHigh)) {         // ref -inf: moves for any score, not for none (NaN)
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float now = fmaxf(ref[u], top - kLow);
            const float keep = now == ref[u] ? 1.0f : __builtin_amdgcn_exp2f(ref[u] - now);
            ref[u] = now;
            l[u] *= keep;
#pragma unroll
            for (int j = 0; j < VJ; ++j) o[u][j] *= keep;
          }
          float p[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = __builtin_amdgcn_exp2f(y[i] - ref[u]);
          if (!full) {                               // masked places may hold anything: zero times NaN is NaN
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = (valid >> i & 1) ? p[i] : 0.f;
            if (u == 0) {
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
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            l[u] += p[i];
            hi[u][i] = (_Float16)p[i];
            lo[u][i] = (_Float16)(p[i] - (float)hi[u][i]);
          }
        }
        accumulate<D, Q8, HT>(t, hi, lo, o);
        load_v<D, Q8>(a, blk, vs_lane, t);
      }
#pragma unroll
      for (int u = 0; u < HT; ++u) {
        if (Q8 && bad[u] && ref[u] > -INFINITY) l[u] = __builtin_nanf("");   // ref: moved by the first token that is seen
        l[u] += __shfl_xor(l[u], 16);
        l[u] += __shfl_xor(l[u], 32);
      }
      if (more) {
        // going on past this head tile: its result if the wave had all of it, else a part
        float *slot = cur.from_start ? nullptr : slot_of(a, 2 * v, D);
#pragma unroll
        for (int u = 0; u < HT; ++u)
          if (16 * u + c < cur.rows) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < VJ; j += 4)
                store_result<D>(a, cur.b, cur.h0, slot, 16 * u + c, VJ * (4 * g + i) + j,
                                f32x4{o[u][j][i], o[u][j + 1][i], o[u][j + 2][i], o[u][j + 3][i]}, ref[u], l[u]);
          }
        cur = fetch;
      }
    }
  }

  // the waves that ended on one head tile join their parts; the leader stores the sum
  if ((uint32_t)wave < live && g == 0) {
#pragma unroll
    for (int u = 0; u < HT; ++u) wave_m[wave][16 * u + c] = ref[u];
  }
  __syncthreads();
  uint32_t lead = 0, tail = 0;                       // first and last wave that end on this wave's head tile
  if ((uint32_t)wave < live) {
    lead = tail = wave;
    while (lead > 0 && line.start(v0 + lead) > cur.u0) --lead;
    while (tail + 1 < live && line.start(v0 + tail + 2) <= cur.u1) ++tail;
#pragma unroll
    for (int u = 0; u < HT; ++u) {
      const int r = 16 * u + c;
      float m = ref[u];
      for (uint32_t k = lead; k <= tail; ++k) m = fmaxf(m, wave_m[k][r]);
      const float f = ref[u] == m ? 1.0f : __builtin_amdgcn_exp2f(ref[u] - m);
      if (g == 0) {
        wave_l[wave][r] = l[u] * f;
        run_m[wave][r] = m;
      }
      if (r < cur.rows) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < VJ; j += 4)
            *reinterpret_cast<f32x4 *>(sums + (wave * a.rows + r) * kPad + VJ * (4 * g + i) + j) =
                f32x4{o[u][j][i] * f, o[u][j + 1][i] * f, o[u][j + 2][i] * f, o[u][j + 3][i] * f};
      }
    }
  }
  __syncthreads();
  if ((uint32_t)wave >= live) return;
  // every wave of the run sums its share of the elements
  float *slot = line.start(v0 + lead) <= cur.u0 && line.start(v0 + tail + 1) >= cur.u1 ? nullptr
                                                                                    : slot_of(a, 2 * (v0 + lead) + 1, D);
  for (int i = 4 * (64 * (wave - (int)lead) + lane); i < cur.rows * D; i += 256 * (int)(tail - lead + 1)) {
    const int r = i / D, d = i & (D - 1);
    f32x4 sum = f32x4{0.f, 0.f, 0.f, 0.f};
    float den = 0.f;
    for (uint32_t k = lead; k <= tail; ++k) {
      sum += *reinterpret_cast<const f32x4 *>(sums + (k * a.rows + r) * kPad + d);
      den += wave_l[k][r];
    }
    store_result<D>(a, cur.b, cur.h0, slot, r, d, sum, run_m[wave][r], den);
  }
}

// Joins the parts of the head tiles that several workgroups (or a wave that went on) hold. Workgroup
// (sequence and head tile, y) takes the heads y, y + gridDim.y, ...: kSplit groups of threads run
// through the parts, four elements of the output a thread and every load independent of the others,
// each with its own maximum and sum, and then join these. Latency-bound (4 to 7 us): the lengths,
// then all parts at once; one element a thread instead of four took 1 to 3 us more.
template <int D, int THREADS>
__global__ __launch_bounds__(THREADS) void attn_join_kernel(AttnArgs a, uint32_t waves) {
  constexpr uint32_t kLanes = D / 4, kSplit = THREADS / kLanes;
  __shared__ float part_m[kSplit], part_l[kSplit];
  __shared__ f32x4 sums[kSplit][kLanes];
  const int32_t b = blockIdx.x / a.head_tiles, ht = blockIdx.x - b * a.head_tiles;
  const Line line = make_line((uint32_t)scalar_load(a.starts_in + a.batch), waves);
  const Seen s = seen_of<false>(a, scalar_load(a.lens + b));
  const uint32_t u0 = (uint32_t)scalar_load(a.starts_in + b) + (uint32_t)ht * s.units;
  const uint32_t u1 = u0 + s.units, w0 = line.holder(u0), w1 = line.holder(u1 - 1);
  if (w0 == w1) return;
  // parts in order: those of workgroups, from the first of their waves, then the last wave's if it
  // went on. Wave w0 ends on the head tile, since it is not the last.
  const bool left = line.start(w1 + 1) > u1;
  const uint32_t e1 = left ? w1 - 1 : w1;            // the last wave that ends on the head tile
  const uint32_t groups = e1 / kWaves - w0 / kWaves + 1, n = groups + (left ? 1 : 0);
  if (n == 1) return;
  const int32_t kvh = ht / a.tiles_per_kv, first_head = (ht - kvh * a.tiles_per_kv) * a.tile_heads;
  const int32_t rows = min(a.tile_heads, a.group - first_head);
  const uint32_t i4 = threadIdx.x % kLanes, part = threadIdx.x / kLanes;
  for (int32_t r = blockIdx.y; r < rows; r += gridDim.y) {
    float m = -INFINITY, l = 0.f;
    f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (uint32_t i = part; i < n; i += kSplit) {
      const uint32_t lead = i == 0 ? w0 : (w0 / kWaves + i) * kWaves;
      const float *p = slot_of(a, i < groups ? 2 * lead + 1 : 2 * w1, D);
      const f32x2 ml = *reinterpret_cast<const f32x2 *>(p + a.rows * D + 2 * r);
      const f32x4 x = *reinterpret_cast<const f32x4 *>(p + r * D + 4 * i4);
      const float now = fmaxf(m, ml[0]);
      const float keep = m == now ? 1.0f : __builtin_amdgcn_exp2f(m - now);
      const float f = ml[0] == now ? 1.0f : __builtin_amdgcn_exp2f(ml[0] - now);
      o = o * keep + x * f;
      l = l * keep + ml[1] * f;
      m = now;
    }
    __syncthreads();                                 // of the previous row
    sums[part][i4] = o;
    if (i4 == 0) {
      part_m[part] = m;
      part_l[part] = l;
    }
    __syncthreads();
    if (part == 0) {
      for (uint32_t k = 1; k < kSplit; ++k) m = fmaxf(m, part_m[k]);
      o = f32x4{0.f, 0.f, 0.f, 0.f};
      l = 0.f;
      for (uint32_t k = 0; k < kSplit; ++k) {
        const float f = part_m[k] == m ? 1.0f : __builtin_amdgcn_exp2f(part_m[k] - m);
        o += sums[k][i4] * f;
        l += part_l[k] * f;
      }
      store_result<D>(a, b, kvh * a.group + first_head, nullptr, r, 4 * (int)i4, o, m, l);
    }
  }
}

namespace {

bool attn_misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// Tiles of a head tile of the longest sequence: of max_len tokens, or of a window that starts
// anywhere in a tile.
int64_t attn_tiles(int64_t max_len, int64_t window) {
  int64_t tiles = (max_len + kTile - 1) / kTile;
  if (window > 0 && window < max_len) {
    const int64_t seen = (window + kTile - 2) / kTile + 1;
    tiles = seen < tiles ? seen : tiles;
  }
  return tiles > 1 ? tiles : 1;
}

// Workgroups of four waves that are resident at once (heads of 64: four a CU, three with 32 heads a
// tile; of 128: two). Heads of 256 would fit two as well, but their parts are 16 KB for 16 heads: one a
// CU writes and joins half as many.
int64_t attn_resident(int64_t dim, int64_t tile_heads) { return dim == 64 ? (tile_heads == 16 ? 1024 : 768) : dim == 128 ? 512 : 256; }

// Heads of a head tile. More than 16 heads of a KV head in two tiles of 16 read and decode its K and V
// twice, so a tile takes 32 where the waves have steps enough for that to count; with few steps
// the larger parts cost more than this gains. 16 against 32 heads a tile, us: 32 sequences of 8192 tokens
// and 8 KV heads of 128 with 32 heads each, fp16 303 : 187, int8 172 : 117; of 6000 and 4 KV heads with
// 20 each, int8, 76 : 53; 32 of 8000 and 2 of 256 with 32 each, fp16 (17 registers spilled) 172 : 124; but
// 16 of up to 8000 and 2 KV heads with 32 each 24.4 : 25.0, one sequence of 4000 and 71 heads of 64
// 9.7 : 11.2. The steps are counted by max_len, since the lengths are on the device, so a ragged batch
// of short ones can get 32 and lose: int8, 32 sequences of up to 8192 (40% of that on average) and one KV
// head of 256 with 32 heads 35.6 : 38.7, with 20 33.4 : 34.5; of up to 4096 and 2 of 128 with 32 23.4 : 24.5;
// 64 of up to 4000 and 71 heads of 64 26.7 : 27.3. With more work ragged ones gain too (32 of up to 8192 and 2
// of 128 with 20 heads, int8 30.5 : 26.6, fp16 41.7 : 30.1).
int32_t attn_tile_heads(int64_t group, int64_t kv_heads, int64_t batch, int64_t tiles, int64_t dim) {
  const int64_t steps = batch * kv_heads * ((group + 15) / 16) * tiles;
  return group > 16 && steps >= 8 * kWaves * attn_resident(dim, 16) ? 32 : 16;
}

// Workgroups of the split: those resident, or as many as there are tiles for.
int32_t attn_grid(int64_t batch, int64_t head_tiles, int64_t tiles, int64_t dim, int64_t tile_heads) {
  const int64_t all = (batch * head_tiles * tiles + kWaves - 1) / kWaves, most = attn_resident(dim, tile_heads);
  return (int32_t)(all < most ? all : most);
}

// A workgroup for each head tile instead of the split, where that is the shorter way: the split
// evens out the work but costs a second launch (about 5 us with its wait), a head tile of n tiles
// keeps one workgroup busy for n / 4 steps. Split against whole, 32 heads on 8 of 128, int8, us:
// 1 sequence of 500 tokens 10.6 : 9.8, of 1000 10.9 : 14.6; 16 of 1000 17.6 : 15.2; 64 of up to
// 2000 38.7 : 34.8; 32 of up to 4096 (fp16) 42.6 : 53.2. Heads of 256, 4 KV heads, 130 sequences: of
// 500 tokens 42.5 : 46, of up to 500 30.1 : 26.8, of 1000 68 : 76, of up to 1000 39.6 : 40.4.
bool attn_whole(int64_t head_tiles, int64_t tiles, int64_t dim) {
  const int64_t most = dim == 256 ? 16 : head_tiles / 4;
  return tiles <= (most < 16 ? 16 : most < 64 ? most : 64);
}

// Waves of such a workgroup: fewer where more short head tiles wait than fit at once, so that more
// of them share the latency of a start (two or three dependent loads) and the LDS holds fewer sums. Four
// waves against these, int8, us: 4 heads of 256 and 130 sequences of 100 tokens 25.9 : 16.6 (one
// wave), 80 of 500 30.4 : 24.3 (two); 8 heads of 128 and 512 of up to 120 tokens 32.4 : 22.2 (one),
// 128 of them 13.1 : 10.2 (two), 64 of 500, which all fit, 16.9 : 19.7 with two. Long ones keep the
// card full with four: fp16, 512 sequences of 1000 tokens on 4 heads of 128 173 : 188 with two.
int whole_waves(int64_t head_tiles, int64_t tiles, int64_t dim, int64_t tile_heads) {
  const int64_t resident = attn_resident(dim, tile_heads);
  if (head_tiles <= resident || tiles > 16) return kWaves;
  return head_tiles >= 4 * resident || (head_tiles > 2 * resident && tiles <= 8) ? 1 : 2;
}

int64_t starts_bytes(int64_t batch) { return (4 * (batch + 1) + 15) / 16 * 16; }

template <int D, bool Q8, int HT>
int launch_attn(const AttnArgs &a, int64_t tiles, hipStream_t s) {
  const size_t lds = sizeof(float) * a.rows * (D + 4);
  const int64_t all = (int64_t)a.batch * a.head_tiles;
  if (attn_whole(all, tiles, D)) {
    const int waves = whole_waves(all, tiles, D, a.tile_heads);
    return launch(attn_kernel<D, Q8, true, HT>, dim3((unsigned)all), dim3(64 * waves), waves * lds, s, a);
  }
  const int32_t grid = attn_grid(a.batch, a.head_tiles, tiles, D, a.tile_heads);
  if (int st = launch(attn_kernel<D, Q8, false, HT>, dim3(grid), dim3(kThreads), kWaves * lds, s, a)) return st;
  // few head tiles: their heads shared out over workgroups (about 2048 in all), the more threads for an
  // element the more parts there are. 128 head tiles of 32 heads: 85 us with one workgroup each, 57 so.
  const uint32_t waves = (uint32_t)grid * kWaves;
  const int64_t share = 2048 / all;
  const dim3 heads((unsigned)all, (unsigned)(share < 1 ? 1 : share < a.rows ? share : a.rows));
  if (grid / all >= 128) return launch(attn_join_kernel<D, 1024>, heads, dim3(1024), 0, s, a, waves);
  return launch(attn_join_kernel<D, 256>, heads, dim3(256), 0, s, a, waves);
}

template <int D>
int launch_dim(const AttnArgs &a, int64_t tiles, bool q8, hipStream_t s) {
  if (a.tile_heads == 16) return q8 ? launch_attn<D, true, 1>(a, tiles, s) : launch_attn<D, false, 1>(a, tiles, s);
  return q8 ? launch_attn<D, true, 2>(a, tiles, s) : launch_attn<D, false, 2>(a, tiles, s);
}

int attn_shape(const qg_kv_pool *pool, int64_t batch, int64_t heads, int64_t max_len, KvLayout *L) {
  if (int st = kv_pool_layout(pool, L)) return st;
  if (batch < 0 || heads < 1 || heads % pool->kv_heads || heads > (1 << 22) || batch > (1 << 22) / heads) return QG_ERR_SHAPE;
  if (max_len < 0 || max_len > (1 << 30)) return QG_ERR_SHAPE;
  // The line fits 31 bits. Its extra units take nothing: a head tile has one below 16 tiles only (16 units
  // at most then), and there is a line only where the longest has more than 16 tiles (attn_whole).
  if (batch * heads * attn_tiles(max_len, 0) > 0x7FFFFFFF) return QG_ERR_SHAPE;
  return QG_OK;
}

}  // namespace

}  // namespace qg

using namespace qg;

extern "C" {

int qg_paged_attention_bytes(const qg_kv_pool *pool, int64_t batch, int64_t heads, int64_t max_len, int64_t *bytes) {
  if (!bytes) return QG_ERR_NULL;
  KvLayout L;
  if (int st = attn_shape(pool, batch, heads, max_len, &L)) return st;
  const int64_t group = heads / pool->kv_heads, tiles = attn_tiles(max_len, 0), dim = pool->head_dim;
  const int64_t tile = attn_tile_heads(group, pool->kv_heads, batch, tiles, dim);
  // a window only shortens the head tiles: what needs no join without one needs none with one, and
  // a call that is left with tiles of 16 heads has no more waves than counted here, nor larger parts
  *bytes = 0;
  if (batch == 0 || attn_whole(batch * pool->kv_heads * ((group + tile - 1) / tile), tiles, dim)) return QG_OK;
  const int64_t slots = 2 * kWaves * attn_grid(batch, (group + 15) / 16 * pool->kv_heads, tiles, dim, 16);
  *bytes = starts_bytes(batch) + 4 * slots * slot_floats((int32_t)(group < tile ? group : tile), (int32_t)dim);
  return QG_OK;
}

int qg_paged_attention(const qg_kv_pool *pool, int64_t layer, const uint16_t *q, int64_t ldq, const int32_t *table,
                       int64_t ld_table, const int32_t *lens, int64_t batch, int64_t heads, int64_t max_len,
                       int64_t window, float scale, void *out, int64_t ldo, int out_f32, float *lse, void *workspace,
                       int64_t workspace_bytes, void *stream) {
  KvLayout L;
  if (int st = attn_shape(pool, batch, heads, max_len, &L)) return st;
  const int64_t cols = heads * pool->head_dim;
  const int64_t pages = (max_len + pool->page_tokens - 1) / pool->page_tokens;
  if (int st = kv_table_check(table, ld_table, batch, pages)) return st;
  if (layer < 0 || layer >= pool->layers || window < 0 || (batch > 1 && (ldq < cols || ldo < cols))) return QG_ERR_SHAPE;
  if (!std::isfinite(scale * kLog2e)) return QG_ERR_RANGE;   // scores are kept in units of log2
  if (batch == 0) return QG_OK;
  int64_t need = 0;
  if (int st = qg_paged_attention_bytes(pool, batch, heads, max_len, &need)) return st;
  if (!q || !lens || !out || (need && !workspace)) return QG_ERR_NULL;
  if (attn_misaligned(q, 16) || attn_misaligned(out, 16) || attn_misaligned(lens, 4) || attn_misaligned(lse, 4) ||
      attn_misaligned(workspace, 16) || (batch > 1 && (ldq % 8 || ldo % (out_f32 ? 4 : 8))))
    return QG_ERR_ALIGN;
  if (workspace_bytes < need) return QG_ERR_WORKSPACE;
  AttnArgs a;
  a.window = (int32_t)(window > max_len ? 0 : window);
  const int64_t tiles = attn_tiles(max_len, a.window);
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
  a.batch = (int32_t)batch;
  a.heads = (int32_t)heads;
  a.group = (int32_t)(heads / pool->kv_heads);
  a.tile_heads = attn_tile_heads(a.group, pool->kv_heads, batch, tiles, pool->head_dim);
  a.tiles_per_kv = (a.group + a.tile_heads - 1) / a.tile_heads;
  a.head_tiles = a.tiles_per_kv * pool->kv_heads;
  a.rows = a.group < a.tile_heads ? a.group : a.tile_heads;
  a.max_len = (int32_t)max_len;
  a.scale_log2 = scale * kLog2e;
  a.out = out;
  a.ldo = batch > 1 ? ldo : cols;
  a.out_f32 = out_f32 != 0;
  a.lse = lse;
  a.starts = static_cast<uint32_t *>(workspace);
  a.starts_in = static_cast<const int32_t *>(workspace);
  a.slots = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + starts_bytes(batch));
  const bool q8 = pool->kind == QG_KV_Q8;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  switch (pool->head_dim) {
    case 64: return launch_dim<64>(a, tiles, q8, s);
    case 128: return launch_dim<128>(a, tiles, q8, s);
    default: return launch_dim<256>(a, tiles, q8, s);
  }
}

}  // extern "C"
