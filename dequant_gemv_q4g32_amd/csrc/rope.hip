// Queries and keys between the projection and the attention, gfx950: the norm of each head, the
// rotation of its pairs by the token's position, and the way of K and V into the paged cache.
//
// A head x of D elements becomes y = x / sqrt(mean x^2 + eps) * w where it has weights (else y = x), and
// the pair (y1, y2) with frequency f becomes factor * (y1 cos t - y2 sin t, y2 cos t + y1 sin t), t =
// position * f. All of it in fp32 with one rounding to fp16 at the end, but in fp64 for int8 keys, the angle, and its cosine and
// sine: a position of 100000 times a frequency near 1 leaves fp32 an error of 0.004 radians. These are made once for all
// heads of a token.
//
// A lane takes 8 elements of a head (16 bytes), D / 8 lanes a head, so that a norm is a sum over 8 to 32
// neighbouring lanes and a pair's other half is 8 elements of another lane of the same head.
//
// HBM bounds it: 8192 tokens of 64 and 8 heads of 128 into fp16 pages, 336 MB read and written, take 67 us, 5.0 TB/s
// (torch's copy of 2 GiB: 4.9), 4099 of 16 and 4 heads of 256, normed, 84 MB, 19 us. A workgroup takes a token, so that
// cosines and sines are made once for all its heads; with fewer than 1024 tokens its heads are shared over several, as a
// single token's would otherwise wait for each other. One token into int8 pages takes 5.0 us and 64 take 5.5: a chain of
// position, frequency and table entry behind a launch.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>

#include "../../include/qgemv.h"
#include "device_common.h"
#include "kv_codec.h"
#include "kv_pages.h"
#include "kv_rows.h"
#include "launch.h"

namespace qg {

typedef float float2_t __attribute__((ext_vector_type(2)));
typedef double double2_t __attribute__((ext_vector_type(2)));

constexpr int kRopeThreads = 256;

struct RopeArgs {
  RowsArgs rows;                 // the cache, K and V (x), the tokens' places; K alone without a cache
  const uint16_t *q;
  int64_t ldq;
  uint16_t *q_out, *k_out;       // k_out: without a cache
  int64_t ld_q_out, ld_k_out;
  const double *freqs;
  const uint16_t *q_weight, *k_weight;
  float eps, factor;
  int32_t half;                  // rotated pairs
  int32_t interleaved;
  int32_t heads, kv_heads;
};

enum RopeTo { kDense, kPagesQ8, kPagesF16 };

__device__ __forceinline__ void unpack8(u32x4 v, float *f) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = half_lo(v[j]);
    f[2 * j + 1] = half_hi(v[j]);
  }
}

// Sum over the D / 8 lanes of a head, in every one of them.
template <int D>
__device__ __forceinline__ float head_sum(float v) {
  v += dpp_move<0xB1, 0xF>(v);                     // quad_perm [1,0,3,2]
  v += dpp_move<0x4E, 0xF>(v);                     // quad_perm [2,3,0,1]
  v += dpp_move<0x141, 0xF>(v);                    // row_half_mirror
  if constexpr (D >= 128) v += dpp_move<0x140, 0xF>(v);   // row_mirror
  if constexpr (D >= 256) v += __shfl_xor(v, 16);
  return v;
}

// A key on its way to int8, in fp64, then rounded to fp32 and to fp16: its largest element of 32 decides the codes of all of
// them, and where that is rounded to fp16 the other way, or a code lies near a tie, a code changes, by up to a hundredth
// of the largest. The rounding to fp32 does that to one element of 2^14, and one code of 200000; in fp32 throughout it would be
// another element in 10000, and which ones would follow from the order of the sums. A decode step takes 0.5 us more for it; for
// fp16 results, where it would be half a step in one of 10000, it would take 82 us in place of 67 (8192 tokens).
template <int D>
__device__ __forceinline__ void key_head(float *y, const float *z, const uint16_t *weight, int away, float eps, const double2_t *turn,
                                         bool rotated, bool interleaved, bool second, int e, int half) {
  double yd[8], zd[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    yd[j] = y[j];
    zd[j] = z[j];
  }
  if (weight) {
    double ss = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += yd[j] * yd[j];
#pragma unroll
    for (int o = 1; o < D / 8; o <<= 1) ss += __shfl_xor(ss, o);
    const double inv = 1.0 / sqrt(ss * (1.0 / D) + (double)eps);
    float w[8], v[8];
    unpack8(*reinterpret_cast<const u32x4 *>(weight), w);
    unpack8(*reinterpret_cast<const u32x4 *>(weight + away), v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      yd[j] *= inv * w[j];
      zd[j] *= inv * v[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    double r = yd[j];
    if (rotated) {
      const double2_t cs = turn[interleaved ? (e + j) / 2 : second ? e - half + j : e + j];
      const double o = (interleaved ? yd[j ^ 1] : zd[j]) * cs[1];
      r = yd[j] * cs[0] + ((interleaved ? (j & 1) == 0 : !second) ? -o : o);
    }
    y[j] = (float)r;
  }
}

// Workgroup (token, y): the token's heads, its K and its V, 2048 / D of them a step.
template <int D, int TO>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a) {
  constexpr int L = D / 8, kUnits = kRopeThreads / L;
  __shared__ float2_t turn[D / 2];                    // factor * (cos, sin) of the pairs; the same
  __shared__ double2_t turn_k[TO == kPagesQ8 ? D / 2 : 1];   // for keys that become int8
  const uint32_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, l = tid % L, e = 8 * l;
  const int32_t pos = a.rows.positions[row];
  if (pos < 0) return;
  if (tid < a.half) {
    const double t = (double)pos * a.freqs[tid] * 0.15915494309189533577;
    const double r = 2 * (t - __builtin_rint(t));
    const double2_t cs = double2_t{a.factor * cospi(r), a.factor * sinpi(r)};
    turn[tid] = float2_t{(float)cs[0], (float)cs[1]};
    if constexpr (TO == kPagesQ8) turn_k[tid] = cs;
  }
  int32_t at = 0;
  uint8_t *page = nullptr;
  if constexpr (TO != kDense) page = row_page(a.rows, row, at);
  __syncthreads();
  const bool rotated = e < 2 * a.half, second = !a.interleaved && e >= a.half;
  const int other = !rotated || a.interleaved ? lane : second ? lane - a.half / 8 : lane + a.half / 8;
  const int32_t units = a.heads + (TO == kDense ? 1 : 2) * a.kv_heads;
  float2_t cs[8];
  if (rotated) {
#pragma unroll
    for (int j = 0; j < 8; ++j) cs[j] = turn[a.interleaved ? (e + j) / 2 : second ? e - a.half + j : e + j];
  }
  for (int32_t u0 = blockIdx.y * kUnits; u0 < units; u0 += gridDim.y * kUnits) {
    const int32_t u = u0 + tid / L;
    const bool live = u < units;
    const int32_t kind = u < a.heads ? 0 : u < a.heads + a.kv_heads ? 1 : 2;   // q, K, V
    const int32_t h = kind == 0 ? u : u - a.heads - (kind - 1) * a.kv_heads;
    u32x4 x = u32x4{0, 0, 0, 0};
    if (live) {
      const uint16_t *from = kind == 0 ? a.q + (int64_t)row * a.ldq : a.rows.x[kind - 1] + (int64_t)row * a.rows.ldx[kind - 1];
      x = *reinterpret_cast<const u32x4 *>(from + (int64_t)h * D + e);
    }
    const uint16_t *weight = kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr;
    float y[8], z[8];                              // the lane's elements, and the other halves of their pairs
    u32x4 p;
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = (uint32_t)__shfl((int)x[j], other);
    unpack8(x, y);
    unpack8(p, z);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(y[j], y[j], ss);
    ss = head_sum<D>(ss);
    if (TO == kPagesQ8 && kind == 1) {
      key_head<D>(y, z, weight ? weight + e : nullptr, 8 * (other - lane), a.eps, turn_k, rotated, a.interleaved, second, e, a.half);
    } else if (weight) {
      const float mean = ss * (1.0f / D) + a.eps;
      float inv = __builtin_amdgcn_rsqf(mean);       // to one step, and to half of one by
      const float rest = __builtin_fmaf(-(mean * inv), inv, 1.0f);
      inv = mean < INFINITY ? __builtin_fmaf(0.5f * inv, rest, inv) : inv;   // of an infinite head, zero as it is
      float w[8];
      unpack8(*reinterpret_cast<const u32x4 *>(weight + e), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = y[j] * inv * w[j];
      unpack8(*reinterpret_cast<const u32x4 *>(weight + e + 8 * (other - lane)), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] = z[j] * inv * w[j];
    }
    if (rotated && kind < (TO == kPagesQ8 ? 1 : 2)) {
      float r[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float o = a.interleaved ? y[j ^ 1] : z[j];
        const bool minus = a.interleaved ? (j & 1) == 0 : !second;
        const float s = o * cs[j][1];
        r[j] = __builtin_fmaf(y[j], cs[j][0], minus ? -s : s);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = r[j];
    }
    u32x4 out;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      out[j] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)y[2 * j]) |
               (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)y[2 * j + 1]) << 16;
    if (!live) continue;
    if (kind == 0) {
      *reinterpret_cast<u32x4 *>(a.q_out + (int64_t)row * a.ld_q_out + (int64_t)h * D + e) = out;
    } else if constexpr (TO == kDense) {
      *reinterpret_cast<u32x4 *>(a.k_out + (int64_t)row * a.ld_k_out + (int64_t)h * D + e) = out;
    } else if (page) {
      const auto place = place_in<TO == kPagesQ8>(a.rows, page, at, (uint32_t)(h * L + l));
      const int64_t off = kind == 1 ? place.off[0] : place.off[1];
      if constexpr (TO == kPagesQ8) {
        uint16_t d;
        const u32x2 codes = kv_encode8(out, d);      // a quad's lanes are of one head, so all four are here
        *reinterpret_cast<u32x2 *>(place.part + off) = codes;
        if ((l & 3) == 0) *reinterpret_cast<uint16_t *>(place.part + (kind == 1 ? place.scale_off[0] : place.scale_off[1])) = d;
      } else {
        *reinterpret_cast<u32x4 *>(place.part + off) = out;
      }
    }
  }
}

namespace {

bool rope_misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

constexpr int64_t kRopeCount = int64_t(1) << 23;    // workgroups of 256 threads in a grid's x axis
constexpr int64_t kRopeHeads = 65536;

int rope_check(const qg_rotary *r, int64_t head_dim, int64_t heads, int64_t kv_heads, int64_t count) {
  if (!r) return QG_ERR_NULL;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return QG_ERR_SHAPE;
  if (heads < 0 || heads > kRopeHeads || kv_heads < 0 || kv_heads > kRopeHeads || count < 0 || count > kRopeCount)
    return QG_ERR_SHAPE;
  if (r->rotary_dim < 0 || r->rotary_dim > head_dim || r->rotary_dim % 16) return QG_ERR_SHAPE;
  if (r->rotary_dim && !r->freqs) return QG_ERR_NULL;
  if (rope_misaligned(r->freqs, 8) || rope_misaligned(r->q_weight, 16) || rope_misaligned(r->k_weight, 16)) return QG_ERR_ALIGN;
  if (!std::isfinite(r->factor)) return QG_ERR_RANGE;
  if ((r->q_weight || r->k_weight) && !(std::isfinite(r->eps) && r->eps >= FLT_MIN)) return QG_ERR_RANGE;
  return QG_OK;
}

// fp16 rows of `cols` elements.
int rope_rows(const uint16_t *x, int64_t ld, int64_t cols, int64_t count) {
  if (count > 1 && cols && ld < cols) return QG_ERR_SHAPE;
  if (cols && !x) return QG_ERR_NULL;
  if (rope_misaligned(x, 16) || (count > 1 && cols && ld % 8)) return QG_ERR_ALIGN;
  return QG_OK;
}

template <int D>
int launch_rope(const RopeArgs &a, int to, int64_t count, hipStream_t s) {
  const int64_t units = a.heads + (to == kDense ? 1 : 2) * a.kv_heads, per = kRopeThreads / (D / 8);
  const int64_t steps = (units + per - 1) / per, share = 1024 / count;
  const dim3 grid((unsigned)count, (unsigned)(share < 1 ? 1 : share < steps ? share : steps)), block(kRopeThreads);
  switch (to) {
    case kDense: return launch(rope_kernel<D, kDense>, grid, block, 0, s, a);
    case kPagesQ8: return launch(rope_kernel<D, kPagesQ8>, grid, block, 0, s, a);
    default: return launch(rope_kernel<D, kPagesF16>, grid, block, 0, s, a);
  }
}

int rope(RopeArgs &a, const qg_rotary *r, int to, int64_t head_dim, int64_t heads, int64_t kv_heads, const uint16_t *q,
         int64_t ldq, const uint16_t *k, int64_t ldk, const int32_t *positions, int64_t count, uint16_t *q_out,
         int64_t ld_q_out, void *stream) {
  a.q = q;
  a.ldq = count > 1 ? ldq : 0;
  a.rows.x[0] = const_cast<uint16_t *>(k);
  a.rows.ldx[0] = count > 1 ? ldk : 0;
  a.rows.positions = positions;
  a.q_out = q_out;
  a.ld_q_out = count > 1 ? ld_q_out : 0;
  a.freqs = r->freqs;
  a.q_weight = r->q_weight;
  a.k_weight = r->k_weight;
  a.eps = r->eps;
  a.factor = r->factor;
  a.half = r->rotary_dim / 2;
  a.interleaved = r->interleaved != 0;
  a.heads = (int32_t)heads;
  a.kv_heads = (int32_t)kv_heads;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  switch (head_dim) {
    case 64: return launch_rope<64>(a, to, count, s);
    case 128: return launch_rope<128>(a, to, count, s);
    default: return launch_rope<256>(a, to, count, s);
  }
}

}  // namespace

}  // namespace qg

using namespace qg;

extern "C" {

int qg_qk_rope(const qg_rotary *rotary, int64_t head_dim, int64_t heads, int64_t kv_heads, const uint16_t *q, int64_t ldq,
               const uint16_t *k, int64_t ldk, const int32_t *positions, int64_t count, uint16_t *q_out, int64_t ld_q_out,
               uint16_t *k_out, int64_t ld_k_out, void *stream) {
  if (int st = rope_check(rotary, head_dim, heads, kv_heads, count)) return st;
  const int64_t cols = heads * head_dim, kv_cols = kv_heads * head_dim;
  if (count == 0 || heads + kv_heads == 0) return QG_OK;
  for (int st : {rope_rows(q, ldq, cols, count), rope_rows(k, ldk, kv_cols, count), rope_rows(q_out, ld_q_out, cols, count),
                 rope_rows(k_out, ld_k_out, kv_cols, count)})
    if (st) return st;
  if (!positions) return QG_ERR_NULL;
  if (rope_misaligned(positions, 4)) return QG_ERR_ALIGN;
  RopeArgs a{};
  a.k_out = k_out;
  a.ld_k_out = count > 1 ? ld_k_out : 0;
  return rope(a, rotary, kDense, head_dim, heads, kv_heads, q, ldq, k, ldk, positions, count, q_out, ld_q_out, stream);
}

int qg_kv_append_rope(const qg_kv_pool *pool, int64_t layer, const int32_t *table, int64_t ld_table, int64_t table_rows,
                      int64_t table_pages, const qg_rotary *rotary, int64_t heads, const uint16_t *q, int64_t ldq,
                      const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv, const int32_t *seqs,
                      const int32_t *positions, int64_t count, uint16_t *q_out, int64_t ld_q_out, void *stream) {
  KvLayout L;
  if (int st = kv_pool_layout(pool, &L)) return st;
  if (int st = kv_table_check(table, ld_table, table_rows, table_pages)) return st;
  if (layer < 0 || layer >= pool->layers) return QG_ERR_SHAPE;
  if (int st = rope_check(rotary, pool->head_dim, heads, pool->kv_heads, count)) return st;
  const int64_t cols = heads * pool->head_dim, kv_cols = (int64_t)pool->kv_heads * pool->head_dim;
  if (count == 0) return QG_OK;
  for (int st : {rope_rows(q, ldq, cols, count), rope_rows(k, ldk, kv_cols, count), rope_rows(v, ldv, kv_cols, count),
                 rope_rows(q_out, ld_q_out, cols, count)})
    if (st) return st;
  if (!positions) return QG_ERR_NULL;
  if (rope_misaligned(positions, 4) || rope_misaligned(seqs, 4)) return QG_ERR_ALIGN;
  RopeArgs a{};
  RowsArgs &w = a.rows;
  w.pool = static_cast<uint8_t *>(pool->pages) + (layer ? layer * pool->layer_stride : 0);
  w.page_bytes = L.page_bytes;
  w.head_bytes = L.head_bytes;
  w.v_off = L.v_off;
  w.ks_off = L.ks_off;
  w.vs_off = L.vs_off;
  w.num_pages = (int32_t)pool->num_pages;
  w.table = table;
  w.ld_table = ld_table;
  w.table_rows = (int32_t)table_rows;
  w.table_pages = (int32_t)table_pages;
  w.x[1] = const_cast<uint16_t *>(v);
  w.ldx[1] = count > 1 ? ldv : 0;
  w.seqs = seqs;
  w.lane_shift = __builtin_ctz(pool->head_dim / 8);
  w.tok_shift = __builtin_ctz(pool->page_tokens);
  return rope(a, rotary, pool->kind == QG_KV_Q8 ? kPagesQ8 : kPagesF16, pool->head_dim, heads, pool->kv_heads, q, ldq, k, ldk,
              positions, count, q_out, ld_q_out, stream);
}

}  // extern "C"
