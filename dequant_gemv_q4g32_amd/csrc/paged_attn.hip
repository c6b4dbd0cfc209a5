// Attention of one new token a sequence over a paged KV cache, gfx950.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/qgemv.h"
#include "device_common.h"
#include "kv_codec.h"
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
  int32_t max_len, window;
  float scale;
  void *out;
  int64_t ldo;
  int32_t out_f32;
  float *lse;
};

// Eight elements of token `at` of a page, K (which = 0) or V, as fp32.
template <int D, bool Q8>
__device__ __forceinline__ void load8(const AttnArgs &a, const uint8_t *head, int which, int at, int e, float *f) {
  u32x4 w;
  if constexpr (Q8) {
    const uint8_t *c = head + (which ? a.v_off : 0) + at * D + e;
    const uint8_t *s = head + (which ? a.vs_off + 2 * (((e / 32) << a.tok_shift) + at) : a.ks_off + 2 * (at * (D / 32) + e / 32));
    w = kv_decode8(ld2(c), half_bits(ldh(s)));
  } else {
    w = ld4(head + (which ? a.v_off : 0) + 2 * (at * D + e));
  }
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = half_lo(w[j]);
    f[2 * j + 1] = half_hi(w[j]);
  }
}

// One wave per (sequence, head): 64 tokens at a time, a lane scores one token, then holds
// D / 64 elements of the output.
template <int D, bool Q8>
__global__ __launch_bounds__(64) void attn_kernel(AttnArgs a) {
  __shared__ float qs[D], p[64], v[64][8];
  const int b = blockIdx.x / a.heads, h = blockIdx.x - b * a.heads, lane = threadIdx.x;
  const int len = min(max(a.lens[b], 0), a.max_len);
  const int first = a.window ? max(0, len - a.window) : 0;
  for (int e = lane; e < D; e += 64) qs[e] = half_bits(a.q[b * a.ldq + (int64_t)h * D + e]);
  __syncthreads();
  float m = -INFINITY, l = 0.f, acc[D / 64] = {};
  for (int t0 = first; t0 < len; t0 += 64) {
    const int t = t0 + lane;
    const uint8_t *head = nullptr;
    if (t < len) {
      const int page = a.table[b * a.ld_table + (t >> a.tok_shift)];
      if (page >= 0 && page < a.num_pages) head = a.pool + page * a.page_bytes + (h / a.group) * a.head_bytes;
    }
    const int at = t & ((1 << a.tok_shift) - 1);
    float s = 0.f;
    if (head)
      for (int e = 0; e < D; e += 8) {
        float f[8];
        load8<D, Q8>(a, head, 0, at, e, f);
        for (int j = 0; j < 8; ++j) s = fmaf(qs[e + j], f[j], s);
      }
    s = head ? s * a.scale : -INFINITY;
    float top = s;
    for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    const float now = fmaxf(m, top);
    const float base = now == -INFINITY ? 0.f : now;
    const float w = head ? expf(s - base) : 0.f;
    const float keep = expf(m - base);
    m = now;
    float sum = w;
    for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
    l = l * keep + sum;
    for (int i = 0; i < D / 64; ++i) acc[i] *= keep;
    p[lane] = w;
    for (int e = 0; e < D; e += 8) {
      float f[8] = {};
      if (head) load8<D, Q8>(a, head, 1, at, e, f);
      __syncthreads();
      for (int j = 0; j < 8; ++j) v[lane][j] = head ? f[j] : 0.f;
      __syncthreads();
      // element e + j belongs to lane (e + j) % 64
      const int j = lane - (e & 63);
      if (j >= 0 && j < 8) {
        float add = 0.f;
        for (int k = 0; k < 64; ++k) add = fmaf(p[k], v[k][j], add);
        for (int i = 0; i < D / 64; ++i)
          if (i == e / 64) acc[i] += add;
      }
    }
    __syncthreads();
  }
  const float inv = l > 0.f ? 1.0f / l : l;     // a NaN stays one
  for (int i = 0; i < D / 64; ++i) {
    const int64_t o = b * a.ldo + (int64_t)h * D + 64 * i + lane;
    const float y = acc[i] * inv;
    if (a.out_f32) static_cast<float *>(a.out)[o] = y;
    else static_cast<uint16_t *>(a.out)[o] = __builtin_bit_cast(uint16_t, (_Float16)y);
  }
  if (a.lse && lane == 0) a.lse[(int64_t)b * a.heads + h] = m + logf(l);
}

namespace {

bool attn_misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

template <int D>
int launch_dim(const AttnArgs &a, bool q8, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.batch * a.heads)), block(64);
  return q8 ? launch(attn_kernel<D, true>, grid, block, 0, s, a) : launch(attn_kernel<D, false>, grid, block, 0, s, a);
}

int attn_shape(const qg_kv_pool *pool, int64_t batch, int64_t heads, int64_t max_len, KvLayout *L) {
  if (int st = kv_pool_layout(pool, L)) return st;
  if (batch < 0 || heads < 1 || heads % pool->kv_heads || heads > (1 << 24) || batch > (1 << 24) / heads) return QG_ERR_SHAPE;
  if (max_len < 0 || max_len > (1 << 30)) return QG_ERR_SHAPE;
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
  *bytes = 16;
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
  if (!std::isfinite(scale)) return QG_ERR_RANGE;
  if (batch == 0) return QG_OK;
  if (!q || !lens || !out || !workspace) return QG_ERR_NULL;
  if (attn_misaligned(q, 16) || attn_misaligned(out, 16) || attn_misaligned(lens, 4) || attn_misaligned(lse, 4) ||
      attn_misaligned(workspace, 16) || (batch > 1 && (ldq % 8 || ldo % (out_f32 ? 4 : 8))))
    return QG_ERR_ALIGN;
  int64_t need = 0;
  if (int st = qg_paged_attention_bytes(pool, batch, heads, max_len, &need)) return st;
  if (workspace_bytes < need) return QG_ERR_WORKSPACE;
  AttnArgs a;
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
  a.max_len = (int32_t)max_len;
  a.window = (int32_t)(window > max_len ? 0 : window);
  a.scale = scale;
  a.out = out;
  a.ldo = batch > 1 ? ldo : cols;
  a.out_f32 = out_f32 != 0;
  a.lse = lse;
  const bool q8 = pool->kind == QG_KV_Q8;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  switch (pool->head_dim) {
    case 64: return launch_dim<64>(a, q8, s);
    case 128: return launch_dim<128>(a, q8, s);
    default: return launch_dim<256>(a, q8, s);
  }
}

}  // extern "C"
