// What the attention kernels over the paged cache share (paged_attn.hip, prefix_attn.hip): the running
// reference of the softmax, a line of work shared out over workers, and a wave's step of 32 tokens against up to 16
// or 32 heads: its loads, the decoding of int8 entries, the scores and the products with V.
#pragma once
#include <hip/hip_runtime.h>

#include "device_common.h"

namespace qg {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kTile = 32;                          // tokens of a wave's step, the grain of the split
// Weights are 2^(s - ref) with ref moved to (largest s) - 7 once s - ref passes 15: they stay below
// fp16's 65504 and small ones lose nothing above 2^-31 of the largest, while most steps find ref good
// as it is. The difference itself is compared, as the weights use it: ref + 15 rounds up to ref + 16
// for scores of 2^24 to 2^28.
// A weight below 2^-14 is a subnormal fp16 number (as a pair: its remainder is), off by up to 2^-25, which is 2^-31 of the
// weights' sum at most: that is 2^6 or more while s - 7 is good to one, below scores of 2^24. Larger scores
// differ by multiples of 2^k, 2^(k + 24) being their size, so that what of a weight is lost is at most 2^-25, 2^-26, 2^-28 and 2^-32
// for k = 0, 1, 2 and from 3 on, while the sum is at least 2^6, 2^5, 2^4 and 1.
constexpr float kLow = 7.0f, kHigh = 15.0f;

template <typename T>
__device__ __forceinline__ T uniform(T v) { return __builtin_amdgcn_readfirstlane(v); }

// Read-only memory at a uniform address, through the scalar cache.
__device__ __forceinline__ int32_t scalar_load(const int32_t *p) {
  return *(const __attribute__((address_space(4))) int32_t *)(uintptr_t)p;
}

// A line of `total` units of work that `waves` workers share, worker v the v-th part: quota units, and one more
// if v < extra.
struct Line {
  uint32_t total, waves, quota, extra, first;
  __device__ __forceinline__ uint32_t start(uint32_t v) const { return first + v * quota + min(v, extra); }
  // the wave that holds unit u
  __device__ __forceinline__ uint32_t holder(uint32_t u) const {
    const uint32_t big = extra * (quota + 1);
    return u < big ? u / (quota + 1) : extra + (u - big) / quota;
  }
};
__device__ __forceinline__ Line make_line(uint32_t total, uint32_t waves) {
  Line l;
  l.total = total;
  l.first = 0;
  l.waves = min(total, waves);
  l.quota = total / l.waves;
  l.extra = total - l.quota * l.waves;
  return l;
}

// Sum of `v` over this lane and those before it: within rows of 16, then over the rows.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false);   // row_shr:1
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false);   // row_shr:2
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false);   // row_shr:4
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false);   // row_shr:8
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false);   // row_bcast:15
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false);   // row_bcast:31
  return v;
}

// 16 codes of one group to 16 fp16 values: code + 128 under the exponent of 1024 (a byte permute
// and an exact subtraction for two), times the scale, rounded to fp16 as qg_kv_dequantize does.
// MODE.FP16_OVFL (set at the start of the kernel) saturates the product at +-65504: without it the
// one scale that can pass it (516) would need two more operations for every pair.
__device__ __forceinline__ uint32_t scaled_pair(uint32_t magic_pair, uint32_t scale) {
  const h2_t off = __builtin_bit_cast(h2_t, 0x64806480u);       // 1152 = 1024 + 128
  return __builtin_bit_cast(uint32_t, (__builtin_bit_cast(h2_t, magic_pair) - off) * __builtin_bit_cast(h2_t, scale));
}
constexpr uint32_t kMagicBytes = 0x64646464u;
constexpr uint32_t kSelLow = 0x04010400u, kSelHigh = 0x04030402u;   // bytes 0, 1 and 2, 3 of the second operand under 0x64

template <int D, bool Q8>
struct Tile {
  static constexpr int KD = D / 32;                 // matrix steps along the head
  static constexpr int VJ = D / 16;                 // elements of one token's V a lane holds
  static constexpr int KR = Q8 ? D / 64 : D / 32;   // 16-byte loads of a K row a lane takes part in
  static constexpr int VW = Q8 ? VJ / 4 : VJ / 2;   // dwords of a V row a lane holds
  u32x4 k[2][KR];
  uint32_t ks[2][Q8 ? D / 64 : 1];
  uint32_t v[8][VW];
  u32x2 vs[2];
};

// A 16-token block in memory: its KV head's part of a page as a buffer resource, and the block's
// first place in the page. A block without a page has an empty range, whose loads give zeros.
struct Block {
  rsrc_t r;
  uint32_t place;
};

// Cache policy: V's codes past the caches (each line is one instruction's), K cached, since two or
// four instructions share each of its lines, and the scales, whose lines many lanes share. 64
// sequences of 8192 tokens: all cached 361 us (fp16) and 205 us (int8), all past the caches 316 and
// 192, this way 322 and 187, and the ragged and short cases all fastest.
template <int N, int AUX>
__device__ __forceinline__ void load_words(rsrc_t r, uint32_t voff, uint32_t soff, uint32_t *w) {
  if constexpr (N == 1) {
    w[0] = bldx1<AUX>(r, voff, soff);
  } else if constexpr (N == 2) {
    const u32x2 t = bldx2<AUX>(r, voff, soff);
    w[0] = t.x;
    w[1] = t.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 t = bldx4<AUX>(r, voff + 16 * i, soff);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[4 * i + j] = t[j];
    }
  }
}

// K of a tile: lane (c = lane % 16, g = lane / 16) takes token c of each 16-token block; of every 64
// elements of its row the 16 at 16 g, eight for each of two matrix steps. The lane's part of an
// address never changes: what does (page, place) is scalar.
template <int D, bool Q8, typename Args>
__device__ __forceinline__ void load_k(const Args &a, const Block *blk, Tile<D, Q8> &t) {
  const uint32_t lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
  for (int st = 0; st < 2; ++st) {
#pragma unroll
    for (int i = 0; i < Tile<D, Q8>::KR; ++i)
      t.k[st][i] = Q8 ? bldx4<0>(blk[st].r, c * D + 16 * g + 64 * i, blk[st].place * D)
                      : bldx4<0>(blk[st].r, c * 2 * D + 32 * g + 128 * (i >> 1) + 16 * (i & 1), blk[st].place * 2 * D);
    if constexpr (Q8) load_words<D / 64, 0>(blk[st].r, c * (D / 16), a.ks_off + blk[st].place * (D / 16), t.ks[st]);
  }
}

// V of a tile: a lane takes the VJ elements at VJ * c of the tokens 4 g .. 4 g + 3 of each block.
template <int D, bool Q8, typename Args>
__device__ __forceinline__ void load_v(const Args &a, const Block *blk, uint32_t vs_lane, Tile<D, Q8> &t) {
  constexpr uint32_t VJ = Tile<D, Q8>::VJ, VW = Tile<D, Q8>::VW, kElem = Q8 ? 1 : 2;
  const uint32_t lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
  for (int st = 0; st < 2; ++st) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      load_words<VW, kNT>(blk[st].r, (4 * g * D + VJ * c) * kElem + i * D * kElem, a.v_off + blk[st].place * (D * kElem),
                     t.v[4 * st + i]);
    if constexpr (Q8) t.vs[st] = bldx2<0>(blk[st].r, vs_lane, a.vs_off + 2 * blk[st].place);
  }
}

// Scores of a block against each 16 heads: S^T [16 tokens x 16 heads] = K Q^T. Lane: head c, tokens 4 g + i.
template <int D, bool Q8, int HT>
__device__ __forceinline__ void scores(const Tile<D, Q8> &t, int st, const half8_t (*q)[D / 32], f32x4 *s) {
#pragma unroll
  for (int u = 0; u < HT; ++u) s[u] = f32x4{0.f, 0.f, 0.f, 0.f};
  if constexpr (Q8) {
    const uint32_t pick = (threadIdx.x & 32) ? 0x03020302u : 0x01000100u;   // the group of the lane's 16 elements
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const uint32_t d = __builtin_amdgcn_perm(t.ks[st][i], t.ks[st][i], pick);
      u32x4 w[2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = t.k[st][i][j] ^ 0x80808080u;
        w[j >> 1][2 * (j & 1)] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, x, kSelLow), d);
        w[j >> 1][2 * (j & 1) + 1] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, x, kSelHigh), d);
      }
#pragma unroll
      for (int u = 0; u < HT; ++u) {
        s[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, w[0]), q[u][2 * i], s[u], 0, 0, 0);
        s[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, w[1]), q[u][2 * i + 1], s[u], 0, 0, 0);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int u = 0; u < HT; ++u)
        s[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, t.k[st][i]), q[u][i], s[u], 0, 0, 0);
  }
}

// Whether the lane's part of q holds a NaN or an infinity. FP16_OVFL makes the matrix units take
// either as a finite number, so with int8 pages such a head is marked instead: its scores are
// infinite or NaN against any finite K, and its softmax is NaN as soon as it sees a token.
template <int KD>
__device__ __forceinline__ bool nonfinite(const half8_t *q) {
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < KD; ++i) {
    const u32x4 x = __builtin_bit_cast(u32x4, q[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) bad |= (x[j] & 0x7C007C00u) + 0x04000400u;   // an exponent of ones carries into bit 15
  }
  return (bad & 0x80008000u) != 0;
}

// O^T += V^T P^T with the weights as hi + lo fp16 pairs. Column c of V^T's block j is element
// VJ * c + j, so O^T's lane holds head c and elements VJ * (4 g + i) + j.
template <int D, bool Q8, int HT>
__device__ __forceinline__ void accumulate(const Tile<D, Q8> &t, const half8_t *hi, const half8_t *lo, f32x4 (*o)[D / 16]) {
  constexpr int VW = Tile<D, Q8>::VW;
#pragma unroll
  for (int w = 0; w < VW; ++w) {
    if constexpr (Q8) {
      // two tokens' dwords interleave to bytes (t0 d, t1 d, t0 d+1, t1 d+1), then to fp16 pairs
      u32x4 e[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t x0 = t.v[2 * p][w] ^ 0x80808080u, x1 = t.v[2 * p + 1][w] ^ 0x80808080u;
        const uint32_t d = t.vs[p >> 1][p & 1];
        const uint32_t a = __builtin_amdgcn_perm(x1, x0, 0x05010400u), b = __builtin_amdgcn_perm(x1, x0, 0x07030602u);
        e[0][p] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, a, kSelLow), d);
        e[1][p] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, a, kSelHigh), d);
        e[2][p] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, b, kSelLow), d);
        e[3][p] = scaled_pair(__builtin_amdgcn_perm(kMagicBytes, b, kSelHigh), d);
      }
#pragma unroll
      for (int u = 0; u < HT; ++u) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[u][4 * w + j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, e[j]), hi[u], o[u][4 * w + j], 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[u][4 * w + j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, e[j]), lo[u], o[u][4 * w + j], 0, 0, 0);
      }
    } else {
      u32x4 e[2];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        e[0][p] = __builtin_amdgcn_perm(t.v[2 * p + 1][w], t.v[2 * p][w], 0x05040100u);
        e[1][p] = __builtin_amdgcn_perm(t.v[2 * p + 1][w], t.v[2 * p][w], 0x07060302u);
      }
#pragma unroll
      for (int u = 0; u < HT; ++u) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          o[u][2 * w + j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, e[j]), hi[u], o[u][2 * w + j], 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          o[u][2 * w + j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, e[j]), lo[u], o[u][2 * w + j], 0, 0, 0);
      }
    }
  }
}

}  // namespace qg
