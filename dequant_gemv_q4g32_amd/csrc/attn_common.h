// What the attention kernels over the paged cache share (paged_attn.hip, prefix_attn.hip): the running
// reference of the softmax, a line of work shared out over workers, the decoding of int8 entries.
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
// Weights are 2^(s - ref) with ref moved to (largest s) - 7 once s - ref passes 15: they stay below
// fp16's 65504 and small ones lose nothing above 2^-31 of the largest, while most steps find ref good
// as it is. The difference itself is compared, as the weights use it: ref + 15 rounds up to ref + 16
// for scores of 2^24 to 2^28.
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

}  // namespace qg
