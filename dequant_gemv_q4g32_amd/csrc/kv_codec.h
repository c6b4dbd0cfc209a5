// The 8-bit KV-cache group codec on 8 consecutive elements a lane (kvcache.hip and paged_kv.hip).
#pragma once
#include <hip/hip_runtime.h>

#include "device_common.h"

namespace qg {

constexpr int kKvGroup = 32;

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, dpp_move<0xB1, 0xF>(v));   // quad_perm [1,0,3,2]
  v = fmaxf(v, dpp_move<0x4E, 0xF>(v));   // quad_perm [2,3,0,1]
  return v;
}

// Eight fp16 values v of a lane to eight codes; the 4 lanes of a quad hold one group and agree
// on its scale, returned as fp16 bits (every lane of the quad must call this together).
__device__ __forceinline__ u32x2 kv_encode8(u32x4 v, uint16_t &scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[8];
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = half_lo(w[j]);
    f[2 * j + 1] = half_hi(w[j]);
    amax = fmaxf(amax, fmaxf(fabsf(f[2 * j]), fabsf(f[2 * j + 1])));
  }
  amax = quad_max(amax);
  // d = smallest fp16 >= amax / 127 (t is finite and non-negative, at most 65504 / 127). The
  // fp32 quotient cannot cross an fp16 value: amax is fp16, so the exact quotient lies either
  // on an fp16 number or at least 2^-18 of its size away from every one, far beyond fp32's
  // rounding.
  const float t = amax / 127.0f;
  _Float16 h = (_Float16)t;
  if ((float)h < t) h = __builtin_bit_cast(_Float16, (uint16_t)(__builtin_bit_cast(uint16_t, h) + 1));
  const float d = (float)h;
  const float inv = d > 0.f ? 1.0f / d : 0.f;   // one division per group
  uint32_t packed[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    // x = a 2^i and d = b 2^k with a, b integers below 2^11 (fp16), so x / d is either a
    // half-integer or at least 1 / (2 b) >= 2^-12 away from every one, which is 1.9e-6 of the
    // largest quotient, 127.5. x * inv (inv = 1 / d rounded once) is within 2^-23 of x / d
    // relative, so q0 = rint(x * inv) is already the nearest integer except at an exact tie,
    // where it may be the odd neighbour. The remainder e = x - q0 d is exact in fp32 (x and d
    // are fp16, |q0| <= 127, and for q0 != 0 |x| >= d / 2, so e is a multiple of half of d's
    // last-place unit below 1.5 d: 13 bits); a tie is 2e = +-d, and then the even code is
    // q0 + sign(e). |x| <= 127 d keeps q within [-127, 127]. (d = 0: inv = 0, q = 0, e = 0.)
    float q = __builtin_rintf(f[j] * inv);
    const float e2 = 2.0f * __builtin_fmaf(-q, d, f[j]);
    const bool fix = __builtin_fabsf(e2) == d && ((int32_t)q & 1) != 0;
    q += fix ? __builtin_copysignf(1.0f, e2) : 0.0f;
    packed[j >> 2] |= ((uint32_t)(int32_t)q & 0xFFu) << (8 * (j & 3));
  }
  scale = __builtin_bit_cast(uint16_t, h);
  return u32x2{packed[0], packed[1]};
}

// Eight codes q of scale d to eight fp16 values.
__device__ __forceinline__ u32x4 kv_decode8(u32x2 q, float d) {
  const uint32_t qw[2] = {q.x, q.y};
  uint32_t out[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t word = qw[j >> 1] >> (16 * (j & 1));
    // d * q is exact in fp32; only 127 * 516 = 65532 lies past the fp16 maximum, saturated
    const float a = fminf(fmaxf((float)(int8_t)(word & 0xFFu) * d, -65504.f), 65504.f);
    const float b = fminf(fmaxf((float)(int8_t)((word >> 8) & 0xFFu) * d, -65504.f), 65504.f);
    out[j] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)a) | ((uint32_t)__builtin_bit_cast(uint16_t, (_Float16)b) << 16);
  }
  return u32x4{out[0], out[1], out[2], out[3]};
}

}  // namespace qg
