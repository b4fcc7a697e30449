// Rows rounded to 8 bits with a scale each.
//
// s = fp32(max |x| / 127), q = rint(x / s): which whole number is nearest to
// the exact quotient, ties to even.  n = rint(x * (1 / s)) is that number or its
// neighbour; the remainder x - n s is a multiple of half a unit in the last
// place of s and not much larger than s / 2, so one fma gives it exactly and it
// decides.  A row whose largest magnitude is below 2^-119 (where s would
// leave fp32's normal range) has s = 0 and codes 0; one with a NaN or infinity
// has s = NaN and codes 0.
#pragma once

#include "i8_core.h"

namespace qmm {

// Sixteen values from x[at].
__device__ __forceinline__ void i8_load16(const void* x, size_t at, int type, float (&v)[16]) {
  if (type == kI8F32) {
    auto p = to_global(reinterpret_cast<const u32x4*>(static_cast<const float*>(x) + at));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4 u = p[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = __uint_as_float(u[j]);
    }
    return;
  }
  auto p = to_global(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + at));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const u32x4 u = p[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * i + 2 * j] = type == kI8F16 ? f16_bits_to_f32((uint16_t)u[j]) : __uint_as_float(u[j] << 16);
      v[8 * i + 2 * j + 1] = type == kI8F16 ? f16_bits_to_f32((uint16_t)(u[j] >> 16)) : __uint_as_float(u[j] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ int i8_round(float x, float s, float inv) {
  const float n = rintf(x * inv);
  const float d = fmaf(-n, s, x);
  const float h = 0.5f * s;
  const int i = (int)n;
  const int up = d > h || (d == h && (i & 1));
  const int down = d < -h || (d == -h && (i & 1));
  return i + up - down;
}

__device__ __forceinline__ i32x4 i8_round16(const float (&v)[16], float s, float inv) {
  i32x4 q;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) w |= (uint32_t)(i8_round(v[4 * i + j], s, inv) & 0xFF) << (8 * j);
    q[i] = (int)w;
  }
  return q;
}

__device__ __forceinline__ uint32_t i8_top(const float (&v)[16], uint32_t top) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t u = __float_as_uint(v[i]) & 0x7FFFFFFFu;  // ordered like the magnitude, NaN above infinity
    top = u > top ? u : top;
  }
  return top;
}

// Scale of a row from the bits of its largest magnitude; 0 and NaN have codes 0.
__device__ __forceinline__ float i8_scale(uint32_t top) {
  if (top >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  if (top < 0x04000000u) return 0.0f;  // 2^-119
  return __fdiv_rn(__uint_as_float(top), 127.0f);
}

__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const uint32_t u = __shfl_xor((int)v, d, 64);
    v = u > v ? u : v;
  }
  return v;
}

}  // namespace qmm
