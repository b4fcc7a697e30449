// Rows rounded to 8 bits with a scale each.
//
// s = fp32(max |x| / 127), q = rint(x / s): which whole number is nearest to
// the exact quotient, ties to even.  n = rint(x * (1 / s)) is that number or its
// neighbour; the remainder x - n s is a multiple of half a unit in the last
// place of s (of fp32's smallest number, if that is more) and not much larger than
// s / 2, so one fma gives it exactly and it decides: n is the nearest if twice the
// remainder is below s (half of the smallest s would not be exact).  A row whose largest magnitude is below 2^-119 (where s would
// leave fp32's normal range) has s = 0 and codes 0; one with a NaN or infinity
// has s = NaN and codes 0.
#pragma once

#include "i8_core.h"

namespace qmm {

// Sixteen bytes of a row: eight values of 16 bits, four of 32.
template <int TYPE>
struct I8Raw {
  static constexpr int V = TYPE == kI8F32 ? 4 : 8;
  u32x4 u;

  __device__ __forceinline__ void load(const void* x, size_t at) { u = *(gptr<u32x4>)((gptr<char>)x + at * (16 / V)); }

  // The largest magnitude so far: bits without the sign order like magnitudes, NaN
  // above infinity (16-bit values two at a time).
  __device__ __forceinline__ void top(uint32_t& t) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == kI8F32) {
        const uint32_t v = u[i] & 0x7FFFFFFFu;
        t = v > t ? v : t;
      } else {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        t = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, t), __builtin_bit_cast(u16x2, u[i] & 0x7FFF7FFFu)));
      }
    }
  }

  // What top() collected, as the bits of one fp32.
  static __device__ __forceinline__ uint32_t top_bits(uint32_t t) {
    if constexpr (TYPE == kI8F32) return t;
    const uint32_t v = (t & 0xFFFF) > (t >> 16) ? t & 0xFFFF : t >> 16;
    return TYPE == kI8BF16 ? v << 16 : __float_as_uint(f16_bits_to_f32((uint16_t)v));
  }

  __device__ __forceinline__ float value(int i) const {
    if constexpr (TYPE == kI8F32) return __uint_as_float(u[i]);
    const uint32_t w = u[i / 2];
    if constexpr (TYPE == kI8F16) return f16_bits_to_f32((uint16_t)(i % 2 ? w >> 16 : w));
    return __uint_as_float(i % 2 ? w & 0xFFFF0000u : w << 16);
  }
};

// Scale of a row from the bits of its largest magnitude; rows of 0 and NaN have codes 0.
__device__ __forceinline__ float i8_scale(uint32_t top) {
  if (top >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  if (top < 0x04000000u) return 0.0f;  // 2^-119
  return __fdiv_rn(__uint_as_float(top), 127.0f);
}

__device__ __forceinline__ int i8_round(float x, float s, float inv) {
  const float n = rintf(x * inv);
  const float d = 2.0f * fmaf(-n, s, x);
  const int i = (int)n;
  const int up = d > s || (d == s && (i & 1));
  const int down = d < -s || (d == -s && (i & 1));
  return i + up - down;
}

// The codes of a Raw, four a word.  x inv + 1.5 * 2^23 has the nearest whole number in its
// low bits (the low byte is the code) and gives it back by a subtraction; where a
// remainder reaches s / 2 (a tie, or a neighbour) all are rounded by the rule.
template <int TYPE>
__device__ __forceinline__ void i8_codes(const I8Raw<TYPE>& raw, float s, float inv, uint32_t (&q)[I8Raw<TYPE>::V / 4]) {
  constexpr int W = I8Raw<TYPE>::V / 4;
  constexpr float kWhole = 12582912.0f;
  float worst = 0.0f;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    uint32_t t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = raw.value(4 * w + j);
      const float f = fmaf(x, inv, kWhole);
      worst = fmaxf(worst, fabsf(fmaf(-(f - kWhole), s, x)));
      t[j] = __float_as_uint(f);
    }
    q[w] = __builtin_amdgcn_perm(t[1], t[0], 0x0C0C0400u) | __builtin_amdgcn_perm(t[3], t[2], 0x04000C0Cu);
  }
  if (2.0f * worst < s) return;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    q[w] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) q[w] |= (uint32_t)(i8_round(raw.value(4 * w + j), s, inv) & 0xFF) << (8 * j);
  }
}

// Codes of a Raw at `to` (global or LDS); none in a row of scale 0 or NaN.
template <int TYPE>
__device__ __forceinline__ void i8_put(void* to, const I8Raw<TYPE>& raw, float s, float inv) {
  uint32_t q[I8Raw<TYPE>::V / 4] = {};
  if (s > 0.0f) i8_codes<TYPE>(raw, s, inv, q);
  if constexpr (I8Raw<TYPE>::V == 8) *static_cast<u32x2*>(to) = u32x2{q[0], q[1]};
  else *static_cast<uint32_t*>(to) = q[0];
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
