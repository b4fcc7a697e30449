// The tile of the products in 8-bit integers: codes of weights times codes of
// activations on the matrix cores,
//     C[n, m] = sum_k W[n, k] X[m, k]      (int32, exact: k <= 131008)
// Both operands are rows of bytes along k, so both go the same way: 128 bytes
// of k (one line of a row) a step, copied from global memory into a ring of
// LDS stages without passing through registers, and read back from there as
// the operands of v_mfma_i32_32x32x32_i8 (lane l: row l % 32, 16 bytes of k at
// 16 (l / 32)).
//
// Banks.  A row of a stage is 128 bytes, half of the 64 banks, so 32 lanes that
// read one 16-byte column would meet on few banks.  The piece c (of 8) of row
// r therefore stands at place c ^ ((r / 2) % 8): the copy writes LDS in lane
// order, so each lane fetches the piece that belongs at its place (within the
// same line of memory), and the reading lane undoes it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "qmm_device.h"

namespace qmm {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

constexpr int kI8Step = 128;  // bytes of k a step
constexpr int kI8Pieces = kI8Step / 16;

// A buffer descriptor of all that follows `base` (the same in every lane):
// every access of the tile is inside its operand by construction.
__device__ __forceinline__ i32x4 i8_rows(const void* base) {
  const uint64_t a = (uint64_t)base;
  return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
               __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32) & 0xFFFF), -1, 0x00020000};
}

// 16 bytes a lane from base + voff + soff straight into LDS at lds + 16 * lane.
// It has no output register; what it wrote may be read after i8_join.  (The
// builtin of the same instruction makes the compiler wait for every copy in
// flight before any LDS read, which undoes the ring.)  s_nop: a scalar register
// that a vector instruction has written may be read by a vector memory
// instruction five wait states later.
__device__ __forceinline__ void i8_copy(uint32_t lds, i32x4 base, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(base), "s"(soff)
               : "memory");
}

// All but this wave's last N copies have landed, its LDS reads are back, and
// the other waves' likewise.
template <int N>
__device__ __forceinline__ void i8_join() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// BM rows of X by BN rows of W on WM x WN waves, a ring of ST stages.
template <int BM_, int BN_, int WM_, int WN_, int ST_>
struct I8Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, ST = ST_;
  static constexpr int WAVES = WM * WN;
  static constexpr int THREADS = 64 * WAVES;
  static constexpr int TM = BM / WM / 32;  // blocks of 32 x 32 a wave
  static constexpr int TN = BN / WN / 32;
  static constexpr int CA = BM / 8 / WAVES;  // copies a wave and step: 8 rows each
  static constexpr int CB = BN / 8 / WAVES;
  static constexpr int STAGE = (BM + BN) * kI8Step;
  static constexpr int LDS = ST * STAGE;
  static_assert(BM % (32 * WM) == 0 && BN % (32 * WN) == 0, "whole blocks");
  static_assert(WAVES % 2 == 0 && BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0, "whole copies");
  static_assert((ST - 2) * (CA + CB) <= 63 && ST >= 2, "vmcnt counts to 63");
};

// One tile.  x_row(i) is the row of x at `xbase` that stands in row i of the
// tile, w_row(i) likewise (any valid row where the tile reaches past the
// operand: what it gives is not stored); steps [s0, s1) of k.
// acc[i][j]: block of X rows i, W rows j of the wave; lane l, register r hold
// the product of W row 8 (r / 4) + 4 (l / 32) + r % 4 and X row l % 32.
// GATED: the tile's BN rows of W are BN / 2 at `wbase` and as many at `wbase2`,
// and of a wave's TN blocks the first half is the former's.
template <class S, bool GATED, class XRow, class WRow>
__device__ __forceinline__ void i8_tile(const int8_t* xbase, XRow x_row, const int8_t* wbase, const int8_t* wbase2,
                                        WRow w_row, int k, int s0, int s1, char* lds, i32x16 (&acc)[S::TM][S::TN]) {
  static_assert(!GATED || (S::TN % 2 == 0 && S::CB % 2 == 0), "halves of whole blocks and copies");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const i32x4 xr = i8_rows(xbase), wr = i8_rows(wbase), wr2 = i8_rows(wbase2);
  // the copies: 8 rows each, of which this lane takes one piece
  const uint32_t piece = (lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7);
  uint32_t xo[S::CA], wo[S::CB];
#pragma unroll
  for (int j = 0; j < S::CA; ++j) xo[j] = (uint32_t)x_row((j * S::WAVES + wave) * 8 + (lane >> 3)) * (uint32_t)k + piece * 16;
#pragma unroll
  for (int j = 0; j < S::CB; ++j) {
    const int i = (j * S::WAVES + wave) * 8 + (lane >> 3);
    wo[j] = (uint32_t)w_row(GATED && j >= S::CB / 2 ? i - S::BN / 2 : i) * (uint32_t)k + piece * 16;
  }
  const uint32_t ring = __builtin_amdgcn_readfirstlane(lds_address(lds));
  // past the end of k the last step reads the row's last piece again; the
  // operands of X are set to zero there
  const int whole = k / kI8Step;            // steps that are whole
  const int pieces = (k % kI8Step) / 16;    // pieces of the step behind them
  const uint32_t back = (int)piece >= pieces ? (piece - (pieces - 1)) * 16 : 0;

  auto copy = [&](int step, int stage) {
    const uint32_t at = ring + stage * S::STAGE + wave * 1024;
    const uint32_t less = step < whole ? 0 : back;
    const uint32_t soff = (uint32_t)step * kI8Step;
#pragma unroll
    for (int j = 0; j < S::CA; ++j) i8_copy(at + j * S::WAVES * 1024, xr, xo[j] - less, soff);
#pragma unroll
    for (int j = 0; j < S::CB; ++j) i8_copy(at + S::BM * kI8Step + j * S::WAVES * 1024, GATED && j >= S::CB / 2 ? wr2 : wr, wo[j] - less, soff);
  };

  const int r = lane & 31, h = lane >> 5;
  const int key = (r >> 1) & 7;
  const char* xs = lds + (wm * S::TM * 32 + r) * kI8Step;
  constexpr int TC = GATED ? S::TN / 2 : S::TN;
  const char* ws = lds + (S::BM + wn * TC * 32 + r) * kI8Step;
  auto multiply = [&](int stage, auto masked, int valid) {
    const int at = stage * S::STAGE;
#pragma unroll
    for (int q = 0; q < kI8Step / 32; ++q) {
      const int o = at + (((2 * q + h) ^ key) << 4);
      i32x4 a[S::TN], b[S::TM];
#pragma unroll
      for (int j = 0; j < S::TN; ++j) a[j] = *reinterpret_cast<const i32x4*>(ws + o + (j < TC ? j * 32 : S::BN / 2 + (j - TC) * 32) * kI8Step);
#pragma unroll
      for (int i = 0; i < S::TM; ++i) b[i] = *reinterpret_cast<const i32x4*>(xs + o + i * 32 * kI8Step);
      if constexpr (decltype(masked)::value) {
        if (2 * q + h >= valid)
#pragma unroll
          for (int i = 0; i < S::TM; ++i) b[i] = i32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < S::TM; ++i)
#pragma unroll
        for (int j = 0; j < S::TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[j], b[i], acc[i][j], 0, 0, 0);
    }
  };
  using Plain = std::false_type;
  using Masked = std::true_type;

#pragma unroll
  for (int s = 0; s < S::ST - 1; ++s)
    if (s0 + s < s1) copy(s0 + s, s);
  int stage = 0;
  for (int s = s0; s < s1; ++s) {
    if (s + S::ST - 2 < s1) i8_join<(S::ST - 2) * (S::CA + S::CB)>();
    else i8_join<0>();
    if (s + S::ST - 1 < s1) copy(s + S::ST - 1, stage == 0 ? S::ST - 1 : stage - 1);
    if (s < whole) multiply(stage, Plain{}, 0);
    else multiply(stage, Masked{}, pieces);
    stage = stage == S::ST - 1 ? 0 : stage + 1;
  }
}

// ------------------------------------------------------------- the scales
// y = fp32(C) sx sw (+ bias), each step rounded to fp32: off by at most 3 half
// steps (the int32 sum, two products; a sum with the bias one more) and, in
// 16 bits, the last rounding.

enum { kI8F32, kI8F16, kI8BF16, kI8Codes };

__device__ __forceinline__ uint16_t i8_bf16(float v) {  // round to nearest even; NaN stays NaN
  const uint32_t u = __float_as_uint(v);
  if (v != v) return (uint16_t)((u >> 16) | 0x40);
  return (uint16_t)((u + 0x7FFF + ((u >> 16) & 1)) >> 16);
}

__device__ __forceinline__ uint16_t i8_f16(float v) { return __builtin_bit_cast(uint16_t, (half_t)v); }

__device__ __forceinline__ float i8_silu(float g) { return g / (1.0f + __expf(-g)); }

// Four neighbouring columns [c, c + 4) of a row, of which `have` exist; wide:
// the row's address at c takes one store.
__device__ __forceinline__ void i8_store(void* y, size_t at, int type, const float (&v)[4], int have, bool wide) {
  if (type == kI8F32) {
    float* o = static_cast<float*>(y) + at;
    if (wide && have >= 4) *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
    else
#pragma unroll
      for (int i = 0; i < 4; ++i) if (i < have) o[i] = v[i];
    return;
  }
  uint16_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = type == kI8F16 ? i8_f16(v[i]) : i8_bf16(v[i]);
  uint16_t* o = static_cast<uint16_t*>(y) + at;
  if (wide && have >= 4) *reinterpret_cast<uint2*>(o) = make_uint2(b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16);
  else
#pragma unroll
    for (int i = 0; i < 4; ++i) if (i < have) o[i] = b[i];
}

}  // namespace qmm
