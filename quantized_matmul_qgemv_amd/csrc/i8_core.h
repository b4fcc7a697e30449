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

// A result is rounded after each scale and again after the bias, by whichever way
// it is computed: no product may be drawn into the addition behind it, here and in
// what includes this.
#pragma clang fp contract(off)

namespace qmm {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

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
// instruction five wait states later.  The compiler holds m0 for its own and warns of
// every asm that names it, once for each copy of the code; nothing else in these
// kernels uses it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void i8_copy(uint32_t lds, i32x4 base, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(base), "s"(soff)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// All but this wave's last N copies have landed.
template <int N>
__device__ __forceinline__ void i8_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// This wave's LDS reads are back, and the other waves are here too.
__device__ __forceinline__ void i8_meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory"); }

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// BM rows of X by BN rows of W on WM x WN waves, a ring of ST stages of a line
// (BK bytes) of k.
template <int BM_, int BN_, int WM_, int WN_, int ST_>
struct I8Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, ST = ST_, BK = 128;
  static constexpr int WAVES = WM * WN;
  static constexpr int THREADS = 64 * WAVES;
  static constexpr int TM = BM / WM / 32;  // blocks of 32 x 32 a wave
  static constexpr int TN = BN / WN / 32;
  static constexpr int PIECES = BK / 16;       // of 16 bytes, of a row
  static constexpr int RC = 64 / PIECES;       // rows a copy
  static constexpr int CX = BM / RC;           // copies a step: X's, then W's,
  static constexpr int CW = BN / RC;
  static constexpr int EACH = (CX + CW) / WAVES;  // dealt to the waves in turn
  static constexpr int STAGE = (BM + BN) * BK;
  static constexpr int LDS = ST * STAGE;
  static_assert(BM % (32 * WM) == 0 && BN % (32 * WN) == 0, "whole blocks");
  static_assert(BM % RC == 0 && BN % RC == 0 && WAVES % 2 == 0 && CX % WAVES == 0 && CW % WAVES == 0, "whole copies");
  static_assert((ST - 1) * EACH <= 63 && ST >= 2, "vmcnt counts to 63");
};

// Where piece c of row r stands in its row of a stage: XOR with this.
__device__ __forceinline__ int i8_key(int r) { return (r >> 1) & 7; }

// One tile.  x_row(i) is the row of x at `xbase` that stands in row i of the
// tile, w_row(i) likewise (any valid row where the tile reaches past the
// operand: what it gives is not stored); steps [s0, s1) of k.
// acc[i][j]: block of X rows i, W rows j of the wave; lane l, register r hold
// the product of W row 8 (r / 4) + 4 (l / 32) + r % 4 and X row l % 32.
// GATED: of each 32 of the tile's BN rows of W 16 are at `wbase` (gate) and the
// same 16 at `wbase2` (up), so that both products of an output stand in one
// lane, eight registers apart.
// `behind` is called behind the first copies.
template <class S, bool GATED, class XRow, class WRow, class Behind>
__device__ __forceinline__ void i8_tile(const int8_t* xbase, XRow x_row, const int8_t* wbase, const int8_t* wbase2,
                                        WRow w_row, int k, int s0, int s1, char* lds, i32x16 (&acc)[S::TM][S::TN],
                                        Behind behind) {
  // 16 rows are 2 copies: which base a copy has is its wave's alone
  static_assert(!GATED || S::WAVES % 4 == 0, "a wave's copies are all gate's or all up's");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const i32x4 xr = i8_rows(xbase), wr = i8_rows(GATED && (wave & 2) ? wbase2 : wbase);
  // the copies: RC rows each, of which this lane takes one piece (its key is the
  // same in all: they are an even number of waves apart)
  const int mine = lane / S::PIECES;
  const int piece = (lane % S::PIECES) ^ i8_key(wave * S::RC + mine);
  uint32_t from[S::EACH];
#pragma unroll
  for (int j = 0; j < S::EACH; ++j) {
    int i = (j * S::WAVES + wave) * S::RC + mine;
    if (j * S::WAVES < S::CX) {
      i = x_row(i);
    } else {
      i -= S::BM;
      i = w_row(GATED ? i / 32 * 16 + i % 16 : i);
    }
    from[j] = (uint32_t)i * (uint32_t)k + piece * 16;
  }
  const uint32_t ring = __builtin_amdgcn_readfirstlane(lds_address(lds));
  // past the end of k the last step reads the row's last piece again; the
  // operands of X are set to zero there
  const int whole = k / S::BK;            // steps that are whole
  const int pieces = (k % S::BK) / 16;    // pieces of the step behind them
  const uint32_t back = piece >= pieces ? (piece - (pieces - 1)) * 16 : 0;

  auto copy = [&](int step, int stage) {
    const uint32_t at = ring + stage * S::STAGE + wave * 1024;
    const uint32_t off = step < whole ? 0 : back;
    const uint32_t soff = (uint32_t)step * S::BK;
#pragma unroll
    for (int j = 0; j < S::EACH; ++j) i8_copy(at + j * S::WAVES * 1024, j * S::WAVES < S::CX ? xr : wr, from[j] - off, soff);
  };
  // all but the copies of the last N steps have landed, in every wave
  auto join = [&](auto n) {
    constexpr int N = decltype(n)::value;
    i8_wait<N * S::EACH>();
    i8_meet();
  };
  using None = std::integral_constant<int, 0>;

  const int r = lane & 31, h = lane >> 5;
  const int key = i8_key(r);
  const char* xs = lds + (wm * S::TM * 32 + r) * S::BK;
  const char* ws = lds + (S::BM + wn * S::TN * 32 + r) * S::BK;
  // a step's products of 32 bytes of k; the operands of the next one are read
  // while one multiplies
  i32x4 a[2][S::TN], b[2][S::TM];
  auto read = [&](int stage, int q, i32x4 (&a)[S::TN], i32x4 (&b)[S::TM]) {
    const int o = stage * S::STAGE + (((2 * q + h) ^ key) << 4);
#pragma unroll
    for (int j = 0; j < S::TN; ++j) a[j] = *reinterpret_cast<const i32x4*>(ws + o + j * 32 * S::BK);
#pragma unroll
    for (int i = 0; i < S::TM; ++i) b[i] = *reinterpret_cast<const i32x4*>(xs + o + i * 32 * S::BK);
  };
  auto multiply = [&](const i32x4 (&a)[S::TN], const i32x4 (&b)[S::TM]) {
#pragma unroll
    for (int i = 0; i < S::TM; ++i)
#pragma unroll
      for (int j = 0; j < S::TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[j], b[i], acc[i][j], 0, 0, 0);
  };
  constexpr int Q = S::BK / 32;

#pragma unroll
  for (int s = 0; s < S::ST; ++s)
    if (s0 + s < s1) copy(s0 + s, s);
  behind();
  if (s0 + S::ST <= s1) join(std::integral_constant<int, S::ST - 1>{});
  else join(None{});
  read(0, 0, a[0], b[0]);
  int stage = 0;
  for (int s = s0; s + 1 < s1; ++s) {
#pragma unroll
    for (int q = 0; q < Q - 1; ++q) {
      read(stage, q + 1, a[(q + 1) & 1], b[(q + 1) & 1]);
      __builtin_amdgcn_sched_barrier(0);
      multiply(a[q & 1], b[q & 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
    // the stage is read: its place takes the copy of ST steps on, and the next
    // stage's first operands come while the last product runs
    if (s + S::ST <= s1) join(std::integral_constant<int, S::ST - 2>{});
    else join(None{});
    if (s + S::ST < s1) copy(s + S::ST, stage);
    stage = stage == S::ST - 1 ? 0 : stage + 1;
    read(stage, 0, a[0], b[0]);
    __builtin_amdgcn_sched_barrier(0);
    multiply(a[(Q - 1) & 1], b[(Q - 1) & 1]);
    __builtin_amdgcn_sched_barrier(0);
  }
  const int valid = s1 <= whole ? S::PIECES : pieces;  // of the last step
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    if (q + 1 < Q) read(stage, q + 1, a[(q + 1) & 1], b[(q + 1) & 1]);
    if (2 * q + h >= valid)
#pragma unroll
      for (int i = 0; i < S::TM; ++i) b[q & 1][i] = i32x4{0, 0, 0, 0};
    multiply(a[q & 1], b[q & 1]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// ------------------------------------------------------------- the scales
// y = fp32(C) sx sw (+ bias), each step rounded to fp32: off by at most 3 half
// steps (the int32 sum, two products; a sum with the bias one more) and, in
// 16 bits, the last rounding.

enum { kI8F32, kI8F16, kI8BF16, kI8Codes };

// Two neighbours in 16 bits, each rounded to nearest even.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t i8_pair(int type, float lo, float hi) {
  if (type == kI8F16) return as_u32(half2_t{(half_t)lo, (half_t)hi});
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
}

__device__ __forceinline__ float i8_silu(float g) { return g / (1.0f + __expf(-g)); }

// The scales of a tile's rows and columns, its bias and where its rows go in y,
// loaded before the product and used behind it.
template <class S>
struct I8Scales {
  static constexpr int NX = (S::BM + S::THREADS - 1) / S::THREADS, NW = (S::BN + S::THREADS - 1) / S::THREADS;
  int32_t row[NX];
  float x[NX], w[NW], b[NW];

  template <class R, class X, class W, class B>
  __device__ __forceinline__ void load(R y_row, X xs, W ws, B bias) {
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int r = threadIdx.x + i * S::THREADS;
      row[i] = r < S::BM ? y_row(r) : 0;
      x[i] = r < S::BM ? xs(r, row[i]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const int c = threadIdx.x + i * S::THREADS;
      w[i] = c < S::BN ? ws(c) : 0.0f;
      b[i] = c < S::BN ? bias(c) : 0.0f;
    }
  }
};

constexpr int kI8OutRow = 144;  // bytes of a row of 128 in LDS: neighbours stand 4 banks on

// The tile's results: scaled, rounded, and by way of LDS (32 rows of 128 bytes
// a wave at a time) out in whole lines, columns [n0, n0 + cols) of n.
// SUMS: the int32 sums as they are.
template <class S, bool GATED, bool SUMS>
__device__ __forceinline__ void i8_finish(const i32x16 (&acc)[S::TM][S::TN], const I8Scales<S>& scales, char* lds, void* y,
                                          int type, bool biased, int n, int n0, int rows, int cols) {
  constexpr int OC = GATED ? 16 : 32;  // output columns of a block
  float* xs = reinterpret_cast<float*>(lds);
  float* ws = xs + S::BM;
  float* bs = ws + S::BN;
  int32_t* ys = reinterpret_cast<int32_t*>(bs + S::BN);
  constexpr int FIRST = (2 * S::BM + 2 * S::BN) * 4;
  static_assert(FIRST % 16 == 0 && FIRST + S::WAVES * 32 * kI8OutRow <= S::LDS, "fits the ring's place");
  __syncthreads();
#pragma unroll
  for (int i = 0; i < I8Scales<S>::NX; ++i) {
    const int r = threadIdx.x + i * S::THREADS;
    if (r < S::BM) {
      xs[r] = scales.x[i];
      ys[r] = scales.row[i];
    }
  }
#pragma unroll
  for (int i = 0; i < I8Scales<S>::NW; ++i) {
    const int c = threadIdx.x + i * S::THREADS;
    if (c < S::BN) {
      ws[c] = scales.w[i];
      bs[c] = scales.b[i];
    }
  }
  __syncthreads();
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int r = lane & 31, h = lane >> 5;
  char* out = lds + FIRST + wave * 32 * kI8OutRow;
  const int width = SUMS || type == kI8F32 ? 4 : 2;
  const int blocks = 128 / (OC * width);  // of OC columns in 128 bytes
  // whole pieces of 16 bytes where every row starts on one
  const bool wide = (size_t)n * width % 16 == 0 && ((uintptr_t)y & 15) == 0;
#pragma unroll
  for (int i = 0; i < S::TM; ++i) {
    const int r0 = (wm * S::TM + i) * 32;
    if (r0 >= rows) break;
    const float sx = xs[r0 + r];
#pragma unroll
    for (int j = 0; j < S::TN; ++j) {
      const int c0 = (wn * S::TN + j) * 32;  // in W's rows
      const int place = j % blocks;
#pragma unroll
      for (int q = 0; q < OC / 8; ++q) {
        const int c = 8 * q + 4 * h;
        const float4_t sw = *reinterpret_cast<const float4_t*>(ws + c0 + c);
        float4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = SUMS ? __int_as_float(acc[i][j][4 * q + e]) : (float)acc[i][j][4 * q + e] * sx * sw[e];
        if constexpr (GATED) {
          const float4_t su = *reinterpret_cast<const float4_t*>(ws + c0 + 16 + c);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = i8_silu(v[e]) * ((float)acc[i][j][4 * q + 8 + e] * sx * su[e]);
        } else if (biased) {
          v += *reinterpret_cast<const float4_t*>(bs + c0 + c);
        }
        char* o = out + r * kI8OutRow + (place * OC + c) * width;
        if (width == 4) *reinterpret_cast<float4_t*>(o) = v;
        else *reinterpret_cast<u32x2*>(o) = u32x2{i8_pair(type, v[0], v[1]), i8_pair(type, v[2], v[3])};
      }
      if (place + 1 < blocks && j + 1 < S::TN) continue;
      // what stands in LDS: columns [s0, s0 + have) of the tile
      const int s0 = (wn * S::TN + j - place) * OC;
      const int most = OC * (place + 1);
      const int have = cols - s0 < most ? cols - s0 : most;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (wide) {
        const int piece = lane & 7;
        const int c = piece * (16 / width);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int rr = t * 8 + (lane >> 3);
          if (r0 + rr < rows && c < have) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(out + rr * kI8OutRow + piece * 16);
            const size_t at = (size_t)ys[r0 + rr] * n + n0 + s0 + c;
            *reinterpret_cast<u32x4*>(static_cast<char*>(y) + at * width) = v;
          }
        }
      } else {
        // number by number, a whole row (two of 4 bytes) of the 128 bytes at a time
        const int two = width == 4;
        const int c = two ? r : lane, step = 1 + two;
        const bool in = c < have;
        const char* from = out + (two ? h : 0) * kI8OutRow + c * width;
        const size_t first = (size_t)n0 + s0 + c;
#pragma unroll 4
        for (int t = 0; t < 32; t += step) {
          const int rr = r0 + t + (two ? h : 0);
          if (!in || rr >= rows) continue;
          const size_t at = (size_t)ys[rr] * n + first;
          if (two) static_cast<uint32_t*>(y)[at] = *reinterpret_cast<const uint32_t*>(from + t * kI8OutRow);
          else static_cast<uint16_t*>(y)[at] = *reinterpret_cast<const uint16_t*>(from + t * kI8OutRow);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }
}

}  // namespace qmm
