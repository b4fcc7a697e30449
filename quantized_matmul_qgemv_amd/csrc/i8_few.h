// Products in 8-bit integers of few rows (a decode step): bound by the weights'
// bytes and by latency.  A wave takes 16 columns (or 16 of gate and the same of up)
// and a part of k: it loads those pieces of the 16 weight rows straight into the
// operand registers of v_mfma_i32_16x16x64_i8 (lane l: row l % 16, 16 bytes of k at
// 16 (l / 16)), a whole batch before the first product, and the partial sums of the
// `kw` waves that share the columns are joined in LDS.  x either is codes, or its
// rows are rounded by every workgroup for itself while its weights are on the way:
// loads come back in order, so x is asked for first and nothing may wait between
// the two, which is why x's type and the batch are fixed at compile time.
#pragma once

#include "i8_core.h"
#include "i8_round.h"

namespace qmm {

constexpr int kI8FewWaves = 8;
constexpr int kI8FewThreads = 64 * kI8FewWaves;
constexpr int kI8FewRows = 16;      // rows of a workgroup: those of one operand
constexpr int kI8FewHead = 256;     // bytes of LDS: scales of the rows, the waves' maxima
constexpr int kI8StageRows = 8;     // rows that a workgroup can round
constexpr int kI8StageHold = 32;    // values of a row a lane

// Waves that share a row when m rows are rounded by eight.
__host__ __device__ inline int i8_stage_group(int m) { return m == 1 ? 8 : m == 2 ? 4 : m <= 4 ? 2 : 1; }
inline bool i8_can_stage(int m, int k) {
  return m <= kI8StageRows && k <= 64 * kI8StageHold * i8_stage_group(m);
}

template <bool GATED>
constexpr int i8_few_sums() { return kI8FewWaves * 16 * (GATED ? 36 : 20) * 4; }

// Bytes of LDS for `rows` rows that are rounded (0: x is codes, of which each wave
// holds a batch of U slices), and for the sums.
template <int U, bool GATED>
size_t i8_few_lds(int rows, int k) {
  const size_t held = rows > 0 ? (size_t)rows * (k + 16) : (size_t)kI8FewWaves * 16 * (U * 64 + 16);
  const size_t sums = i8_few_sums<GATED>();
  return kI8FewHead + (held > sums ? held : sums);
}

// Waves that share 16 columns: 8 with few blocks, 2 with many.  us of a call with
// 8 / 4 / 2 (graph, weights from memory, fp16 x, one row): 9728 x 2560 (608 blocks): 9.3 /
// 12.2 / 11.8; 16384 x 1024 (1024): 8.0 / 7.4 / 6.4; 20480 x 2560 (1280): 13.4 / 17.2 /
// 18.7; 32752 x 1024 (2047): 12.9 / 10.4 / 9.3; 32752 x 2560: 19.0 / 21.9 / 20.3; 40960 x
// 1024 (2560): 15.0 / 11.9 / 11.5; 151936 x 1024 (9496): - / 34.7 / 32.0 (1: 39.8).  In
// between it is k that decides (short rows want 2, long ones 8) and 4 is seldom best of
// all but never far behind: up to 28 % behind 8 and 19 % behind 2.  4 rows, 6144 x 2560:
// 8.4 / 9.0 / 11.9.  Of codes 8 is best (16 rows, 9728 x 2560: 10.2 / 15.7 / 13.5).
inline int i8_few_kw(long blocks, bool codes) {
  return codes || blocks < 1024 ? 8 : blocks < 2048 ? 4 : 2;
}

struct I8FewTile {
  const int8_t* w;    // first of the workgroup's columns
  const int8_t* w2;   // GATED: up's
  const float* sw;    // at the same column
  const float* sw2;
  const float* bias;  // or null
  const void* x;
  const float* sx;    // null where x is rounded here
  void* y;
  int y_type, n, n0, cols, rows, k;
  int kw;             // waves that share 16 columns: 1, 2, 4 or 8
};

// rows <= 16 (rounded here: 8); cols <= 16 * 8 / kw.  TYPE: x's.  U: slices of 64 bytes
// of k a batch; LOOP: a wave's part of k may be more than one batch.
template <int U, bool LOOP, bool GATED, int TYPE, class XRow, class YRow>
__device__ __forceinline__ void i8_few(const I8FewTile& t, char* lds, XRow x_row, YRow y_row) {
  constexpr int NB = GATED ? 2 : 1;
  constexpr bool STAGED = TYPE != kI8Codes;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lk = (lane >> 4) * 16;
  float* sx = reinterpret_cast<float*>(lds);
  uint32_t* tops = reinterpret_cast<uint32_t*>(lds + 128);
  char* body = lds + kI8FewHead;
  const int k = t.k, kw = t.kw;
  const int block = wave / kw;  // of 16 columns
  const int slices = (k + 63) / 64, each = (slices + kw - 1) / kw;
  int s = wave % kw * each;
  const int end = s + each < slices ? s + each : slices;

  // x's rows, as they are
  using Raw = I8Raw<STAGED ? TYPE : kI8F32>;
  constexpr int HOLD = STAGED ? kI8StageHold / Raw::V : 1;
  Raw raw[HOLD];
  const int group = STAGED ? i8_stage_group(t.rows) : 8;
  const int place = (wave % group * 64 + lane) * Raw::V, span = 64 * group * Raw::V;
  const bool mine = STAGED && wave / group < t.rows;
  if constexpr (STAGED) {
    const size_t at = (size_t)x_row(mine ? wave / group : 0) * k;
#pragma unroll
    for (int i = 0; i < HOLD; ++i) raw[i].load(t.x, at + (place + i * span < k ? place + i * span : 0));
  } else if ((int)threadIdx.x < t.rows) {
    sx[threadIdx.x] = t.sx[x_row(threadIdx.x)];
  }

  gptr<int8_t> wp[NB];
  {
    const int c = block * 16 + li;
    const size_t at = (size_t)(c < t.cols ? c : t.cols - 1) * k;
    wp[0] = to_global(t.w) + at;
    if constexpr (GATED) wp[1] = to_global(t.w2) + at;
  }
  const int row = li < t.rows ? li : t.rows - 1;
  // codes of x are read along their rows and turned into operands by way of LDS
  // (16 rows, 9728 x 2560: 2.2 us less than straight into the operands)
  constexpr int XS = U * 64 + 16;  // bytes of a row of a batch
  char* held = body + wave * 16 * XS;
  uint32_t xo[STAGED ? 1 : U];
  if constexpr (!STAGED)
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int r = (i * 64 + lane) / (U * 4);
      xo[i] = (uint32_t)x_row(r < t.rows ? r : t.rows - 1) * (uint32_t)k;
    }

  struct Batch {
    i32x4 w[U][NB], x[STAGED ? 1 : U];
  };
  auto load = [&](Batch& b, int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int o = (s + u < end ? s + u : end - 1) * 64 + lk;  // past the end: the last slice once more, which is not used
      o = o >= 0 && o < k ? o : 0;
#pragma unroll
      for (int i = 0; i < NB; ++i) b.w[u][i] = *(gptr<i32x4>)(wp[i] + o);
    }
    if constexpr (!STAGED)
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int o = s * 64 + (i * 64 + lane) % (U * 4) * 16;
        b.x[i] = *(gptr<i32x4>)((gptr<char>)t.x + (xo[i] + (uint32_t)(o < k ? o : 0)));
      }
  };
  i32x4 acc[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) acc[i] = i32x4{0, 0, 0, 0};
  auto multiply = [&](const Batch& b, int s) {
    if constexpr (!STAGED) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int p = i * 64 + lane;
        *reinterpret_cast<i32x4*>(held + p / (U * 4) * XS + p % (U * 4) * 16) = b.x[i];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int o = (s + u) * 64 + lk;
      const bool in = s + u < end && o < k;
      i32x4 v;
      if constexpr (STAGED) v = *reinterpret_cast<const i32x4*>(body + row * (k + 16) + (in ? o : 0));
      else v = *reinterpret_cast<const i32x4*>(held + row * XS + u * 64 + lk);
      if (!in) v = i32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < NB; ++i) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b.w[u][i], v, acc[i], 0, 0, 0);
    }
    if constexpr (!STAGED) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  };
  Batch one, two;
  load(one, s);

  if constexpr (STAGED) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < HOLD; ++i) raw[i].top(top);
    top = wave_umax(Raw::top_bits(top));
    if (group > 1) {  // the same in every wave
      if (lane == 0) tops[wave] = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kI8FewWaves; ++i) {
        const uint32_t v = tops[i];
        top = i / group == wave / group && v > top ? v : top;
      }
    }
    const float scale = i8_scale(top);
    if (mine) {
      const int r = wave / group;
      if (place == 0) sx[r] = scale;
      const float inv = scale > 0.0f ? 1.0f / scale : 0.0f;
#pragma unroll
      for (int i = 0; i < HOLD; ++i)
        if (place + i * span < k) i8_put<TYPE>(body + r * (k + 16) + place + i * span, raw[i], scale, inv);
    }
    __syncthreads();
  }

  if constexpr (LOOP) {
    while (s < end) {
      load(two, s + U);
      multiply(one, s);
      s += U;
      if (s >= end) break;
      load(one, s + U);
      multiply(two, s);
      s += U;
    }
  } else {
    multiply(one, s);
  }
  __syncthreads();  // the codes are read: the sums take their place
  constexpr int LD = NB * 16 + 4;
  int32_t* part = reinterpret_cast<int32_t*>(body);
#pragma unroll
  for (int i = 0; i < NB; ++i)
    *reinterpret_cast<i32x4*>(part + (wave * 16 + li) * LD + i * 16 + (lane >> 4) * 4) = acc[i];
  __syncthreads();
  const int wide = 16 * (kI8FewWaves / kw);  // output columns of the workgroup
  for (int o = threadIdx.x; o < t.rows * wide; o += kI8FewThreads) {
    const int c = o % wide, m = o / wide;
    if (c >= t.cols) continue;
    const int32_t* from = part + (c / 16 * kw * 16 + m) * LD + c % 16;
    int32_t sum = 0, up = 0;
    for (int i = 0; i < kw; ++i) {
      sum += from[i * 16 * LD];
      if constexpr (GATED) up += from[i * 16 * LD + 16];
    }
    float v = (float)sum * sx[m] * t.sw[c];
    if constexpr (GATED) v = i8_silu(v) * ((float)up * sx[m] * t.sw2[c]);
    else if (t.bias) v += t.bias[c];
    const size_t at = (size_t)y_row(m) * t.n + t.n0 + c;
    if (t.y_type == kI8F32) static_cast<float*>(t.y)[at] = v;
    else static_cast<uint16_t*>(t.y)[at] = (uint16_t)i8_pair(t.y_type, v, v);
  }
}

}  // namespace qmm
