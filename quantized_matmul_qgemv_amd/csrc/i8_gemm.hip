// Products in 8-bit integers (include/qmm.h, qmm_i8_*): rows rounded to 8 bits
// with a scale each, and y = sx sw (codes of x) (codes of w)^T [+ bias].
#include <stdlib.h>

#include "i8_core.h"
#include "qmm_internal.h"

namespace qmm {

// ---------------------------------------------------------------- rounding
// s = fp32(max |x| / 127), q = rint(x / s): which whole number is nearest to
// the exact quotient, ties to even.  n = rint(x * (1 / s)) is that number or its
// neighbour; the remainder x - n s is a multiple of half a unit in the last
// place of s and not much larger than s / 2, so one fma gives it exactly and it
// decides.  A row whose largest magnitude is below 2^-119 (where s would
// leave fp32's normal range) has s = 0 and codes 0; one with a NaN or infinity
// has s = NaN and codes 0.
//
// Sixteen values a lane: one 16-byte store of codes, two (16-bit x) or four
// (fp32 x) 16-byte loads.  A row is taken by WPR waves, which hold it in registers
// up to 16 * 64 * WPR * R values; what is longer is read a second time.

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

constexpr int kI8RoundThreads = 256;

// WPR waves a row (1 or 4), R chunks of 16 values a lane held.
template <int WPR, int R>
__global__ __launch_bounds__(kI8RoundThreads) void i8_quantize_kernel(I8QuantizeArgs g) {
  __shared__ uint32_t tops[4];
  int b = blockIdx.x, job = 0;
  while (job + 1 < g.count && b >= g.job[job + 1].first) ++job;
  const I8QuantizeJob& jb = g.job[job];
  b -= jb.first;
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int row = WPR == 1 ? b * 4 + wave : b;
  if (row >= jb.m) return;  // whole waves; with WPR = 4 whole workgroups
  const int place = WPR == 1 ? lane : threadIdx.x;
  constexpr int SPAN = 64 * WPR;
  const int chunks = jb.k / 16;
  const size_t at = (size_t)row * jb.k;
  float v[R][16];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int c = place + i * SPAN;
    if (c < chunks) i8_load16(jb.x, at + (size_t)c * 16, jb.type, v[i]);
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (place + i * SPAN < chunks) top = i8_top(v[i], top);
  for (int c = place + R * SPAN; c < chunks; c += SPAN) {
    float u[16];
    i8_load16(jb.x, at + (size_t)c * 16, jb.type, u);
    top = i8_top(u, top);
  }
  top = wave_umax(top);
  if constexpr (WPR > 1) {
    if (lane == 0) tops[wave] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) top = tops[i] > top ? tops[i] : top;
  }
  const float s = i8_scale(top);
  if (place == 0) jb.scales[row] = s;
  const bool some = s > 0.0f;
  const float inv = some ? 1.0f / s : 0.0f;
  auto store = [&](int c, const float (&u)[16]) {
    i32x4 q = some ? i8_round16(u, s, inv) : i32x4{0, 0, 0, 0};
    *reinterpret_cast<i32x4*>(jb.codes + at + (size_t)c * 16) = q;
  };
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (place + i * SPAN < chunks) store(place + i * SPAN, v[i]);
  for (int c = place + R * SPAN; c < chunks; c += SPAN) {
    float u[16];
    i8_load16(jb.x, at + (size_t)c * 16, jb.type, u);
    store(c, u);
  }
}

hipError_t launch_i8_quantize(I8QuantizeArgs& g, hipStream_t st) {
  // one wave a row where the row fits its registers
  long most = 0;
  for (int i = 0; i < g.count; ++i) most = g.job[i].k > most ? g.job[i].k : most;
  const int wpr = most <= 4096 ? 1 : 4;
  long blocks = 0;
  for (int i = 0; i < g.count; ++i) {
    g.job[i].first = (int)blocks;
    blocks += wpr == 1 ? (g.job[i].m + 3) / 4 : g.job[i].m;
  }
  if (blocks == 0) return hipSuccess;
  if (wpr == 1 && most <= 1024) hipLaunchKernelGGL((i8_quantize_kernel<1, 1>), dim3(blocks), dim3(kI8RoundThreads), 0, st, g);
  else if (wpr == 1) hipLaunchKernelGGL((i8_quantize_kernel<1, 4>), dim3(blocks), dim3(kI8RoundThreads), 0, st, g);
  else hipLaunchKernelGGL((i8_quantize_kernel<4, 4>), dim3(blocks), dim3(kI8RoundThreads), 0, st, g);
  return hipGetLastError();
}

// ----------------------------------------------------------------- products

constexpr int kI8Band = 8;

template <class S>
__global__ __launch_bounds__(S::THREADS) void i8_gemm_kernel(I8GemmArgs g) {
  __shared__ __attribute__((aligned(16))) char lds[S::LDS];
  // workgroups are dealt to the 8 XCDs in turn: each XCD gets a run of tiles
  const int each = gridDim.x / 8, more = gridDim.x % 8, xcd = blockIdx.x % 8;
  int b = xcd * each + (xcd < more ? xcd : more) + blockIdx.x / 8, which = 0;
  while (which + 1 < g.count && b >= g.p[which + 1].first) ++which;
  const I8Problem& p = g.p[which];
  b -= p.first;
  const int tiles_m = (p.m + S::BM - 1) / S::BM, tiles_n = (p.n + S::BN - 1) / S::BN;
  // bands of kI8Band row tiles, down each column of a band
  const int band = b / (kI8Band * tiles_n), in = b - band * kI8Band * tiles_n;
  const int high = tiles_m - band * kI8Band < kI8Band ? tiles_m - band * kI8Band : kI8Band;
  const int tm = band * kI8Band + in % high, tn = in / high;
  const int m0 = tm * S::BM, n0 = tn * S::BN;
  const int rows = p.m - m0 < S::BM ? p.m - m0 : S::BM;
  const int cols = p.n - n0 < S::BN ? p.n - n0 : S::BN;
  i32x16 acc[S::TM][S::TN];
#pragma unroll
  for (int i = 0; i < S::TM; ++i)
#pragma unroll
    for (int j = 0; j < S::TN; ++j) acc[i][j] = i32x16{};
  I8Scales<S> scales;
  scales.load([&](int i) { return m0 + (i < rows ? i : rows - 1); }, [&](int, int row) { return p.sx[row]; },
              [&](int i) { return p.sw[n0 + (i < cols ? i : cols - 1)]; },
              [&](int i) { return p.bias ? p.bias[n0 + (i < cols ? i : cols - 1)] : 0.0f; });
  i8_tile<S, false>(p.x + (size_t)m0 * p.k, [&](int i) { return i < rows ? i : rows - 1; }, p.w + (size_t)n0 * p.k,
                    p.w, [&](int i) { return i < cols ? i : cols - 1; }, p.k, 0, (p.k + S::BK - 1) / S::BK, lds, acc);
  i8_finish<S, false>(acc, scales, lds, p.y, p.y_type, p.bias != nullptr, p.n, n0, rows, cols);
}

template <class S>
static hipError_t launch_shape(I8GemmArgs& g, hipStream_t st) {
  long tiles = 0;
  for (int i = 0; i < g.count; ++i) {
    g.p[i].first = (int)tiles;
    tiles += (long)((g.p[i].m + S::BM - 1) / S::BM) * ((g.p[i].n + S::BN - 1) / S::BN);
  }
  if (tiles == 0) return hipSuccess;
  hipLaunchKernelGGL((i8_gemm_kernel<S>), dim3((unsigned)tiles), dim3(S::THREADS), 0, st, g);
  return hipGetLastError();
}

// Tile shapes and what a tile costs alone on its CU (shapes of 160 KB / LDS > 1:
// with that many beside it): `fixed` us and `step` us for 128 bytes of k.  Measured on
// products with cold weights (m x n x k, us with about 4 us of launch):
//   shape        512x2560x4096  512x9728x2560  1024x9728x2560  2048x2560x9728  2048x9728x2560  16384x2560x9728
//   64 x 64               22.9           35.1            58.8            97.1             103              692
//   64 x 128              19.9           41.1            64.5           101.8             123                -
//   128 x 128             24.4           38.4            54.9            94.2              87              456
//   128 x 192             29.0           25.7            47.0            62.6              81                -
//   256 x 192             45.7           38.8            39.6           102.9              74              432
//   256 x 256             54.8           44.7            45.1           123.0              80              403
//   256 x 320             62.6           49.2            49.7           137.1              57              349
// A larger tile moves fewer bytes for its products; which one is best is mostly a
// matter of how evenly its tiles fall on the 256 CUs.
struct I8Choice {
  int bm, bn, at_once;  // tiles a CU holds
  float fixed, step;
};
constexpr I8Choice kI8Choices[] = {
    {64, 64, 3, 3.0f, 0.55f},  {64, 128, 1, 3.0f, 0.45f},  {128, 128, 1, 4.0f, 0.60f}, {128, 192, 1, 5.0f, 0.75f},
    {256, 192, 1, 7.0f, 1.25f}, {256, 256, 1, 8.0f, 1.52f}, {256, 320, 1, 9.0f, 1.72f},
};
constexpr int kI8Shapes = sizeof(kI8Choices) / sizeof(kI8Choices[0]);

static int i8_choose(const I8GemmArgs& g) {
  if (const char* env = getenv("QMM_I8_FORCE")) {  // tuning sweeps and tests: a shape by its place
    const int f = atoi(env);
    if (f >= 0 && f < kI8Shapes) return f;
  }
  int best = 0;
  double least = 1e30;
  for (int c = 0; c < kI8Shapes; ++c) {
    const I8Choice& h = kI8Choices[c];
    double tiles = 0, steps = 0;
    for (int i = 0; i < g.count; ++i) {
      const double t = (double)((g.p[i].m + h.bm - 1) / h.bm) * ((g.p[i].n + h.bn - 1) / h.bn);
      tiles += t;
      steps += t * ((g.p[i].k + 127) / 128);
    }
    const double slots = 256.0 * h.at_once;
    const double rounds = (double)(long)((tiles + slots - 1) / slots);
    // fewer tiles than places: they share a CU with fewer others
    const double share = tiles < slots && h.at_once > 1 ? 0.5 + 0.5 * tiles / slots : 1.0;
    const double cost = rounds * (h.fixed + h.step * share * steps / tiles);
    if (cost < least) {
      least = cost;
      best = c;
    }
  }
  return best;
}

hipError_t launch_i8_gemm(I8GemmArgs& g, hipStream_t st) {
  switch (i8_choose(g)) {
    case 0: return launch_shape<I8Shape<64, 64, 2, 2, 3, 128>>(g, st);
    case 1: return launch_shape<I8Shape<64, 128, 2, 4, 6, 128>>(g, st);
    case 2: return launch_shape<I8Shape<128, 128, 2, 4, 3, 128>>(g, st);
    case 3: return launch_shape<I8Shape<128, 192, 4, 2, 3, 128>>(g, st);
    case 4: return launch_shape<I8Shape<256, 192, 4, 2, 2, 128>>(g, st);
    case 5: return launch_shape<I8Shape<256, 256, 2, 4, 2, 128>>(g, st);
    default: return launch_shape<I8Shape<256, 320, 4, 2, 2, 128>>(g, st);
  }
}

}  // namespace qmm
