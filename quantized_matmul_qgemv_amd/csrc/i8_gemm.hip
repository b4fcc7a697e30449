// Products in 8-bit integers (include/qmm.h, qmm_i8_*): rows rounded to 8 bits
// with a scale each, and y = sx sw (codes of x) (codes of w)^T [+ bias].
#include <stdlib.h>

#include "i8_core.h"
#include "i8_few.h"
#include "i8_round.h"
#include "qmm_internal.h"

namespace qmm {

// ---------------------------------------------------------------- rounding
// A row is taken by WPR waves (1 or 4), which hold it in registers up to 16 R bytes a
// lane; what is longer is read a second time.

constexpr int kI8RoundThreads = 256;

template <int TYPE, int WPR, int R>
__global__ __launch_bounds__(kI8RoundThreads) void i8_quantize_kernel(I8QuantizeArgs g) {
  __shared__ uint32_t tops[4];
  using Raw = I8Raw<TYPE>;
  int b = blockIdx.x, job = 0;
  while (job + 1 < g.count && b >= g.job[job + 1].first) ++job;
  const I8QuantizeJob& jb = g.job[job];
  b -= jb.first;
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int row = WPR == 1 ? b * 4 + wave : b;
  if (row >= jb.m) return;  // whole waves; with WPR = 4 whole workgroups
  const int place = (WPR == 1 ? lane : threadIdx.x) * Raw::V, k = jb.k;
  constexpr int SPAN = 64 * WPR * Raw::V;
  const size_t at = (size_t)row * k;
  Raw raw[R];
#pragma unroll
  for (int i = 0; i < R; ++i) raw[i].load(jb.x, at + (place + i * SPAN < k ? place + i * SPAN : 0));  // the first again changes no maximum
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) raw[i].top(top);
  for (int c = place + R * SPAN; c < k; c += SPAN) {
    Raw more;
    more.load(jb.x, at + c);
    more.top(top);
  }
  top = wave_umax(Raw::top_bits(top));
  if constexpr (WPR > 1) {
    if (lane == 0) tops[wave] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) top = tops[i] > top ? tops[i] : top;
  }
  const float s = i8_scale(top);
  if (place == 0) jb.scales[row] = s;
  const float inv = s > 0.0f ? 1.0f / s : 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (place + i * SPAN < k) i8_put<TYPE>(jb.codes + at + place + i * SPAN, raw[i], s, inv);
  for (int c = place + R * SPAN; c < k; c += SPAN) {
    Raw more;
    more.load(jb.x, at + c);
    i8_put<TYPE>(jb.codes + at + c, more, s, inv);
  }
}

template <int TYPE, int WPR, int R>
static hipError_t launch_quantize_kernel(I8QuantizeArgs& g, hipStream_t st) {
  long blocks = 0;
  for (int i = 0; i < g.count; ++i) {
    g.job[i].first = (int)blocks;
    blocks += WPR == 1 ? (g.job[i].m + 3) / 4 : g.job[i].m;
  }
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL((i8_quantize_kernel<TYPE, WPR, R>), dim3((unsigned)blocks), dim3(kI8RoundThreads), 0, st, g);
  return hipGetLastError();
}

// One wave a row where it holds the row and there are rows enough to fill the chip,
// four otherwise; two pieces a lane where that is enough.
template <int TYPE>
static hipError_t launch_quantize_type(I8QuantizeArgs& g, hipStream_t st) {
  constexpr int V = I8Raw<TYPE>::V;
  long most = 0, rows = 0;
  for (int i = 0; i < g.count; ++i) {
    most = g.job[i].k > most ? g.job[i].k : most;
    rows += g.job[i].m;
  }
  if (most <= 64 * V * 8 && rows >= 2048)
    return most <= 64 * V * 2 ? launch_quantize_kernel<TYPE, 1, 2>(g, st) : launch_quantize_kernel<TYPE, 1, 8>(g, st);
  return most <= 256 * V * 2 ? launch_quantize_kernel<TYPE, 4, 2>(g, st) : launch_quantize_kernel<TYPE, 4, 8>(g, st);
}

hipError_t launch_i8_quantize(const I8QuantizeArgs& g, hipStream_t st) {
  for (int type = kI8F32; type <= kI8BF16; ++type) {  // a launch for each type
    I8QuantizeArgs of{};
    for (int i = 0; i < g.count; ++i)
      if (g.job[i].type == type) of.job[of.count++] = g.job[i];
    if (of.count == 0) continue;
    const hipError_t err = type == kI8F32 ? launch_quantize_type<kI8F32>(of, st)
                           : type == kI8F16 ? launch_quantize_type<kI8F16>(of, st) : launch_quantize_type<kI8BF16>(of, st);
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

// ----------------------------------------------------------------- products

constexpr int kI8Band = 8;

template <class S, bool PARTS>
__global__ __launch_bounds__(S::THREADS) void i8_gemm_kernel(I8GemmArgs g, int splits) {
  __shared__ __attribute__((aligned(16))) char lds[S::LDS];
  // workgroups are dealt to the 8 XCDs in turn: each XCD gets a run of tiles
  const int all = gridDim.x, each = all / 8, more = all % 8, xcd = blockIdx.x % 8;
  int b = xcd * each + (xcd < more ? xcd : more) + blockIdx.x / 8, which = 0;
  const int split = PARTS ? b / (all / splits) : 0;  // one part of k after the other
  if (PARTS) b -= split * (all / splits);
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
  auto load = [&]() {
    scales.load([&](int i) { return m0 + (i < rows ? i : rows - 1); }, [&](int, int row) { return p.sx[row]; },
                [&](int i) { return p.sw[n0 + (i < cols ? i : cols - 1)]; },
                [&](int i) { return p.bias ? p.bias[n0 + (i < cols ? i : cols - 1)] : 0.0f; });
  };
  const int steps = (p.k + S::BK - 1) / S::BK;
  const int s0 = PARTS ? (int)((long)steps * split / splits) : 0, s1 = PARTS ? (int)((long)steps * (split + 1) / splits) : steps;
  i8_tile<S, false>(static_cast<const int8_t*>(p.x) + (size_t)m0 * p.k, [&](int i) { return i < rows ? i : rows - 1; },
                    p.w + (size_t)n0 * p.k, p.w, [&](int i) { return i < cols ? i : cols - 1; }, p.k, s0, s1, lds, acc, load);
  void* y = PARTS ? static_cast<void*>(p.sums + (size_t)split * p.m * p.n) : p.y;
  i8_finish<S, false, PARTS>(acc, scales, lds, y, p.y_type, !PARTS && p.bias != nullptr, p.n, n0, rows, cols);
}

// The sums of the parts of k, scaled and rounded: V neighbouring columns a thread.
template <int V>
__global__ __launch_bounds__(256) void i8_sum_kernel(I8GemmArgs g, int splits) {
  int b = blockIdx.x, which = 0;
  while (which + 1 < g.count && b >= g.p[which + 1].first) ++which;
  const I8Problem& p = g.p[which];
  const long at = ((long)(b - p.first) * 256 + threadIdx.x) * V, outputs = (long)p.m * p.n;
  if (at >= outputs) return;
  const int row = (int)(at / p.n), c = (int)(at % p.n);
  typedef int32_t vec __attribute__((ext_vector_type(V)));
  vec sum = *reinterpret_cast<const vec*>(p.sums + at);
  for (int i = 1; i < splits; ++i) sum += *reinterpret_cast<const vec*>(p.sums + at + i * outputs);
  const float sx = p.sx[row];
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = (float)sum[i] * sx * p.sw[c + i];
    if (p.bias) v[i] += p.bias[c + i];
  }
  if (p.y_type == kI8F32) {
#pragma unroll
    for (int i = 0; i < V; ++i) static_cast<float*>(p.y)[at + i] = v[i];
  } else {
    uint16_t* y = static_cast<uint16_t*>(p.y) + at;
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = (uint16_t)i8_pair(p.y_type, v[i], v[i]);
  }
}

static hipError_t launch_sum(I8GemmArgs& g, int splits, hipStream_t st) {
  bool four = true;
  for (int i = 0; i < g.count; ++i) four = four && g.p[i].n % 4 == 0;
  long blocks = 0;
  for (int i = 0; i < g.count; ++i) {
    g.p[i].first = (int)blocks;
    blocks += ((long)g.p[i].m * g.p[i].n / (four ? 4 : 1) + 255) / 256;
  }
  if (four) hipLaunchKernelGGL((i8_sum_kernel<4>), dim3((unsigned)blocks), dim3(256), 0, st, g, splits);
  else hipLaunchKernelGGL((i8_sum_kernel<1>), dim3((unsigned)blocks), dim3(256), 0, st, g, splits);
  return hipGetLastError();
}

template <class S>
static hipError_t launch_shape(I8GemmArgs& g, int splits, hipStream_t st) {
  long tiles = 0;
  for (int i = 0; i < g.count; ++i) {
    g.p[i].first = (int)tiles;
    tiles += (long)((g.p[i].m + S::BM - 1) / S::BM) * ((g.p[i].n + S::BN - 1) / S::BN);
  }
  if (tiles == 0) return hipSuccess;
  if (splits == 1) {
    hipLaunchKernelGGL((i8_gemm_kernel<S, false>), dim3((unsigned)tiles), dim3(S::THREADS), 0, st, g, 1);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((i8_gemm_kernel<S, true>), dim3((unsigned)(tiles * splits)), dim3(S::THREADS), 0, st, g, splits);
  const hipError_t err = hipGetLastError();
  return err != hipSuccess ? err : launch_sum(g, splits, st);
}

// Tile shapes and what a round of their tiles costs on a full chip (of shapes that a
// CU holds several of: of all it holds): `fixed` us and `step` us for 128 bytes of k.
// Measured, k in one part (m x n x k, us of a call of codes, graph, weights from memory;
// in brackets from the last-level cache, which holds 256 MB):
//   shape      64x1024x4096  512x2560x4096  512x9728x2560  1024x2560x9728  2048x2560x9728  2048x9728x2560  16384x2560x9728
//   64 x 64     15.2 (11.2)    19.6 (14.5)           31.7            58.5            94.7           101.1              649
//   64 x 128    17.6 (13.7)    16.9 (14.5)           38.2            67.3           102.7           121.9              632
//   128 x 128   20.0 (18.2)    21.3 (18.7)           35.5            47.3            92.9            86.3              485
//   128 x 192   25.0 (24.1)    26.4 (25.0)           23.8            57.0            67.0            83.2              465
//   256 x 192   40.5 (37.8)    42.0 (39.3)           35.0            93.7            93.8            72.0              420
//   256 x 256   45.5 (44.1)    50.6 (47.9)           39.8           110.9           111.0            79.2              385
//   256 x 320   58.5 (56.9)    60.1 (58.0)           44.9           129.5           130.2            58.2              346
// The model takes the fastest of each column but one (512 x 2560 x 4096 from memory), and
// overstates large tiles where there are few of them: 256 x 320, 64 x 1024 x 4096: 76 us.
// A larger tile moves fewer bytes for its products; which one is best is mostly a
// matter of how evenly its tiles fall on the 256 CUs.
struct I8Choice {
  int bm, bn, at_once;  // tiles a CU holds
  float fixed, step;
};
constexpr I8Choice kI8Choices[] = {
    {64, 64, 3, 3.0f, 0.70f},  {64, 128, 1, 3.5f, 0.42f},  {128, 128, 1, 5.0f, 0.55f}, {128, 192, 1, 4.0f, 0.78f},
    {256, 192, 1, 7.0f, 1.30f}, {256, 256, 1, 8.0f, 1.65f}, {256, 320, 1, 9.0f, 2.10f},
};
constexpr int kI8Shapes = sizeof(kI8Choices) / sizeof(kI8Choices[0]);

// Parts of k, where there are too few tiles for the CUs: the sums of each part go
// through memory (int32, so that their order does not matter) and a second launch adds
// them up: `kI8SumFixed` us and 8 bytes an output and part at 4 TB/s.  64 x 2560 x
// 9728: 31.1 us in one part, 14.5 in six; 64 x 1024 x 4096: 15.2, 10.2 in four.
constexpr float kI8SumFixed = 4.0f, kI8SumRate = 4.0e6f;
constexpr long kI8SumMost = 64l << 20;  // bytes of sums

static void i8_choose(const I8GemmArgs& g, I8Way& way) {
  const int forced = way.shape;
  double least = 1e30;
  double outputs = 0;
  int fewest = 1 << 30;
  for (int i = 0; i < g.count; ++i) {
    const int steps = (g.p[i].k + 127) / 128;
    fewest = steps < fewest ? steps : fewest;
    outputs += (double)g.p[i].m * g.p[i].n;
  }
  const char* force = getenv("QMM_I8_SPLITS");  // tuning sweeps and tests
  for (int c = 0; c < kI8Shapes; ++c) {
    const I8Choice& h = kI8Choices[c];
    double tiles = 0, steps = 0;
    for (int i = 0; i < g.count; ++i) {
      const double t = (double)((g.p[i].m + h.bm - 1) / h.bm) * ((g.p[i].n + h.bn - 1) / h.bn);
      tiles += t;
      steps += t * ((g.p[i].k + 127) / 128);
    }
    if (forced >= 0 && c != forced) continue;
    const double slots = 256.0 * h.at_once;
    for (int splits = 1; splits <= 16 && splits <= fewest; ++splits) {
      if (splits > 1 && (tiles * splits > slots || outputs * splits * 4 > kI8SumMost)) break;
      if (force != nullptr && atoi(force) > 0 && atoi(force) <= fewest && splits != atoi(force)) continue;
      const double parts = tiles * splits;
      // whole rounds; where a CU holds several, its share of one
      const double full = (double)(long)((parts + slots - 1) / slots);
      const double share = parts / 256 > 1 ? parts / slots : 1.0 / h.at_once;
      double cost = (h.at_once > 1 ? share : full) * h.step * steps / parts + full * h.fixed;
      if (splits > 1) cost += kI8SumFixed + outputs * splits * 8 / kI8SumRate;
      if (cost < least) {
        least = cost;
        way.shape = c;
        way.splits = splits;
      }
    }
  }
}

template <int U, bool LOOP, int TYPE>
__global__ __launch_bounds__(kI8FewThreads) __attribute__((amdgpu_waves_per_eu(4))) void i8_few_kernel(I8GemmArgs g, int kw) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int b = blockIdx.x, which = 0;
  while (which + 1 < g.count && b >= g.p[which + 1].first) ++which;
  const I8Problem& p = g.p[which];
  const int wide = 16 * (kI8FewWaves / kw), n0 = (b - p.first) * wide;
  const I8FewTile t{p.w + (size_t)n0 * p.k, nullptr, p.sw + n0, nullptr, p.bias ? p.bias + n0 : nullptr, p.x, p.sx, p.y,
                    p.y_type, p.n, n0, p.n - n0 < wide ? p.n - n0 : wide, p.m, p.k, kw};
  auto same = [](int i) { return i; };
  i8_few<U, LOOP, false, TYPE>(t, lds, same, same);
}

template <int U, bool LOOP, int TYPE>
static hipError_t launch_few_kernel(I8GemmArgs& g, int kw, hipStream_t st) {
  long blocks = 0;
  size_t lds = 0;
  const int wide = 16 * (kI8FewWaves / kw);
  for (int i = 0; i < g.count; ++i) {
    g.p[i].first = (int)blocks;
    blocks += (g.p[i].n + wide - 1) / wide;
    const size_t need = i8_few_lds<U, false>(TYPE == kI8Codes ? 0 : g.p[i].m, g.p[i].k);
    lds = need > lds ? need : lds;
  }
  hipLaunchKernelGGL((i8_few_kernel<U, LOOP, TYPE>), dim3((unsigned)blocks), dim3(kI8FewThreads), lds, st, g, kw);
  return hipGetLastError();
}

static long i8_blocks(const I8GemmArgs& g) {  // of 16 columns
  long blocks = 0;
  for (int i = 0; i < g.count; ++i) blocks += (g.p[i].n + 15) / 16;
  return blocks;
}

template <int TYPE>
static hipError_t launch_few(I8GemmArgs& g, hipStream_t st) {
  int most = 0;
  for (int i = 0; i < g.count; ++i) most = g.p[i].k > most ? g.p[i].k : most;
  const int kw = i8_few_kw(i8_blocks(g), TYPE == kI8Codes);
  const int each = ((most + 63) / 64 + kw - 1) / kw;  // slices a wave
  if (each <= 2) return launch_few_kernel<2, false, TYPE>(g, kw, st);
  if (each <= 5) return launch_few_kernel<5, false, TYPE>(g, kw, st);
  if constexpr (TYPE != kI8Codes)
    if (each <= 8) return launch_few_kernel<8, false, TYPE>(g, kw, st);
  return launch_few_kernel<5, true, TYPE>(g, kw, st);
}

// How a call runs, decided once: `staged` (the product rounds x itself) goes with
// few rows only.  us of a call, rounding of fp16 x included (graph, weights from memory):
//   rows x n x k          rounded in the product   few rows, codes   tiles of 64 x 64
//    1 x 9728 x 2560                 9.5                 11.1              14.0
//    4 x 9728 x 2560                10.0                 11.7              14.3
//    4 x 2560 x 9728                   -                 15.4              17.5 (k whole: 34.7)
//    8 x 1024 x 1024                 5.3                  6.8               9.2
//    8 x 151936 x 1024              32.6                 39.0              37.7
//   16 x 9728 x 2560                   -                 13.6              14.6
//   16 x 16384 x 1024                  -                  9.7              10.2
//   16 x 32768 x 1024                  -                 13.7              12.6
//   16 x 151936 x 1024                 -                 40.9              38.4
// (The workspace's size follows from it: it looks at m, n, k and x's type alone.)
I8Way i8_gemm_way(const I8GemmArgs& g) {
  I8Way way{false, false, -1, 1};
  const char* force = getenv("QMM_I8_FORCE");  // tuning sweeps and tests: a tile shape by its place
  if (force != nullptr && atoi(force) >= 0 && atoi(force) < kI8Shapes) {
    way.shape = atoi(force);
    i8_choose(g, way);
    return way;
  }
  int most = 0;
  way.staged = true;
  for (int i = 0; i < g.count; ++i) {
    most = g.p[i].m > most ? g.p[i].m : most;
    if (g.p[i].x_type == kI8Codes || g.p[i].x_type != g.p[0].x_type || !i8_can_stage(g.p[i].m, g.p[i].k)) way.staged = false;
  }
  way.few = way.staged || (most <= kI8FewRows && i8_blocks(g) <= 1024);
  if (!way.few) i8_choose(g, way);
  return way;
}

hipError_t launch_i8_gemm(I8GemmArgs& g, I8Way way, hipStream_t st) {
  if (way.few) switch (g.p[0].x_type) {
    case kI8F32: return launch_few<kI8F32>(g, st);
    case kI8F16: return launch_few<kI8F16>(g, st);
    case kI8BF16: return launch_few<kI8BF16>(g, st);
    default: return launch_few<kI8Codes>(g, st);
  }
  switch (way.shape) {
    case 0: return launch_shape<I8Shape<64, 64, 2, 2, 3>>(g, way.splits, st);
    case 1: return launch_shape<I8Shape<64, 128, 2, 4, 6>>(g, way.splits, st);
    case 2: return launch_shape<I8Shape<128, 128, 2, 4, 3>>(g, way.splits, st);
    case 3: return launch_shape<I8Shape<128, 192, 4, 2, 3>>(g, way.splits, st);
    case 4: return launch_shape<I8Shape<256, 192, 4, 2, 2>>(g, way.splits, st);
    case 5: return launch_shape<I8Shape<256, 256, 2, 4, 2>>(g, way.splits, st);
    default: return launch_shape<I8Shape<256, 320, 4, 2, 2>>(g, way.splits, st);
  }
}

}  // namespace qmm
