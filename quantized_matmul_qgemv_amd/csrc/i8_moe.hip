// Products in 8-bit integers by expert (include/qmm.h, qmm_i8_gemm_grouped and
// qmm_i8_moe_gate_up_swiglu) from a routing plan of qmm_moe_route: each
// workgroup takes rows of one expert from the plan's list, gathers their codes
// and multiplies them by that expert's weights.
#include <stdlib.h>

#include "i8_few.h"
#include "moe_plan.h"
#include "qmm_internal.h"

namespace qmm {

// NaN in an output of any type.
__device__ __forceinline__ void i8_nan_all(const I8MoeArgs& g) {
  const long pairs = (long)g.t * g.top_k;
  if (g.y_type == kI8F32) fill_nan_all(static_cast<float*>(g.y), pairs, g.n, g.n, __builtin_nanf(""));
  else fill_nan_all(static_cast<uint16_t*>(g.y), pairs, g.n, g.n, (uint16_t)(g.y_type == kI8F16 ? 0x7E00 : 0x7FC0));
}

__device__ __forceinline__ void i8_nan_rows(const I8MoeArgs& g, const int32_t* sorted, const MoeTile& mt, int c0, int bn) {
  if (g.y_type == kI8F32) fill_nan_rows(static_cast<float*>(g.y), sorted, mt, c0, bn, g.n, __builtin_nanf(""));
  else fill_nan_rows(static_cast<uint16_t*>(g.y), sorted, mt, c0, bn, g.n, (uint16_t)(g.y_type == kI8F16 ? 0x7E00 : 0x7FC0));
}

template <class S, bool GATED>
__global__ __launch_bounds__(S::THREADS) void i8_moe_kernel(I8MoeArgs g, int n_tiles) {
  __shared__ __attribute__((aligned(16))) char lds[S::LDS];
  constexpr int BC = GATED ? S::BN / 2 : S::BN;  // output columns
  const int32_t* ws = g.plan;
  const int pairs = g.t * g.top_k;
  // a plan built for other counts is not used: the whole output becomes NaN
  const i32x4 head = *reinterpret_cast<const i32x4*>(ws);
  if (head[1] != g.plan_rows || head[2] != pairs || head[3] != g.e) {
    i8_nan_all(g);
    return;
  }
  // Each XCD (workgroups are dealt to the 8 in turn) takes an equal run of the row tiles
  // that there are, with all their columns: an expert's tiles stand together.
  const int listed = __builtin_amdgcn_readfirstlane(head[0]);
  const int each = (listed * g.subs + kMoeXcds - 1) / kMoeXcds, mine = blockIdx.x / kMoeXcds;
  if (mine >= each * n_tiles) return;
  const int tn = mine % n_tiles;
  int tile = blockIdx.x % kMoeXcds * each + mine / n_tiles;
  const int sub = tile % g.subs;
  tile /= g.subs;
  if (tile >= listed) return;
  const MoeTile* list = reinterpret_cast<const MoeTile*>(ws + kPlanHeaderInts + pairs);
  MoeTile mt = list[tile];  // in scalar registers
  mt.expert = __builtin_amdgcn_readfirstlane(mt.expert);
  mt.start = __builtin_amdgcn_readfirstlane(mt.start);
  mt.rows = __builtin_amdgcn_readfirstlane(mt.rows);
  if (g.plan_rows < S::BM) {
    // several of the list's tiles at once, from every `span`-th of an expert's;
    // the expert's tiles stand together, all but the last whole
    const int span = S::BM / g.plan_rows;
    const int lane = threadIdx.x & 63;
    int before = 0;  // tiles of the same expert before this one
    for (int first = tile - 1;; first -= 64) {  // ends at the list's first
      const int i = first - lane;
      const uint64_t other = __ballot(i < 0 || list[i < 0 ? 0 : i].expert != mt.expert);
      before += other ? __builtin_ctzll(other) : 64;
      if (other) break;
    }
    if (before % span) return;
    for (int i = 1; i < span && tile + i < listed; ++i)
      if (list[tile + i].expert == mt.expert) mt.rows += list[tile + i].rows;
    mt.rows = __builtin_amdgcn_readfirstlane(mt.rows);
  } else {
    mt.start += sub * S::BM;
    mt.rows -= sub * S::BM;
    if (mt.rows <= 0) return;
    if (mt.rows > S::BM) mt.rows = S::BM;
  }
  const int32_t* sorted = ws + kPlanHeaderInts;
  const int n0 = tn * BC;
  if (mt.expert < 0) {
    i8_nan_rows(g, sorted, mt, n0, BC);
    return;
  }
  sorted += mt.start;
  const int cols = g.n - n0 < BC ? g.n - n0 : BC;
  const size_t at = ((size_t)mt.expert * g.n + n0) * g.k;
  i32x16 acc[S::TM][S::TN];
#pragma unroll
  for (int i = 0; i < S::TM; ++i)
#pragma unroll
    for (int j = 0; j < S::TN; ++j) acc[i][j] = i32x16{};
  auto pair = [&](int i) { return sorted[i < mt.rows ? i : mt.rows - 1]; };
  auto row = [&](int p) { return g.a_row_per_pair ? p : p / g.top_k; };
  I8Scales<S> scales;
  const size_t column = (size_t)mt.expert * g.n + n0;
  auto load = [&]() {
    scales.load(pair, [&](int, int p) { return g.sx[row(p)]; },
                [&](int i) {
                  const bool up = GATED && i % 32 >= 16;
                  if (GATED) i = i / 32 * 16 + i % 16;
                  return (up ? g.sw2 : g.sw)[column + (i < cols ? i : cols - 1)];
                },
                [](int) { return 0.0f; });
  };
  i8_tile<S, GATED>(static_cast<const int8_t*>(g.x), [&](int i) { return row(pair(i)); }, g.w + at, GATED ? g.w2 + at : g.w + at,
                    [&](int i) { return i < cols ? i : cols - 1; }, g.k, 0, (g.k + S::BK - 1) / S::BK, lds, acc, load);
  i8_finish<S, GATED, false>(acc, scales, lds, g.y, g.y_type, false, g.n, n0, mt.rows, cols);
}

// Workgroups of a call: whole rounds of the XCDs for as many row tiles as there can be.
template <class S, bool GATED>
static long i8_moe_groups(const I8MoeArgs& g) {
  constexpr int BC = GATED ? S::BN / 2 : S::BN;
  const long m_tiles = (long)max_row_tiles(g.t * g.top_k, g.e, g.plan_rows) * ((g.plan_rows + S::BM - 1) / S::BM);
  return (m_tiles + kMoeXcds - 1) / kMoeXcds * kMoeXcds * ((g.n + BC - 1) / BC);
}

template <class S, bool GATED>
static hipError_t launch_moe_shape(I8MoeArgs& g, hipStream_t st) {
  constexpr int BC = GATED ? S::BN / 2 : S::BN;
  const int n_tiles = (g.n + BC - 1) / BC;
  g.subs = (g.plan_rows + S::BM - 1) / S::BM;
  hipLaunchKernelGGL((i8_moe_kernel<S, GATED>), dim3((unsigned)i8_moe_groups<S, GATED>(g)), dim3(S::THREADS), 0, st, g, n_tiles);
  return hipGetLastError();
}

// Few rows an expert: 16 * 8 / kw columns of one row tile a workgroup.
template <int U, bool LOOP, bool GATED, int TYPE>
__global__ __launch_bounds__(kI8FewThreads) __attribute__((amdgpu_waves_per_eu(4))) void i8_moe_few_kernel(I8MoeArgs g, int n_tiles, int kw) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int32_t* ws = g.plan;
  const int pairs = g.t * g.top_k;
  if (ws[1] != g.plan_rows || ws[2] != pairs || ws[3] != g.e) {
    i8_nan_all(g);
    return;
  }
  const int tile = blockIdx.x / n_tiles, tn = blockIdx.x % n_tiles;
  if (tile >= ws[0]) return;
  MoeTile mt = reinterpret_cast<const MoeTile*>(ws + kPlanHeaderInts + pairs)[tile];
  mt.expert = __builtin_amdgcn_readfirstlane(mt.expert);
  mt.start = __builtin_amdgcn_readfirstlane(mt.start);
  mt.rows = __builtin_amdgcn_readfirstlane(mt.rows);
  const int32_t* sorted = ws + kPlanHeaderInts;
  const int wide = 16 * (kI8FewWaves / kw), n0 = tn * wide;
  if (mt.expert < 0) {
    i8_nan_rows(g, sorted, mt, n0, wide);
    return;
  }
  sorted += mt.start;
  const size_t column = (size_t)mt.expert * g.n + n0, at = column * g.k;
  const I8FewTile t{g.w + at, GATED ? g.w2 + at : nullptr, g.sw + column, GATED ? g.sw2 + column : nullptr, nullptr, g.x, g.sx, g.y,
                    g.y_type, g.n, n0, g.n - n0 < wide ? g.n - n0 : wide, mt.rows, g.k, kw};
  auto pair = [&](int i) { return sorted[i]; };
  auto row = [&](int i) { const int p = sorted[i]; return g.a_row_per_pair ? p : p / g.top_k; };
  i8_few<U, LOOP, GATED, TYPE>(t, lds, row, pair);
}

template <int U, bool LOOP, bool GATED, int TYPE>
static hipError_t launch_moe_few_kernel(I8MoeArgs& g, int kw, hipStream_t st) {
  const int wide = 16 * (kI8FewWaves / kw), n_tiles = (g.n + wide - 1) / wide;
  const int pairs = g.t * g.top_k, tiles = max_row_tiles(pairs, g.e, g.plan_rows);
  const size_t lds = i8_few_lds<U, GATED>(TYPE == kI8Codes ? 0 : pairs, g.k);
  hipLaunchKernelGGL((i8_moe_few_kernel<U, LOOP, GATED, TYPE>), dim3((unsigned)tiles * n_tiles), dim3(kI8FewThreads), lds, st, g,
                     n_tiles, kw);
  return hipGetLastError();
}

template <bool GATED, int TYPE>
static hipError_t launch_moe_few(I8MoeArgs& g, hipStream_t st) {
  const long pairs = (long)g.t * g.top_k, tiles = pairs < g.e ? pairs : g.e;  // about as many as have rows
  const int kw = i8_few_kw(tiles * ((g.n + 15) / 16), TYPE == kI8Codes);
  const int each = ((g.k + 63) / 64 + kw - 1) / kw;
  if (each <= 2) return launch_moe_few_kernel<2, false, GATED, TYPE>(g, kw, st);
  if (each <= 4) return launch_moe_few_kernel<4, false, GATED, TYPE>(g, kw, st);
  return launch_moe_few_kernel<4, true, GATED, TYPE>(g, kw, st);
}

template <bool GATED>
static hipError_t launch_moe_few_type(I8MoeArgs& g, hipStream_t st) {
  switch (g.x_type) {
    case kI8F32: return launch_moe_few<GATED, kI8F32>(g, st);
    case kI8F16: return launch_moe_few<GATED, kI8F16>(g, st);
    case kI8BF16: return launch_moe_few<GATED, kI8BF16>(g, st);
    default: return launch_moe_few<GATED, kI8Codes>(g, st);
  }
}

// How a call runs, decided once: few rows, where no row tile can have more than 16
// (`staged`: not more than a workgroup rounds for itself), or tiles.  us of a call, 128
// experts, weights from memory, fp16 rows: rounded in the product / before it / tiles
//   one token, 8 pairs:   gate and up of 768 x 2048   9.7 / 12.8 / 23.3   down    7.1 /  9.4 / 11.5
//   two tokens, 16 pairs:                               - / 16.3 / 24.4   down      - / 13.0 / 12.5
I8Way i8_moe_way(const I8MoeArgs& g) {
  const long pairs = (long)g.t * g.top_k;
  I8Way way{pairs <= kI8FewRows, false, g.plan_rows >= 128 ? 1 : 0, 1};
  if (const char* env = getenv("QMM_I8_MOE_FORCE")) {  // tuning sweeps and tests
    way.few = false;
    way.shape = atoi(env) != 0;
  }
  way.staged = way.few && g.x_type != kI8Codes && i8_can_stage((int)pairs, g.k);
  return way;
}

using I8MoeTall = I8Shape<128, 192, 4, 2, 2>;
using I8MoeFlat = I8Shape<64, 256, 2, 4, 2>;

// Few rows: at most 16 row tiles of 2^21 columns, always below.
bool i8_moe_fits(const I8MoeArgs& g, I8Way way) {
  if (way.few) return true;
  long threads;
  if (way.shape == 1) threads = (g.w2 ? i8_moe_groups<I8MoeTall, true>(g) : i8_moe_groups<I8MoeTall, false>(g)) * I8MoeTall::THREADS;
  else threads = (g.w2 ? i8_moe_groups<I8MoeFlat, true>(g) : i8_moe_groups<I8MoeFlat, false>(g)) * I8MoeFlat::THREADS;
  return threads < 1l << 32;
}

// Tile shapes, us a call (plan rows 32: 64 tokens, way back; 64: 2048 tokens, way
// back; 128: 16384 tokens, gate and up; 128 experts, top-8, 768 x 2048, some experts
// liked more than others, rounding of the rows included; * with a third stage in LDS):
//   plan   64x128   64x128*   64x256   64x256*   128x128   128x192   128x256*   256x192
//     32     26.4      25.7     23.5      26.4      27.0      29.0       27.7      41.1
//     64     94.0     103.4       95     105.2      97.5      93.1      100.4     117.5
//    128    616.9     690.8      583     704.9      558.6     505.4      594.8     582.1
// Two workgroups a CU (80 KB of LDS each) beat larger tiles and longer rings: one
// stores while the other multiplies.  Equal runs of row tiles for the XCDs, by the
// number that there is, beat runs of eight dealt in turn where tiles are few (333
// tokens on 35 experts: 25.1 -> 20.7).
hipError_t launch_i8_moe(I8MoeArgs& g, I8Way way, hipStream_t st) {
  if (way.few) return g.w2 ? launch_moe_few_type<true>(g, st) : launch_moe_few_type<false>(g, st);
  if (way.shape == 1) return g.w2 ? launch_moe_shape<I8MoeTall, true>(g, st) : launch_moe_shape<I8MoeTall, false>(g, st);
  return g.w2 ? launch_moe_shape<I8MoeFlat, true>(g, st) : launch_moe_shape<I8MoeFlat, false>(g, st);
}

}  // namespace qmm
