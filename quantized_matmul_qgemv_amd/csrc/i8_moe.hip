// Products in 8-bit integers by expert (include/qmm.h, qmm_i8_gemm_grouped and
// qmm_i8_moe_gate_up_swiglu) from a routing plan of qmm_moe_route: each
// workgroup takes rows of one expert from the plan's list, gathers their codes
// and multiplies them by that expert's weights.
#include "i8_core.h"
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

// GATED: the tile's rows of W are half gate, half up: a wave's first TN / 2
// blocks of columns are gate's and the others the same columns of up, so both
// products of an output stand in the same lane and register.
template <class S, bool GATED>
__global__ __launch_bounds__(S::THREADS) void i8_moe_kernel(I8MoeArgs g, int n_tiles) {
  __shared__ __attribute__((aligned(16))) char lds[S::LDS];
  __shared__ int32_t pair_of[S::BM];
  constexpr int BC = GATED ? S::BN / 2 : S::BN;  // output columns
  constexpr int TC = GATED ? S::TN / 2 : S::TN;
  const int32_t* ws = g.plan;
  const int pairs = g.t * g.top_k;
  int tile, tn;
  moe_tile_of(n_tiles, kMoeRun * g.subs, tile, tn);
  const int sub = tile % g.subs;
  tile /= g.subs;
  // a plan built for other counts is not used: the whole output becomes NaN
  if (ws[1] != g.plan_rows || ws[2] != pairs || ws[3] != g.e) {
    i8_nan_all(g);
    return;
  }
  if (tile >= ws[0]) return;
  MoeTile mt = reinterpret_cast<const MoeTile*>(ws + kPlanHeaderInts + pairs)[tile];
  mt.start += sub * S::BM;
  mt.rows -= sub * S::BM;
  if (mt.rows <= 0) return;
  if (mt.rows > S::BM) mt.rows = S::BM;
  const int32_t* sorted = ws + kPlanHeaderInts;
  const int n0 = tn * BC;
  if (mt.expert < 0) {
    i8_nan_rows(g, sorted, mt, n0, BC);
    return;
  }
  for (int i = threadIdx.x; i < S::BM; i += S::THREADS) pair_of[i] = sorted[mt.start + (i < mt.rows ? i : mt.rows - 1)];
  __syncthreads();
  const int cols = g.n - n0 < BC ? g.n - n0 : BC;
  const size_t at = ((size_t)mt.expert * g.n + n0) * g.k;
  i32x16 acc[S::TM][S::TN];
#pragma unroll
  for (int i = 0; i < S::TM; ++i)
#pragma unroll
    for (int j = 0; j < S::TN; ++j) acc[i][j] = i32x16{};
  auto x_row = [&](int i) { const int p = pair_of[i]; return g.a_row_per_pair ? p : p / g.top_k; };
  i8_tile<S, GATED>(g.x, x_row, g.w + at, GATED ? g.w2 + at : g.w + at,
                    [&](int i) { return i < cols ? i : cols - 1; }, g.k, 0, (g.k + kI8Step - 1) / kI8Step, lds, acc);
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int wm = wave / S::WN, wn = wave % S::WN;
  const bool wide = g.n % 4 == 0 && ((uintptr_t)g.y & (g.y_type == kI8F32 ? 15 : 7)) == 0;
  const float* sw = g.sw + (size_t)mt.expert * g.n + n0;
  const float* sw2 = GATED ? g.sw2 + (size_t)mt.expert * g.n + n0 : nullptr;
#pragma unroll
  for (int i = 0; i < S::TM; ++i) {
    const int r = (wm * S::TM + i) * 32 + (lane & 31);
    if (r >= mt.rows) continue;
    const int pair = pair_of[r];
    const float sx = g.sx[g.a_row_per_pair ? pair : pair / g.top_k];
    const size_t row = (size_t)pair * g.n + n0;
#pragma unroll
    for (int j = 0; j < TC; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = (wn * TC + j) * 32 + 8 * q + 4 * (lane >> 5);
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int cc = c + e < cols ? c + e : cols - 1;
          v[e] = (float)acc[i][j][4 * q + e] * sx * sw[cc];
          if constexpr (GATED) v[e] = i8_silu(v[e]) * ((float)acc[i][j + TC][4 * q + e] * sx * sw2[cc]);
        }
        i8_store(g.y, row + c, g.y_type, v, cols - c, wide);
      }
  }
}

template <class S, bool GATED>
static hipError_t launch_moe_shape(I8MoeArgs& g, hipStream_t st) {
  constexpr int BC = GATED ? S::BN / 2 : S::BN;
  const int n_tiles = (g.n + BC - 1) / BC;
  g.subs = (g.plan_rows + S::BM - 1) / S::BM;
  const int m_tiles = max_row_tiles(g.t * g.top_k, g.e, g.plan_rows) * g.subs;
  hipLaunchKernelGGL((i8_moe_kernel<S, GATED>), dim3(moe_grid(m_tiles, n_tiles, kMoeRun * g.subs)), dim3(S::THREADS), 0, st, g, n_tiles);
  return hipGetLastError();
}

hipError_t launch_i8_moe(I8MoeArgs& g, hipStream_t st) {
  using S = I8Shape<32, 128, 1, 4, 2>;
  using D = I8Shape<32, 256, 1, 4, 2>;
  return g.w2 ? launch_moe_shape<D, true>(g, st) : launch_moe_shape<S, false>(g, st);
}

}  // namespace qmm
