// The routing plan on the device (include/qmm.h, "Routing plan / workspace
// image") and the order of a grouped launch's workgroups, shared by every
// kernel that runs from a plan.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmm {

struct MoeTile {
  int32_t expert;  // -1: the pairs whose expert id lies outside [0, E)
  int32_t start;   // first slot in the sorted pair list
  int32_t rows;
};

// Workspace layout (int32 units): a header of kPlanHeaderInts words
//   [0] row tiles in the list   [1] row tile (rows)   [2] pairs   [3] experts
//   [4] pairs whose expert id is outside [0, E) (their output rows are NaN)
//   [5..7] zero
// then the sorted pairs (P words) and the tile list (3 words per tile).  The
// same image is the routing plan that one bucketing pass builds for several
// grouped GEMMs on the same expert ids.  Pairs with an out-of-range id sit
// after every valid bucket and get row tiles of their own (expert -1), so
// the bound on row tiles counts E + 1 buckets.
constexpr int kPlanHeaderInts = 8;

inline int max_row_tiles(int pairs, int experts, int bm) {
  const long by_pairs = (long)(pairs + bm - 1) / bm + experts + 1;
  return by_pairs < pairs ? (int)by_pairs : (pairs > 0 ? pairs : 1);
}

// Output of a grouped launch that cannot be computed: a plan built for
// another row tile, pair count or expert count.  The whole output
// (rows x cols elements, row stride ld) is filled with NaN by the launch's
// workgroups together, so the failure shows in every result.
template <typename T>
__device__ void fill_nan_all(T* out, long rows, int cols, int ld, T nan) {
  const long total = rows * cols;
  const long stride = (long)gridDim.x * blockDim.x;
  for (long i = (long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride)
    out[(i / cols) * ld + i % cols] = nan;
}

// Rows of the pairs of an out-of-range row tile (expert -1): NaN in the
// tile's columns [c0, c0 + bn) (bounded by n).
template <typename T>
__device__ void fill_nan_rows(T* out, const int32_t* sorted, const MoeTile& mt, int c0, int bn, int n,
                              T nan) {
  const int cols = n - c0 < bn ? n - c0 : bn;
  for (int i = threadIdx.x; i < mt.rows * cols; i += blockDim.x) {
    const long row = sorted[mt.start + i / cols];
    out[row * n + c0 + i % cols] = nan;
  }
}

// Workgroup -> (row tile, column tile).  Workgroups are dealt round-robin
// to the 8 XCDs (workgroup b runs on XCD b % 8), each with its own L2.  All
// column tiles of one row tile gather the same A rows (the expert's tokens),
// and consecutive row tiles of the list belong mostly to one expert and read
// the same weights; so runs of kMoeRun consecutive row tiles, with all their
// column tiles, are placed on one XCD, next to each other in its dispatch
// order, and the runs are dealt round-robin across the XCDs:
//   b -> xcd = b % 8, i = b / 8, k = i / n_tiles;
//   row tile = (k / R) * 8R + xcd * R + k % R,  column tile = i % n_tiles
// (R = kMoeRun).  The grid is ceil(row tiles / 8R) * 8R * n_tiles
// workgroups.  Against one row tile per run (R = 1) this halved the bytes
// the grouped GEMM and the fused gate/up fetch at 2048 tokens (443 -> 243 MB
// and 998 -> 493 MB per launch) and took the fused gate/up from 177 to
// 160 us.
constexpr int kMoeXcds = 8;
constexpr int kMoeRun = 8;

__device__ __forceinline__ void moe_tile_of(int n_tiles, int run, int& tile, int& tn) {
  const int xcd = blockIdx.x % kMoeXcds;
  const int i = blockIdx.x / kMoeXcds;
  const int k = i / n_tiles;
  tile = (k / run) * (kMoeXcds * run) + xcd * run + k % run;
  tn = i % n_tiles;
}

inline unsigned moe_grid(int m_tiles, int n_tiles, int run) {
  const int per = kMoeXcds * run;
  return (unsigned)((m_tiles + per - 1) / per) * per * n_tiles;
}

}  // namespace qmm
