// Low-rank adapters of many requests beside a shared projection:
//
//   y[p, :] = base[p, :] + scale[a] * B_s (A_s x[row(p), :]),   a = adapter_ids[p / top_k]
//
// with s = a (dense projections) or a * experts + expert_ids[p] (the experts'
// products of a routed layer), A_s [rank, k] and B_s [n, rank] in fp16.
// a = -1 leaves the row as base has it; an id out of range makes it NaN.
//
// Everything works on tiles of rows that share a slot s:
//   shrink  v = A_s x, fp32 (products of fp16, exact in fp32);
//   expand  y = base + scale * B_s v.  On the matrix cores, which take fp16,
//           each row of v is scaled by a power of two that brings its largest
//           value into [2^14, 2^15) and split into v = hi + lo, both fp16
//           (error 2^-23 of that largest value: one rounding of fp32), which
//           stand side by side along the contraction: [hi | lo] x [B | B].
// Few rows with a small A take both in one launch of dot products, others one
// or two launches on the matrix cores (lora_layout chooses).  Small calls find
// their tiles from ballots over the ids of all rows; beyond kLoraFewRows (or
// kLoraDirectRows) one or two short launches sort the rows by slot into a tile
// list first.
//
// Every row is computed on its own (neither its tile nor its place in it
// enters the sums), so results do not depend on scheduling.  All large calls
// are bound by memory: x, base and y once, and the slots' weights.
#include "qmm_device.h"
#include "qmm_internal.h"

namespace qmm {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));

constexpr int kLoraThreads = 256;
constexpr int kNone = -1;  // slot of a row without adapter
constexpr int kBad = -2;   // slot of a row whose ids are out of range

struct LoraTile {
  int32_t slot, start, rows, pad;
};

// The slot of row p.
__device__ __forceinline__ int lora_slot(const LoraArgs& g, int p) {
  const int a = g.adapter_ids[g.top_k == 1 ? p : p / g.top_k];
  if (a == -1) return kNone;
  if (a < 0 || a >= g.adapters) return kBad;
  if (g.expert_ids == nullptr) return a;
  const int e = g.expert_ids[p];
  return e < 0 || e >= g.experts ? kBad : a * g.experts + e;
}

// The row of x that row p reads.
__device__ __forceinline__ int lora_x_row(const LoraArgs& g, const LoraProblem& p, int row) {
  return p.x_row_per_pair || g.top_k == 1 ? row : row / g.top_k;
}

// A workgroup's rows of one slot.
template <int BM>
struct TileRows {
  int32_t rows[BM];
  int32_t slot, count;
};

// Direct: the workgroup of row p owns the tile that starts at p, if an equal
// number of rows with p's slot, a multiple of BM, comes before it.  The
// workgroup has a thread for every row, up to ROWS.
template <int ROWS, int BM>
__device__ __forceinline__ bool find_tile(const LoraArgs& g, int p, TileRows<BM>& t) {
  __shared__ uint64_t masks[ROWS / 64];
  const int tid = threadIdx.x;
  const int s = tid < g.rows ? lora_slot(g, tid) : 0;
  if (tid == p) t.slot = s;
  __syncthreads();
  const bool same = tid < g.rows && s == t.slot;
  const uint64_t m = __ballot(same);
  if ((tid & 63) == 0) masks[tid >> 6] = m;
  __syncthreads();
  int before = 0, total = 0, mine = 0;
#pragma unroll
  for (int w = 0; w < ROWS / 64; ++w) {
    const uint64_t b = masks[w];
    const int lo = p - w * 64, li = tid - w * 64;
    before += __popcll(lo >= 64 ? b : lo > 0 ? b & ((1ull << lo) - 1) : 0);
    mine += __popcll(li >= 64 ? b : li > 0 ? b & ((1ull << li) - 1) : 0);
    total += __popcll(b);
  }
  if (before % BM != 0) return false;
  if (same && mine >= before && mine < before + BM) t.rows[mine - before] = tid;
  if (tid == 0) t.count = total - before < BM ? total - before : BM;
  __syncthreads();
  return true;
}

// Routed: the tile of workgroup i.  Workgroups are dealt round-robin to the
// 8 XCDs (the grid's first dimension is a multiple of 8); each XCD takes a
// run of the list, so that the tiles of a slot, next to each other there, read
// its weights through one L2.
constexpr int kXcds = 8;
template <int BM>
__device__ __forceinline__ bool read_tile(const LoraArgs& g, int i, TileRows<BM>& t) {
  const int tiles = g.plan[0];
  const int run = (tiles + kXcds - 1) / kXcds;
  if (i / kXcds >= run) return false;
  i = i % kXcds * run + i / kXcds;
  if (i >= tiles) return false;
  const int32_t* sorted = g.plan + kLoraPlanHeader;
  const LoraTile lt = reinterpret_cast<const LoraTile*>(g.plan + g.plan_tiles)[i];
  if (threadIdx.x < BM && threadIdx.x < lt.rows) t.rows[threadIdx.x] = sorted[lt.start + threadIdx.x];
  if (threadIdx.x == 0) {
    t.slot = lt.slot;
    t.count = lt.rows;
  }
  __syncthreads();
  return true;
}

// ------------------------------------------------------------------ shrink
// Tiles of 16 rows (few rows a slot: the weights are what is read).  One
// workgroup: up to 64 ranks (RT blocks of 16) and one k range; the four waves
// take turns at 64 values of k and are joined in LDS.  A lane's two 16-byte
// loads per step are neighbours in k (the same permutation of k for both
// operands leaves the sum as it is), so a wave's loads cover whole 128-byte
// lines.  Bound by latency and the 15 bytes a clock and CU that L1 gives to
// loads of 16 rows at once: 8.3 us for 64 rows on 64 slots, rank 64, k 2560 (21
// MB of A, 2.5 TB/s).
template <bool ROUTED, int RT>
__global__ __launch_bounds__(kLoraThreads) void lora_shrink16_kernel(LoraArgs g) {
  __shared__ TileRows<16> tile;
  __shared__ f4 part[3][RT][64];
  const LoraProblem& p = g.p[blockIdx.z];
  const int chunks = (p.rank + 63) >> 6;
  const int split = blockIdx.y / chunks;
  const int r0 = (blockIdx.y - split * chunks) * 64;
  if (split >= p.splits) return;
  if (!(ROUTED ? read_tile(g, blockIdx.x, tile) : find_tile<kLoraThreads>(g, blockIdx.x, tile))) return;
  if (tile.slot < 0) return;
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int li = lane & 15;
  const int q = lane >> 4;

  const int row = tile.rows[li < tile.count ? li : tile.count - 1];
  auto xp = to_global(p.x) + (size_t)lora_x_row(g, p, row) * p.k + q * 16;
  gptr<uint16_t> ap[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = r0 + i * 16 + li < p.rank ? r0 + i * 16 + li : p.rank - 1;
    ap[i] = to_global(p.a) + ((size_t)tile.slot * p.rank + r) * p.k + q * 16;
  }
  f4 acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = f4{0, 0, 0, 0};
  const int kend = (split + 1) * p.k_per_split < p.k ? (split + 1) * p.k_per_split : p.k;
#pragma unroll 2
  for (int k = split * p.k_per_split + wave * 64; k < kend; k += 256) {
    const h8 x0 = *(gptr<h8>)(xp + k), x1 = *(gptr<h8>)(xp + k + 8);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const h8 a0 = *(gptr<h8>)(ap[i] + k), a1 = *(gptr<h8>)(ap[i] + k + 8);
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, x0, acc[i], 0, 0, 0);
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, x1, acc[i], 0, 0, 0);
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i < RT; ++i) part[wave - 1][i][lane] = acc[i];
  }
  __syncthreads();
  if (wave > 0 || li >= tile.count) return;
  float* v = g.v + p.v_offset + ((size_t)split * g.rows + row) * p.rank_pad + r0 + q * 4;
#pragma unroll
  for (int i = 0; i < RT; ++i)
    if (r0 + i * 16 < p.rank) *reinterpret_cast<f4*>(v + i * 16) = acc[i] + part[0][i][lane] + part[1][i][lane] + part[2][i][lane];
}

// Tiles of 64 rows (many rows a slot: x is what is read).  One workgroup: up
// to 64 ranks and one k range, in steps of 64 values of k that all threads
// bring into LDS by whole 128-byte lines (straight into the operand layout,
// whose neighbouring lanes are 16 different rows, every quad of lanes
// would touch four lines); each wave multiplies 16 of the rows.  The next
// two steps' loads are in flight while one is multiplied (four: no faster).
// 6.4 us for 2048 x 2560, rank 16 (1.6 TB/s, latency); 51 us for 16384 x 4096,
// rank 64 (2.6 TB/s, while the y of the launch before is still written back;
// by itself 35 us).
constexpr int kStage = 72;  // halves from row to row in LDS: 16 lanes' 16 bytes fall into 64 different banks
template <int RT>
__global__ __launch_bounds__(kLoraThreads) void lora_shrink64_kernel(LoraArgs g) {
  __shared__ TileRows<64> tile;
  __shared__ __attribute__((aligned(16))) uint16_t xs[2][64 * kStage];
  __shared__ __attribute__((aligned(16))) uint16_t as[2][RT * 16 * kStage];
  const LoraProblem& p = g.p[blockIdx.z];
  const int chunks = (p.rank + 63) >> 6;
  const int split = blockIdx.y / chunks;
  const int r0 = (blockIdx.y - split * chunks) * 64;
  if (split >= p.splits) return;
  if (!read_tile(g, blockIdx.x, tile)) return;
  if (tile.slot < 0) return;
  const int count = tile.count;
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int li = lane & 15;
  const int q = lane >> 4;

  // staging: 8 threads bring 128 bytes of a row
  constexpr int XL = 2, AL = (RT + 1) / 2;
  const int sr = threadIdx.x >> 3;
  const int sc = (threadIdx.x & 7) * 8;
  gptr<uint16_t> xp[XL], ap[AL];
#pragma unroll
  for (int j = 0; j < XL; ++j) {
    const int at = sr + 32 * j < count ? sr + 32 * j : count - 1;
    xp[j] = to_global(p.x) + (size_t)lora_x_row(g, p, tile.rows[at]) * p.k + sc;
  }
#pragma unroll
  for (int j = 0; j < AL; ++j) {
    const int r = r0 + sr + 32 * j < p.rank ? r0 + sr + 32 * j : p.rank - 1;
    ap[j] = to_global(p.a) + ((size_t)tile.slot * p.rank + r) * p.k + sc;
  }
  u32x4 xr[2][XL], ar[2][AL];  // two steps in flight
  const int kbeg = split * p.k_per_split;
  const int kend = kbeg + p.k_per_split < p.k ? kbeg + p.k_per_split : p.k;
  auto fetch = [&](int set, int k) {
    if (k >= kend) return;
#pragma unroll
    for (int j = 0; j < XL; ++j) xr[set][j] = *(gptr<u32x4>)(xp[j] + k);
#pragma unroll
    for (int j = 0; j < AL; ++j) ar[set][j] = *(gptr<u32x4>)(ap[j] + k);
  };
  auto stage = [&](int set, int buf) {
#pragma unroll
    for (int j = 0; j < XL; ++j) *reinterpret_cast<u32x4*>(&xs[buf][(sr + 32 * j) * kStage + sc]) = xr[set][j];
#pragma unroll
    for (int j = 0; j < AL; ++j)
      if (RT > 1 || sr < 16) *reinterpret_cast<u32x4*>(&as[buf][(sr + 32 * j) * kStage + sc]) = ar[set][j];
  };
  f4 acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = f4{0, 0, 0, 0};
  auto multiply = [&](int buf) {
    if (wave * 16 >= count) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const h8 x = *reinterpret_cast<const h8*>(&xs[buf][(wave * 16 + li) * kStage + h * 32 + q * 8]);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const h8 a = *reinterpret_cast<const h8*>(&as[buf][(i * 16 + li) * kStage + h * 32 + q * 8]);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, x, acc[i], 0, 0, 0);
      }
    }
  };
  fetch(0, kbeg);
  fetch(1, kbeg + 64);
  stage(0, 0);
  fetch(0, kbeg + 128);
  for (int k = kbeg; k < kend; k += 128) {
    __syncthreads();
    if (k + 64 < kend) stage(1, 1);
    fetch(1, k + 192);
    multiply(0);
    if (k + 64 >= kend) break;
    __syncthreads();
    if (k + 128 < kend) stage(0, 0);
    fetch(0, k + 256);
    multiply(1);
  }
  const int at = wave * 16 + li;
  if (at >= count) return;
  float* v = g.v + p.v_offset + ((size_t)split * g.rows + tile.rows[at]) * p.rank_pad + r0 + q * 4;
#pragma unroll
  for (int i = 0; i < RT; ++i)
    if (r0 + i * 16 < p.rank) *reinterpret_cast<f4*>(v + i * 16) = acc[i];
}

// ------------------------------------------------------------------ expand
// The second product of a tile's BM rows and a workgroup's columns, 64 for
// each wave at a time: rows x columns on the matrix cores, D[row][column].
// Block t of a wave's four takes the columns 4 j + t, j = 0 .. 15, so that a
// lane ends with four neighbouring columns of a row and 16 lanes load base
// and store y by 256 bytes (rows in the lanes' place: 64-byte pieces, 222
// against 80 us for 16384 x 2560, rank 64).  base and y pass once and are
// larger than the caches where it matters: non-temporal, 35 against 41 us
// for 2048 x 9728, rank 16 (4.6 TB/s); in place, or between a producer and a
// consumer of y, within 4 % either way.  Where n is no multiple of 4, or y or
// base not on 16 bytes, single columns are loaded and stored one after the
// other (base may be y): whole calls of 2048 x 2560 x 9729 65 us against 45 of
// 9728, 16384 x 4096 x 2561 of rank 64 216 against 108.  RC: ranks in steps of 32.
template <int BM, int RC>
struct Columns {
  static constexpr int CT = BM / 16;
  static constexpr int LD = 2 * RC * 32 + 8;  // halves from row to row of [hi | lo] in LDS
  f4 o[CT][4];  // base: row 4 q + i of block c, four columns
  h8 b[RC][4];

  __device__ __forceinline__ void load(const LoraProblem& p, const TileRows<BM>& tile, int n, int end, bool wide) {
    const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int col = n + t < p.n ? n + t : p.n - 1;
      auto bp = to_global(p.b) + ((size_t)tile.slot * p.n + col) * p.rank;
      const int units = p.rank >> 3;
#pragma unroll
      for (int c = 0; c < RC; ++c) b[c][t] = *(gptr<h8>)(bp + (c * 4 + q < units ? c * 4 + q : units - 1) * 8);
    }
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[c][i] = f4{0, 0, 0, 0};
        const int at = c * 16 + q * 4 + i;
        if (wide && p.base && at < tile.count && n < end)
          o[c][i] = __builtin_nontemporal_load((gptr<f4>)(to_global(p.base) + (size_t)tile.rows[at] * p.n + n));
      }
  }

  __device__ __forceinline__ void finish(const LoraProblem& p, const TileRows<BM>& tile, int n, int end, bool wide,
                                         const half_t* vs, const float* back, float scale) {
    const int li = threadIdx.x & 15;
    const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      if (c * 16 >= tile.count) break;
      f4 acc[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[t] = f4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < 2 * RC; ++k) {
        const h8 v = *reinterpret_cast<const h8*>(&vs[(c * 16 + li) * LD + k * 32 + q * 8]);
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, b[k % RC][t], acc[t], 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = c * 16 + q * 4 + i;
        if (at >= tile.count || n >= end) continue;
        const float undo = back[at];
        float* y = p.y + (size_t)tile.rows[at] * p.n + n;
        if (wide) {
#pragma unroll
          for (int t = 0; t < 4; ++t) o[c][i][t] = fmaf(scale, acc[t][i] * undo, o[c][i][t]);
          __builtin_nontemporal_store(o[c][i], (gptr_mut<f4>)to_global_mut(y));
        } else {
          const float* from = p.base ? p.base + (size_t)tile.rows[at] * p.n + n : nullptr;
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (n + t < end) y[t] = fmaf(scale, acc[t][i] * undo, from ? from[t] : 0.0f);
        }
      }
    }
  }
};

// Rows of a tile without weights of their own: base as it is, or NaN.
template <int BM>
__device__ __forceinline__ void plain_rows(const LoraProblem& p, const TileRows<BM>& tile, int first, int end, bool wide) {
  if (tile.slot == kNone && p.base == p.y) return;
  const int lane = threadIdx.x & 63;
  for (int i = threadIdx.x >> 6; i < tile.count; i += blockDim.x >> 6) {
    const size_t at = (size_t)tile.rows[i] * p.n;
    const float fill = tile.slot == kBad ? __builtin_nanf("") : 0.0f;
    const float* from = tile.slot == kBad ? nullptr : p.base;
    if (wide) {
      for (int n0 = first + lane * 4; n0 < end; n0 += 256 * 8) {  // eight loads in flight
        f4 o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j] = f4{fill, fill, fill, fill};
          if (from && n0 + j * 256 < end) o[j] = *(gptr<f4>)(to_global(from) + at + n0 + j * 256);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (n0 + j * 256 < end) *reinterpret_cast<f4*>(p.y + at + n0 + j * 256) = o[j];
      }
    } else {
      for (int n = first + lane; n < end; n += 64) p.y[at + n] = from ? from[at + n] : fill;
    }
  }
}

// v of row m, of which this thread (u0 of TPR neighbours) holds UT units of 8
// ranks (f[j]: unit u0 + j * TPR), into LDS as [hi | lo].
template <int RC, int LD, int TPR, int UT>
__device__ __forceinline__ void split_row(const f4 (&f)[UT][2], int m, int u0, half_t* vs, float* back) {
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < UT; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = fabsf(f[j][i >> 2][i & 3]);
      if (a < __builtin_inff()) top = fmaxf(top, a);  // what is not finite stays so
    }
#pragma unroll
  for (int d = 1; d < TPR; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
  const int ex = __builtin_amdgcn_frexp_expf(top) - 15;
  if (u0 == 0) back[m] = ldexpf(1.0f, ex);
#pragma unroll
  for (int j = 0; j < UT; ++j) {
    const int u = u0 + j * TPR;
    if (u >= 4 * RC) break;
    h8 hi, lo;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = ldexpf(f[j][i >> 2][i & 3], -ex);
      hi[i] = (half_t)x;
      lo[i] = (half_t)(fabsf(x) < __builtin_inff() ? x - (float)hi[i] : 0.0f);
    }
    *reinterpret_cast<h8*>(&vs[m * LD + u * 8]) = hi;
    *reinterpret_cast<h8*>(&vs[m * LD + RC * 32 + u * 8]) = lo;
  }
}

__device__ __forceinline__ bool wide_columns(const LoraProblem& p) {
  return (p.n & 3) == 0 && ((uintptr_t)p.y & 15) == 0 && ((uintptr_t)p.base & 15) == 0;
}

template <bool ROUTED, int BM, int RC>
__global__ __launch_bounds__(kLoraThreads) void lora_expand_kernel(LoraArgs g) {
  using C = Columns<BM, RC>;
  __shared__ TileRows<BM> tile;
  __shared__ __attribute__((aligned(16))) half_t vs[BM * C::LD];
  __shared__ float back[BM];  // what undoes a row's power of two
  const LoraProblem& p = g.p[blockIdx.z];
  const int first = blockIdx.y * g.columns;
  if (first >= p.n) return;
  if (!(ROUTED ? read_tile(g, blockIdx.x, tile) : find_tile<kLoraThreads>(g, blockIdx.x, tile))) return;
  const int end = first + g.columns < p.n ? first + g.columns : p.n;
  const bool wide = wide_columns(p);
  if (tile.slot < 0) {
    plain_rows(p, tile, first, end, wide);
    return;
  }
  const int step = (threadIdx.x >> 6) * 64 + (threadIdx.x & 15) * 4;
  C cols;
  cols.load(p, tile, first + step, end, wide);  // in flight while v is formed

  constexpr int TPR = kLoraThreads / BM;               // threads of a row
  constexpr int UT = 4 * RC > TPR ? 4 * RC / TPR : 1;  // units of a thread
  const int m = threadIdx.x / TPR;
  const int u0 = threadIdx.x % TPR;
  const int row = tile.rows[m < tile.count ? m : tile.count - 1];
  f4 f[UT][2];
#pragma unroll
  for (int j = 0; j < UT; ++j) {
    f[j][0] = f[j][1] = f4{0, 0, 0, 0};
    if ((u0 + j * TPR) * 8 < p.rank) {
      auto vp = to_global(g.v) + p.v_offset + (size_t)row * p.rank_pad + (u0 + j * TPR) * 8;
      for (int s = 0; s < p.splits; ++s, vp += (size_t)g.rows * p.rank_pad) {
        f[j][0] += *(gptr<f4>)vp;
        f[j][1] += *(gptr<f4>)(vp + 4);
      }
    }
  }
  split_row<RC, C::LD, TPR, UT>(f, m, u0, vs, back);
  __syncthreads();

  const float scale = g.scales ? g.scales[tile.slot / g.experts] : 1.0f;
  for (int n = first;;) {
    cols.finish(p, tile, n + step, end, wide, vs, back, scale);
    n += kLoraThreads;
    if (n >= end) break;
    cols.load(p, tile, n + step, end, wide);
  }
}

// ---------------------------------------------------------------- few rows
// Few rows, a small A of rank up to 64: both products in one launch, as dot
// products of up to kFewRows rows with lanes along memory: a load of 16
// bytes a lane covers 1 KB of one row of A (or of neighbouring rows of B),
// where the matrix cores' operand layout touches 16 rows with neighbouring
// lanes and L1 gives a third of the rate (15 against 44 bytes a clock and CU).
// Every workgroup forms its tile's v itself (the others of the tile read the
// same A from L2), then goes on to its columns, whose first loads it has
// issued before.  Tiles of two rows against four: 64 rows on one slot 7.1 / 9.3
// us, 256 rows on 64 slots 10.6 / 15.2 (rank 16, 2560, 4096), as more tiles are
// at work and a wave holds fewer sums.  One row of 1024 x 2048, rank 16:
// 4.5-5.0 us, a launch and three dependent loads (ids, A, v through LDS).
constexpr int kFewThreads = 512;
constexpr int kFewWaves = kFewThreads / 64;
constexpr int kFewRows = 2;

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float lane_add(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, false);
  return v + __builtin_bit_cast(float, o);
}
// The sum over the wave, in its last lane: within the rows of 16, then across
// them (lanes of rows that receive nothing add zero).
__device__ __forceinline__ float sum_to_last(float v) {
  v = lane_add<0xB1>(v);
  v = lane_add<0x4E>(v);
  v = lane_add<0x141>(v);
  v = lane_add<0x140>(v);
  v = lane_add<0x142, 0xA>(v);
  return lane_add<0x143, 0xC>(v);
}

// v of NR rows by dot products: wave w forms rank / 8 of the ranks (at most U).
template <int U, int NR>
__device__ __forceinline__ void few_rows_shrink(const LoraArgs& g, const LoraProblem& p, const TileRows<kFewRows>& tile,
                                                float (*v)[64]) {
  constexpr int UK = U <= 2 ? 4 / NR : U == 4 && NR == 1 ? 2 : 1;  // steps of 512 values of k in flight
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int ranks = p.rank >> 3;
  auto ap = to_global(p.a) + ((size_t)tile.slot * p.rank + wave * ranks) * p.k;
  gptr<uint16_t> xp[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r)
    xp[r] = to_global(p.x) + (size_t)lora_x_row(g, p, tile.rows[r < tile.count ? r : tile.count - 1]) * p.k;
  float acc[U][NR];
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[i][r] = 0.0f;
  // Lanes past the end of k load nothing: they leave the loop, or have zeros
  // for both A and x (an infinity loaded in their place, times zero, is NaN).
  for (int k0 = lane * 8; k0 < p.k; k0 += 512 * UK) {
    u32x4 a[UK][U] = {}, x[UK][NR] = {};
#pragma unroll
    for (int u = 0; u < UK; ++u) {
      const int k = k0 + u * 512;
      if (u > 0 && k >= p.k) break;
#pragma unroll
      for (int i = 0; i < U; ++i) a[u][i] = *(gptr<u32x4>)(ap + (size_t)(i < ranks ? i : 0) * p.k + k);
#pragma unroll
      for (int r = 0; r < NR; ++r) x[u][r] = *(gptr<u32x4>)(xp[r] + k);
    }
#pragma unroll
    for (int u = 0; u < UK; ++u)
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][r] = dot2(a[u][i][j], x[u][r][j], acc[i][r]);
  }
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float s = sum_to_last(acc[i][r]);
      if (lane == 63 && i < ranks) v[r][wave * ranks + i] = s;
    }
}

// A wave's columns by dot products: U neighbouring lanes (rank / 8 of them at
// work, a power of two in all) share a column, a load covers 64 / U columns,
// four loads are one turn.  Lane u of
// the U adds to base and stores the rows u, u + U, ... (RH of them; rows and
// columns past the end are loaded again from the last one and not stored).
template <int U, int NR>
struct FewColumns {
  static constexpr int kPerLoad = 64 / U;
  static constexpr int RH = (NR + U - 1) / U;
  const LoraProblem& p;
  gptr<uint16_t> bp;
  size_t row[RH];
  bool live[RH];
  int unit, col;
  h8 b[4];
  float o[4][RH];

  __device__ __forceinline__ FewColumns(const LoraProblem& p_, const TileRows<kFewRows>& tile) : p(p_) {
    unit = threadIdx.x & (U - 1);
    col = (threadIdx.x & 63) / U;
    const int units = p.rank >> 3;
    bp = to_global(p.b) + (size_t)tile.slot * p.n * p.rank + (unit < units ? unit : units - 1) * 8;
#pragma unroll
    for (int h = 0; h < RH; ++h) {
      const int r = h * U + unit;
      live[h] = r < tile.count;
      row[h] = (size_t)tile.rows[live[h] ? r : tile.count - 1] * p.n;
    }
  }

  __device__ __forceinline__ void load(int n0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + j * kPerLoad + col < p.n ? n0 + j * kPerLoad + col : p.n - 1;
      b[j] = *(gptr<h8>)(bp + (size_t)n * p.rank);
#pragma unroll
      for (int h = 0; h < RH; ++h) o[j][h] = 0.0f;
    }
    if (p.base == nullptr) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + j * kPerLoad + col < p.n ? n0 + j * kPerLoad + col : p.n - 1;
#pragma unroll
      for (int h = 0; h < RH; ++h) o[j][h] = to_global(p.base)[row[h] + n];
    }
  }

  __device__ __forceinline__ void finish(int n0, int end, const float (&v)[NR][8], float scale) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + j * kPerLoad + col;
      float d[RH * U];
#pragma unroll
      for (int r = 0; r < RH * U; ++r) {
        d[r] = 0.0f;
        if (r >= NR) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) d[r] = fmaf((float)b[j][i], v[r][i], d[r]);
        if (U > 1) d[r] = lane_add<0xB1>(d[r]);
        if (U > 2) d[r] = lane_add<0x4E>(d[r]);
        if (U > 4) d[r] = lane_add<0x141>(d[r]);
      }
#pragma unroll
      for (int h = 0; h < RH; ++h) {
        float mine = d[h * U];
#pragma unroll
        for (int u = 1; u < U; ++u) mine = unit == u ? d[h * U + u] : mine;
        if (live[h] && n < end) to_global_mut(p.y)[row[h] + n] = fmaf(scale, mine, o[j][h]);
      }
    }
  }
};

template <int U, int NR>
__device__ __forceinline__ void few_rows(const LoraArgs& g, const LoraProblem& p, const TileRows<kFewRows>& tile,
                                         int first, int end, float (*vs)[64]) {
  using C = FewColumns<U, NR>;
  const int wave = threadIdx.x >> 6;
  const float scale = g.scales ? g.scales[tile.slot / g.experts] : 1.0f;
  C cols(p, tile);
  int n0 = first + wave * 4 * C::kPerLoad;
  cols.load(n0);
  few_rows_shrink<U, NR>(g, p, tile, vs);
  __syncthreads();
  float v[NR][8];
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[r][i] = cols.unit * 8 < p.rank ? vs[r][cols.unit * 8 + i] : 0.0f;
  for (;;) {
    cols.finish(n0, end, v, scale);
    n0 += kFewWaves * 4 * C::kPerLoad;
    if (n0 >= end) break;
    cols.load(n0);
  }
}

template <bool ROUTED, int U>
__global__ __launch_bounds__(kFewThreads) void lora_few_kernel(LoraArgs g) {
  __shared__ TileRows<kFewRows> tile;
  __shared__ float vs[kFewRows][64];
  // the grid's second dimension counts the column ranges of all problems
  int problem = 0;
  while (problem + 1 < g.count && (int)blockIdx.y >= g.first_range[problem + 1]) ++problem;
  const LoraProblem& p = g.p[problem];
  const int first = ((int)blockIdx.y - g.first_range[problem]) * g.columns;
  if (!(ROUTED ? read_tile(g, blockIdx.x, tile) : find_tile<kFewThreads>(g, blockIdx.x, tile))) return;
  const int end = first + g.columns < p.n ? first + g.columns : p.n;
  if (tile.slot < 0) {
    plain_rows(p, tile, first, end, wide_columns(p));
    return;
  }
  if (tile.count == 1) few_rows<U, 1>(g, p, tile, first, end, vs);
  else few_rows<U, kFewRows>(g, p, tile, first, end, vs);
}

// ---------------------------------------------------------------- fused 16
// Sorted tiles of 16 rows, a small A: both products in one launch on the
// matrix cores, as above: the workgroup forms its tile's v (eight waves taking
// turns at 64 values of k, joined in LDS) and goes on to its columns, whose
// first loads it has issued before.  24.7 us for 4096 pairs on 512 slots, 768 x
// 2048, rank 16 (119 MB, 4.8 TB/s: the rate of a large copy).
template <int RT>
__global__ __launch_bounds__(kFewThreads) void lora_fused16_kernel(LoraArgs g) {
  constexpr int RC = (RT + 1) / 2;
  using C = Columns<16, RC>;
  __shared__ TileRows<16> tile;
  __shared__ f4 part[kFewWaves][RT][64];
  __shared__ __attribute__((aligned(16))) half_t vs[16 * C::LD];
  __shared__ float back[16];
  const LoraProblem& p = g.p[blockIdx.z];
  const int first = blockIdx.y * g.columns;
  if (first >= p.n) return;
  if (!read_tile(g, blockIdx.x, tile)) return;
  const int end = first + g.columns < p.n ? first + g.columns : p.n;
  const bool wide = wide_columns(p);
  if (tile.slot < 0) {
    plain_rows(p, tile, first, end, wide);
    return;
  }
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int li = lane & 15;
  const int q = lane >> 4;
  const int row = tile.rows[li < tile.count ? li : tile.count - 1];
  auto xp = to_global(p.x) + (size_t)lora_x_row(g, p, row) * p.k + q * 16;
  gptr<uint16_t> ap[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = i * 16 + li < p.rank ? i * 16 + li : p.rank - 1;
    ap[i] = to_global(p.a) + ((size_t)tile.slot * p.rank + r) * p.k + q * 16;
  }
  f4 acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = f4{0, 0, 0, 0};
#pragma unroll 2
  for (int k = wave * 64; k < p.k; k += kFewWaves * 64) {
    const h8 x0 = *(gptr<h8>)(xp + k), x1 = *(gptr<h8>)(xp + k + 8);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const h8 a0 = *(gptr<h8>)(ap[i] + k), a1 = *(gptr<h8>)(ap[i] + k + 8);
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, x0, acc[i], 0, 0, 0);
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, x1, acc[i], 0, 0, 0);
    }
  }
  const int step = wave * 64 + li * 4;
  C cols;
  cols.load(p, tile, first + step, end, wide);
#pragma unroll
  for (int i = 0; i < RT; ++i) part[wave][i][lane] = acc[i];
  __syncthreads();
  // thread (m, u0 of 32): the 8 ranks of unit u0 are two quads of a block's 16
  constexpr int TPR = kFewThreads / 16;
  const int m = threadIdx.x / TPR;
  const int u0 = threadIdx.x % TPR;
  f4 f[1][2];
  f[0][0] = f[0][1] = f4{0, 0, 0, 0};
  if (u0 * 8 < p.rank) {
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
      f[0][0] += part[w][u0 >> 1][(u0 & 1) * 32 + m];
      f[0][1] += part[w][u0 >> 1][(u0 & 1) * 32 + 16 + m];
    }
  }
  split_row<RC, C::LD, TPR, 1>(f, m, u0, vs, back);
  __syncthreads();

  const float scale = g.scales ? g.scales[tile.slot / g.experts] : 1.0f;
  for (int n = first;;) {
    cols.finish(p, tile, n + step, end, wide, vs, back, scale);
    n += kFewThreads;
    if (n >= end) break;
    cols.load(p, tile, n + step, end, wide);
  }
}

// ------------------------------------------------------------------- route
// Rows sorted by slot, and tiles of up to tile_rows rows of one slot, as
// two launches over chunks of the rows (one if there is one chunk): count
// the slots of each chunk, then place its rows behind those of the chunks
// before it.  Buckets slots and slots + 1 hold the rows without adapter and
// those with bad ids.  Latency of loads, LDS atomics and a scan: 4.6 us for 2048
// rows, 6.2 us for 4096 pairs, 4.8 + 5.0 us for 16384 rows.
constexpr int kRouteThreads = 1024;
static_assert(kFewRows <= 16, "the smallest tile");
static_assert(kLoraOneChunk == 4 * kRouteThreads, "one chunk's rows are four of each thread");
constexpr int kLoraBuckets = kLoraMaxSlots + 2;

constexpr int kBatch = 4;  // rows of a thread whose ids are loaded together

// The buckets of rows p, p + kRouteThreads, ...; -1 from row `end` on.
__device__ __forceinline__ void lora_buckets(const LoraArgs& g, int p, int end, int (&b)[kBatch]) {
  int a[kBatch], e[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int at = p + i * kRouteThreads < end ? p + i * kRouteThreads : end - 1;
    a[i] = g.adapter_ids[g.top_k == 1 ? at : at / g.top_k];
    e[i] = g.expert_ids ? g.expert_ids[at] : 0;
  }
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const bool ok = a[i] >= 0 && a[i] < g.adapters && e[i] >= 0 && e[i] < g.experts;
    b[i] = p + i * kRouteThreads >= end ? -1 : ok ? a[i] * g.experts + e[i] : a[i] == -1 ? g.slots : g.slots + 1;
  }
}

// Adds one to the row's counter and returns what it was.  A wave whose rows
// all share a bucket, as in a prompt, does so once.
__device__ __forceinline__ int lora_take(int32_t* counters, int b) {
  const int first = __builtin_amdgcn_readfirstlane(b);
  if (__all(b == first)) {
    int at = 0;
    const int lane = threadIdx.x & 63;
    if (lane == 0 && first >= 0) at = atomicAdd(&counters[first], 64);
    return __builtin_amdgcn_readfirstlane(at) + lane;
  }
  return b >= 0 ? atomicAdd(&counters[b], 1) : 0;
}

__global__ __launch_bounds__(kRouteThreads) void lora_count_kernel(LoraArgs g) {
  __shared__ int32_t h[kLoraBuckets];
  const int buckets = g.slots + 2;
  for (int i = threadIdx.x; i < buckets; i += kRouteThreads) h[i] = 0;
  __syncthreads();
  const int p0 = blockIdx.x * g.chunk;
  const int p1 = p0 + g.chunk < g.rows ? p0 + g.chunk : g.rows;
  for (int base = p0; base < p1; base += kBatch * kRouteThreads) {
    int b[kBatch];
    lora_buckets(g, base + threadIdx.x, p1, b);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) lora_take(h, b[i]);
  }
  __syncthreads();
  int32_t* out = g.plan + g.plan_counts + (size_t)blockIdx.x * buckets;
  for (int i = threadIdx.x; i < buckets; i += kRouteThreads) out[i] = h[i];
}

__global__ __launch_bounds__(kRouteThreads) void lora_place_kernel(LoraArgs g) {
  __shared__ int32_t total[kLoraBuckets];
  __shared__ int32_t cursor[kLoraBuckets];  // rows in earlier chunks, then the next place
  __shared__ int32_t wave_rows[kRouteThreads / 64], wave_tiles[kRouteThreads / 64];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = tid >> 6;
  const int buckets = g.slots + 2;
  const int p0 = blockIdx.x * g.chunk;
  const int p1 = p0 + g.chunk < g.rows ? p0 + g.chunk : g.rows;
  // the chunk's first rows stay in registers: all of them where there is one
  // chunk (kLoraOneChunk rows), whose counting also places them
  int b[kBatch], at[kBatch];
  lora_buckets(g, p0 + tid, p1, b);
  for (int i = tid; i < buckets; i += kRouteThreads) total[i] = cursor[i] = 0;
  __syncthreads();
  if (g.chunks == 1) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) at[i] = lora_take(total, b[i]);
  } else {
    const int32_t* counts = g.plan + g.plan_counts;
    const int words = buckets * g.chunks;
    for (int base = tid; base < words; base += kBatch * kRouteThreads) {
      int n[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) n[i] = base + i * kRouteThreads < words ? counts[base + i * kRouteThreads] : 0;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (n[i] == 0) continue;
        const int c = (base + i * kRouteThreads) / buckets;
        const int k = base + i * kRouteThreads - c * buckets;
        atomicAdd(&total[k], n[i]);
        if (c < (int)blockIdx.x) atomicAdd(&cursor[k], n[i]);
      }
    }
  }
  __syncthreads();
  // thread i scans `per` neighbouring buckets, then the threads are scanned
  const int per = (buckets + kRouteThreads - 1) / kRouteThreads;
  int rows = 0, tiles = 0;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    const int n = b < buckets ? total[b] : 0;
    rows += n;
    tiles += (n + g.tile_rows - 1) / g.tile_rows;
  }
  int row_sum = rows, tile_sum = tiles;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int r = __shfl_up(row_sum, d, 64), t = __shfl_up(tile_sum, d, 64);
    if (lane >= d) {
      row_sum += r;
      tile_sum += t;
    }
  }
  if (lane == 63) {
    wave_rows[wave] = row_sum;
    wave_tiles[wave] = tile_sum;
  }
  __syncthreads();
  int start = row_sum - rows, tile = tile_sum - tiles;
  for (int w = 0; w < wave; ++w) {
    start += wave_rows[w];
    tile += wave_tiles[w];
  }
  LoraTile* list = reinterpret_cast<LoraTile*>(g.plan + g.plan_tiles);
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b >= buckets) break;
    const int n = total[b];
    cursor[b] += start;
    if (blockIdx.x == 0) {
      const int slot = b < g.slots ? b : b == g.slots ? kNone : kBad;
      for (int j = 0; j < n; j += g.tile_rows)
        list[tile++] = LoraTile{slot, start + j, n - j < g.tile_rows ? n - j : g.tile_rows, 0};
    }
    start += n;
  }
  if (blockIdx.x == 0 && tid == kRouteThreads - 1) g.plan[0] = tile;
  __syncthreads();
  int32_t* sorted = g.plan + kLoraPlanHeader;
  if (g.chunks == 1) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (b[i] >= 0) sorted[cursor[b[i]] + at[i]] = p0 + tid + i * kRouteThreads;
    return;
  }
  for (int base = p0; base < p1; base += kBatch * kRouteThreads) {
    if (base > p0) lora_buckets(g, base + tid, p1, b);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int to = lora_take(cursor, b[i]);
      if (b[i] >= 0) sorted[to] = base + tid + i * kRouteThreads;
    }
  }
}

// -------------------------------------------------------------------- host

static size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }

static long lora_tiles(int rows, int tile_rows, int slots) {
  const long most = (long)rows / tile_rows + slots + 2;  // a last tile of each bucket besides the whole ones
  return most < rows ? most : rows;
}

// The way a call takes, its tile height, splits of k, chunks of the route and
// the places of everything in the workspace; its size.  By total time of the
// launches of a call (k and n as given, microseconds):
//   one launch of dot products (few) against two on the matrix cores, 64
//     rows: 7.0 / 13.6 (rank 16, 2560, 4096), 9.9 / 16.2 (rank 16, 9728,
//     4096), 14.7 / 19.2 (rank 32, 9728: A of 608 KB), 34.9 / 32.0 (rank 64,
//     9728: 1.2 MB); 256 rows of rank 64 (2560, 4096): 35.1 / 29.8, of rank
//     32: 20.2 / 22.3; 512 rows of rank 16 against sorted ones (1024, 1024):
//     9.7 / 13.9.  Hence A up to 640 KB and rows x rank up to 8192.
//   sorted rows, tiles of 2 for dot products against fused tiles of 16 (768,
//     2048): rank 8 with 4 rows a slot 20.4 / 21.7 and with 8 35.5 / 27.7,
//     rank 16 with 2 18.3 / 21.7 and with 4 24.8 / 24.2, rank 32 with 1
//     37.6 / 36.3 and with 2 30.2 / 24.9.  Hence rows x rank up to 48 a slot.
//   sorted rows in tiles of 16, one launch of both products against two (4096
//     pairs on 512 slots): 28.5 / 33.7 (rank 16, 768, 2048), 53.2 / 57.5
//     (rank 64, 768, 2048: A of 96 KB), 36.4 / 37.2 (rank 32, 2048, 768),
//     58.5 / 58.2 (rank 64, 2048, 768: 256 KB).  Hence A up to 128 KB.
//   two launches on the matrix cores, tiles found by ballots against sorted
//     rows (2560, 4096): 8 rows of rank 128 12.1 / 14.8 on one slot and 11.7 /
//     15.0 on 8, 64 rows on 64 slots 29.8 / 33.6; 256 rows on 256 slots of rank
//     64 51.2 / 51.7, of rank 128 99.8 / 101.1.  Rows that share slots are sorted
//     faster from 32 on: 32 rows of rank 128 on one slot 16.6 / 15.6, 256 on 8
//     of rank 64 29.7 / 16.7, on one 47.3 / 16.7.  Hence ballots up to
//     kLoraDirectRows (a thread for each row), which is late for such calls.
//   sorted rows, tiles of 16 against tiles of 64 (2560, 4096): rank 64 with 24
//     rows a slot, 2048 rows 48.0 / 42.2 and 8192 rows 156.5 / 133.1; with 20,
//     48.4 / 47.3 and 176.6 / 149.8; with 12, 52.8 / 60.5 and 203.8 / 201.5.
//     Rank 128 with 24, 2048 rows 62.4 / 66.1; with 12, 80.3 / 111.7.  Hence 24
//     rows a slot.  520 rows on one slot, rank 64 19.8 / 22.5, rank 128 25.8 /
//     27.7, rank 16 22.3 / 18.1; 1000 rows on 10 slots 26.9 / 24.1, 38.6 / 32.4
//     and 26.5 / 19.1.  Hence 1024 rows, which is late for small ranks.
//     [hi | lo] of a rank over 128 outgrows LDS in tiles of 64.
size_t lora_layout(LoraArgs& g) {
  int rank = 0;
  long a_bytes = 0;  // the largest A of a slot
  for (int i = 0; i < g.count; ++i) {
    rank = g.p[i].rank > rank ? g.p[i].rank : rank;
    const long a = 2L * g.p[i].rank * g.p[i].k;
    a_bytes = a > a_bytes ? a : a_bytes;
  }
  const bool small = rank <= 64 && a_bytes <= 640 * 1024;
  g.way = small && g.rows <= kLoraFewRows && rank * g.rows <= 8192 ? kLoraFew
          : g.rows <= kLoraDirectRows                              ? kLoraDirect
                                                                   : kLoraRouted;
  const bool direct = g.way == kLoraFew || g.way == kLoraDirect;
  g.tile_rows = !direct && small && (long)g.rows * rank <= 48L * g.slots                   ? kFewRows
                : direct || rank > 128 || g.rows < 24 * g.slots || g.rows < 1024 ? 16
                                                                                  : 64;
  if (!direct && g.tile_rows == 16 && rank <= 64 && a_bytes <= 128 * 1024) g.way = kLoraRouted16;
  size_t ints = 0;
  g.tiles = g.rows;
  if (!direct) {
    const int buckets = g.slots + 2;
    g.chunks = kLoraCountWords / buckets;
    g.chunks = g.chunks < 1 ? 1 : g.chunks > 64 ? 64 : g.chunks;
    g.chunk = (g.rows + g.chunks - 1) / g.chunks;
    g.chunk = g.chunk < kLoraChunkMin ? kLoraChunkMin : g.chunk;
    if (g.rows <= kLoraOneChunk) g.chunk = g.rows;
    g.chunks = (g.rows + g.chunk - 1) / g.chunk;
    g.tiles = lora_tiles(g.rows, g.tile_rows, g.slots);
    g.plan_tiles = up(kLoraPlanHeader + (size_t)g.rows, 4);
    g.plan_counts = g.plan_tiles + 4 * (size_t)g.tiles;
    ints = g.plan_counts + (g.chunks > 1 ? (size_t)g.chunks * buckets : 0);
  }
  size_t at = up(ints * 4, 256) / 4;  // in floats
  for (int i = 0; i < g.count; ++i) {
    LoraProblem& p = g.p[i];
    int splits = (p.k + 511) / 512;
    if (g.tile_rows == 64) {
      const long wgs = (long)(g.rows + 63) / 64 * ((p.rank + 63) / 64);
      const long want = (256 + wgs - 1) / wgs;
      splits = splits < want ? splits : (int)want;
    }
    splits = splits > 8 ? 8 : splits;
    const int unit = g.tile_rows == 16 ? 256 : 64;
    p.k_per_split = ((p.k + splits - 1) / splits + unit - 1) / unit * unit;
    p.splits = (p.k + p.k_per_split - 1) / p.k_per_split;
    p.rank_pad = (p.rank + 15) / 16 * 16;
    p.v_offset = at;
    at += up((size_t)p.splits * g.rows * p.rank_pad, 64);
  }
  return at * sizeof(float);
}

template <bool ROUTED, int BM>
static void launch_lora_products(LoraArgs g, hipStream_t st) {
  int shrink_y = 1, rank = 1, n = 1;
  long blocks = 0;  // tiles x 256 columns of all problems
  for (int i = 0; i < g.count; ++i) {
    const LoraProblem& p = g.p[i];
    const int y = p.splits * ((p.rank + 63) / 64);
    shrink_y = y > shrink_y ? y : shrink_y;
    rank = p.rank > rank ? p.rank : rank;
    n = p.n > n ? p.n : n;
    blocks += (long)((p.n + 255) / 256) * ((g.rows + BM - 1) / BM);
  }
  const unsigned tiles = (unsigned)(ROUTED ? up(g.tiles, kXcds) : g.tiles);
  const dim3 block(kLoraThreads);
  const dim3 sg(tiles, shrink_y, g.count);
  if constexpr (BM == 64) {
    if (rank <= 16) hipLaunchKernelGGL(lora_shrink64_kernel<1>, sg, block, 0, st, g);
    else if (rank <= 32) hipLaunchKernelGGL(lora_shrink64_kernel<2>, sg, block, 0, st, g);
    else hipLaunchKernelGGL(lora_shrink64_kernel<4>, sg, block, 0, st, g);
  } else {
    if (rank <= 16) hipLaunchKernelGGL((lora_shrink16_kernel<ROUTED, 1>), sg, block, 0, st, g);
    else if (rank <= 32) hipLaunchKernelGGL((lora_shrink16_kernel<ROUTED, 2>), sg, block, 0, st, g);
    else hipLaunchKernelGGL((lora_shrink16_kernel<ROUTED, 4>), sg, block, 0, st, g);
  }
  // A workgroup's columns.  256 against 512 at once (calls of rank 16, k 2560):
  // 2048 rows, 4096 + 1024 + 1024 columns (768 blocks) 31.5 / 40.4 us; 9728
  // columns (1216) 46.0 / 45.0; 9728 + 9728 (2432) 77.7 / 72.7; 8192 rows,
  // 4096 + 1024 + 1024 columns 100.3 / 97.4.  Over 512 the last workgroups of a
  // launch run alone for too long (1280: 86.9 and 112.2).
  g.columns = blocks >= 1024 ? 512 : 256;
  const dim3 eg(tiles, (n + g.columns - 1) / g.columns, g.count);
  if (rank <= 32) hipLaunchKernelGGL((lora_expand_kernel<ROUTED, BM, 1>), eg, block, 0, st, g);
  else if (rank <= 64) hipLaunchKernelGGL((lora_expand_kernel<ROUTED, BM, 2>), eg, block, 0, st, g);
  else if (rank <= 128) hipLaunchKernelGGL((lora_expand_kernel<ROUTED, BM, 4>), eg, block, 0, st, g);
  else if constexpr (BM == 16) hipLaunchKernelGGL((lora_expand_kernel<ROUTED, BM, 8>), eg, block, 0, st, g);
}

// Tiles of `height` rows, at most: whole ones and a last one of each slot.
static long likely_tiles(const LoraArgs& g, int height) {
  const long spread = (long)g.rows / height + g.slots;
  return spread < g.rows ? spread : g.rows;
}

static void launch_lora_fused16(LoraArgs g, hipStream_t st) {
  int n = 1, rank = 8;
  long columns = 0;  // of all problems
  for (int i = 0; i < g.count; ++i) {
    n = g.p[i].n > n ? g.p[i].n : n;
    rank = g.p[i].rank > rank ? g.p[i].rank : rank;
    columns += g.p[i].n;
  }
  const long per = (columns * likely_tiles(g, 16) / 512 + 511) / 512 * 512;
  g.columns = (int)(per < 512 ? 512 : per < 4096 ? per : 4096);
  const dim3 grid((unsigned)up(g.tiles, kXcds), (n + g.columns - 1) / g.columns, g.count), block(kFewThreads);
  if (rank <= 16) hipLaunchKernelGGL(lora_fused16_kernel<1>, grid, block, 0, st, g);
  else if (rank <= 32) hipLaunchKernelGGL(lora_fused16_kernel<2>, grid, block, 0, st, g);
  else hipLaunchKernelGGL(lora_fused16_kernel<4>, grid, block, 0, st, g);
}

template <bool ROUTED>
static void launch_lora_few(LoraArgs g, hipStream_t st) {
  int rank = 8, ranges = 0;
  long columns = 0;  // of all problems
  for (int i = 0; i < g.count; ++i) {
    rank = g.p[i].rank > rank ? g.p[i].rank : rank;
    columns += g.p[i].n;
  }
  const int units = rank <= 8 ? 1 : rank <= 16 ? 2 : rank <= 32 ? 4 : 8;
  const int turn = kFewWaves * 4 * 64 / units;  // columns of a workgroup's turn
  long per = (columns * likely_tiles(g, kFewRows) + 255) / 256;  // one workgroup a CU
  per = (per + turn - 1) / turn * turn;
  g.columns = (int)(per < 4096 ? per : 4096);
  for (int i = 0; i < g.count; ++i) {
    g.first_range[i] = ranges;
    ranges += (g.p[i].n + g.columns - 1) / g.columns;
  }
  const dim3 grid((unsigned)(ROUTED ? up(g.tiles, kXcds) : g.rows), ranges), block(kFewThreads);
  switch (units) {
    case 1: hipLaunchKernelGGL((lora_few_kernel<ROUTED, 1>), grid, block, 0, st, g); break;
    case 2: hipLaunchKernelGGL((lora_few_kernel<ROUTED, 2>), grid, block, 0, st, g); break;
    case 4: hipLaunchKernelGGL((lora_few_kernel<ROUTED, 4>), grid, block, 0, st, g); break;
    default: hipLaunchKernelGGL((lora_few_kernel<ROUTED, 8>), grid, block, 0, st, g); break;
  }
}

hipError_t launch_lora(const LoraArgs& g, hipStream_t st) {
  if (g.way == kLoraFew) {
    launch_lora_few<false>(g, st);
    return hipGetLastError();
  }
  if (g.way == kLoraDirect) {
    launch_lora_products<false, 16>(g, st);
    return hipGetLastError();
  }
  if (g.chunks > 1) hipLaunchKernelGGL(lora_count_kernel, dim3(g.chunks), dim3(kRouteThreads), 0, st, g);
  hipLaunchKernelGGL(lora_place_kernel, dim3(g.chunks), dim3(kRouteThreads), 0, st, g);
  if (g.tile_rows == kFewRows) launch_lora_few<true>(g, st);
  else if (g.way == kLoraRouted16) launch_lora_fused16(g, st);
  else if (g.tile_rows == 64) launch_lora_products<true, 64>(g, st);
  else launch_lora_products<true, 16>(g, st);
  return hipGetLastError();
}

}  // namespace qmm
