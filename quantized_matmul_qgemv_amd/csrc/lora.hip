// Low-rank adapters of many requests beside a shared projection:
//
//   y[p, :] = base[p, :] + scale[a] * B_s (A_s x[row(p), :]),   a = adapter_ids[p / top_k]
//
// with s = a (dense projections) or a * experts + expert_ids[p] (the experts'
// products of a routed layer), A_s [rank, k] and B_s [n, rank] in fp16.
// a = -1 leaves the row as base has it; an id out of range makes it NaN.
//
// Two launches over tiles of rows that share a slot s (up to BM rows each):
//   shrink  v = A_s x: matrix cores, ranks x rows, k split over waves and
//           workgroups; every split leaves its fp32 partial in the workspace.
//   expand  sums the partials of a row in split order and multiplies by B_s
//           on the matrix cores.  v is an fp32 number and the matrix cores
//           take fp16: each row is scaled by a power of two that brings its
//           largest value into [2^14, 2^15) and split into v = hi + lo, both
//           fp16 (error 2^-23 of that largest value), which stand side by
//           side along the contraction: [hi | lo] x [B | B].
// Up to kLoraDirectRows rows every workgroup finds its tile itself, from
// ballots over the ids of all rows.  Beyond that two short launches sort the
// rows by slot into a tile list first.
//
// Every row is computed on its own (neither its tile nor its place in it
// enters the sums), so results do not depend on scheduling.
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

// A workgroup's rows of one slot.
template <int BM>
struct TileRows {
  int32_t rows[BM];
  int32_t slot, count;
};

// Direct: the workgroup of row p owns the tile that starts at p, if an equal
// number of rows with p's slot, a multiple of BM, comes before it.
template <int BM>
__device__ __forceinline__ bool find_tile(const LoraArgs& g, int p, TileRows<BM>& t, uint64_t* masks) {
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int s = tid < g.rows ? lora_slot(g, tid) : 0;
  if (tid == p) t.slot = s;
  __syncthreads();
  const bool same = tid < g.rows && s == t.slot;
  const uint64_t m = __ballot(same);
  if (lane == 0) masks[tid >> 6] = m;
  __syncthreads();
  int before = 0, total = 0, mine = 0;
#pragma unroll
  for (int w = 0; w < kLoraDirectRows / 64; ++w) {
    const uint64_t b = masks[w];
    const int lo = p - w * 64, li = tid - w * 64;
    before += __popcll(lo >= 64 ? b : lo > 0 ? b & ((1ull << lo) - 1) : 0);
    mine += __popcll(li >= 64 ? b : li > 0 ? b & ((1ull << li) - 1) : 0);
    total += __popcll(b);
  }
  if (before % BM != 0) return false;
  const int count = total - before < BM ? total - before : BM;
  if (same && mine >= before && mine < before + BM) t.rows[mine - before] = tid;
  if (tid == 0) t.count = count;
  __syncthreads();
  return true;
}

// Routed: tile `i` of the list.
template <int BM>
__device__ __forceinline__ bool read_tile(const LoraArgs& g, int i, TileRows<BM>& t) {
  if (i >= g.plan[0]) return false;
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
// One workgroup: a tile's rows, up to 64 ranks (RT blocks of 16) and one k
// range.  Direct: 16 rows, the four waves take turns at 64 values of k and
// are joined in LDS.  Routed: 64 rows, 16 for each wave.
// A lane's two 16-byte loads per step are neighbours in k (the same
// permutation of k for both operands leaves the sum as it is), so a wave's
// loads cover whole 128-byte lines.
template <bool ROUTED, int RT>
__global__ __launch_bounds__(kLoraThreads) void lora_shrink_kernel(LoraArgs g) {
  constexpr int BM = ROUTED ? kLoraTileRows : 16;
  __shared__ TileRows<BM> tile;
  __shared__ uint64_t masks[kLoraDirectRows / 64];
  const LoraProblem& p = g.p[blockIdx.z];
  const int chunks = (p.rank + 63) >> 6;
  const int split = blockIdx.y / chunks;
  const int r0 = (blockIdx.y - split * chunks) * 64;
  if (split >= p.splits) return;
  if (!(ROUTED ? read_tile(g, blockIdx.x, tile) : find_tile(g, blockIdx.x, tile, masks))) return;
  if (tile.slot < 0) return;
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int li = lane & 15;
  const int q = lane >> 4;
  const int first = ROUTED ? wave * 16 : 0;
  if (first >= tile.count) return;  // routed only: no barrier follows

  const int slot_row = first + li < tile.count ? first + li : tile.count - 1;
  const int row = tile.rows[slot_row];
  const int xrow = p.x_row_per_pair || g.top_k == 1 ? row : row / g.top_k;
  const int kbeg = split * p.k_per_split;
  const int kend = kbeg + p.k_per_split < p.k ? kbeg + p.k_per_split : p.k;
  auto xp = to_global(p.x) + (size_t)xrow * p.k + q * 16;
  gptr<uint16_t> ap[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int r = r0 + i * 16 + li < p.rank ? r0 + i * 16 + li : p.rank - 1;
    ap[i] = to_global(p.a) + ((size_t)tile.slot * p.rank + r) * p.k + q * 16;
  }
  f4 acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = f4{0, 0, 0, 0};
  constexpr int STEP = ROUTED ? 64 : 256;
#pragma unroll 2
  for (int k = kbeg + (ROUTED ? 0 : wave * 64); k < kend; k += STEP) {
    const h8 x0 = *(gptr<h8>)(xp + k), x1 = *(gptr<h8>)(xp + k + 8);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const h8 a0 = *(gptr<h8>)(ap[i] + k), a1 = *(gptr<h8>)(ap[i] + k + 8);
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, x0, acc[i], 0, 0, 0);
      acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, x1, acc[i], 0, 0, 0);
    }
  }
  if constexpr (!ROUTED) {
    __shared__ f4 part[3][RT][64];
    if (wave > 0) {
#pragma unroll
      for (int i = 0; i < RT; ++i) part[wave - 1][i][lane] = acc[i];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] += part[0][i][lane] + part[1][i][lane] + part[2][i][lane];
  }
  if (first + li >= tile.count) return;
  float* v = g.v + p.v_offset + ((size_t)split * g.rows + row) * p.rank_pad + r0 + q * 4;
#pragma unroll
  for (int i = 0; i < RT; ++i)
    if (r0 + i * 16 < p.rank) *reinterpret_cast<f4*>(v + i * 16) = acc[i];
}

// ------------------------------------------------------------------ expand
// One workgroup: a tile's rows and 64 * NT columns, 16 * NT for each wave.
// KC: 32-wide steps of the contraction over [hi | lo] (2 * rank).  CT: blocks
// of 16 rows that share a load of B.
template <bool ROUTED, int KC, int CT, int NT>
__global__ __launch_bounds__(kLoraThreads) void lora_expand_kernel(LoraArgs g) {
  constexpr int BM = ROUTED ? kLoraTileRows : 16;
  __shared__ TileRows<BM> tile;
  __shared__ uint64_t masks[kLoraDirectRows / 64];
  const LoraProblem& p = g.p[blockIdx.z];
  const int n0 = blockIdx.y * (64 * NT);
  if (n0 >= p.n) return;
  if (!(ROUTED ? read_tile(g, blockIdx.x, tile) : find_tile(g, blockIdx.x, tile, masks))) return;
  const int slot = tile.slot;
  if (slot < 0) {
    if (slot == kNone && p.base == p.y) return;
    const int cols = p.n - n0 < 64 * NT ? p.n - n0 : 64 * NT;
    for (int i = threadIdx.x; i < tile.count * cols; i += kLoraThreads) {
      const size_t at = (size_t)tile.rows[i / cols] * p.n + n0 + i % cols;
      p.y[at] = slot == kBad ? __builtin_nanf("") : p.base ? p.base[at] : 0.0f;
    }
    return;
  }
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int li = lane & 15;
  const int q = lane >> 4;
  const int blocks = p.rank >> 3;
  const float scale = g.scales ? g.scales[slot / g.experts] : 1.0f;
  const bool wide = (p.n & 3) == 0 && ((uintptr_t)p.y & 15) == 0 && ((uintptr_t)p.base & 15) == 0;
  const int c0 = n0 + wave * (16 * NT);
  if (c0 >= p.n) return;

  for (int first = 0; first < tile.count; first += 16 * CT) {
    // [hi | lo] of CT x 16 rows: lane (li, q) holds 8 values of row li
    h8 v[CT][KC];
    float back[CT];
    int rows[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      const int at = first + t * 16 + li;
      rows[t] = at < tile.count ? tile.rows[at] : -1;
      const int row = at < tile.count ? rows[t] : tile.rows[tile.count - 1];
      float f[KC][8];
      float top = 0.0f;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const int u = c * 4 + q;
        f4 s0 = f4{0, 0, 0, 0}, s1 = s0;
        if (u < 2 * blocks) {
          auto vp = to_global(g.v) + p.v_offset + (size_t)row * p.rank_pad + (u < blocks ? u : u - blocks) * 8;
          for (int s = 0; s < p.splits; ++s, vp += (size_t)g.rows * p.rank_pad) {
            s0 += *(gptr<f4>)vp;
            s1 += *(gptr<f4>)(vp + 4);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[c][j] = j < 4 ? s0[j & 3] : s1[j & 3];
          const float m = fabsf(f[c][j]);
          if (m < __builtin_inff()) top = fmaxf(top, m);  // what is not finite stays so
        }
      }
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const int ex = __builtin_amdgcn_frexp_expf(top) - 15;
      back[t] = ldexpf(1.0f, ex);
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const bool low = c * 4 + q >= blocks;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = ldexpf(f[c][j], -ex);
          const half_t hi = (half_t)x;
          const float rest = fabsf(x) < __builtin_inff() ? x - (float)hi : 0.0f;
          v[t][c][j] = low ? (half_t)rest : hi;
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int nb = c0 + nt * 16;
      if (nb >= p.n) break;
      const int bn = nb + li < p.n ? nb + li : p.n - 1;
      auto bp = to_global(p.b) + ((size_t)slot * p.n + bn) * p.rank;
      f4 acc[CT];
#pragma unroll
      for (int t = 0; t < CT; ++t) acc[t] = f4{0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const int u = c * 4 + q;
        h8 b = {0, 0, 0, 0, 0, 0, 0, 0};
        if (u < 2 * blocks) b = *(gptr<h8>)(bp + (u < blocks ? u : u - blocks) * 8);
#pragma unroll
        for (int t = 0; t < CT; ++t) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, v[t][c], acc[t], 0, 0, 0);
      }
      const int n = nb + q * 4;
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        if (rows[t] < 0 || n >= p.n) continue;
        const size_t at = (size_t)rows[t] * p.n + n;
        const f4 d = acc[t] * back[t];
        if (wide) {
          f4 o = p.base ? *(gptr<f4>)(to_global(p.base) + at) : f4{0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = fmaf(scale, d[j], o[j]);
          *reinterpret_cast<f4*>(p.y + at) = o;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n + j < p.n) p.y[at + j] = fmaf(scale, d[j], p.base ? p.base[at + j] : 0.0f);
        }
      }
    }
  }
}

// ------------------------------------------------------------------- route
// Rows sorted by slot, and tiles of up to kLoraTileRows rows of one slot, as
// two launches over chunks of the rows (one if there is one chunk): count
// the slots of each chunk, then place its rows behind those of the chunks
// before it.  Buckets slots and slots + 1 hold the rows without adapter and
// those with bad ids.
constexpr int kRouteThreads = 1024;
constexpr int kLoraBuckets = kLoraMaxSlots + 2;

__device__ __forceinline__ int lora_bucket(const LoraArgs& g, int p) {
  const int s = lora_slot(g, p);
  return s >= 0 ? s : s == kNone ? g.slots : g.slots + 1;
}

__global__ __launch_bounds__(kRouteThreads) void lora_count_kernel(LoraArgs g) {
  __shared__ int32_t h[kLoraBuckets];
  const int buckets = g.slots + 2;
  for (int i = threadIdx.x; i < buckets; i += kRouteThreads) h[i] = 0;
  __syncthreads();
  const int p0 = blockIdx.x * g.chunk;
  const int p1 = p0 + g.chunk < g.rows ? p0 + g.chunk : g.rows;
  for (int p = p0 + threadIdx.x; p < p1; p += kRouteThreads) atomicAdd(&h[lora_bucket(g, p)], 1);
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
  for (int i = tid; i < buckets; i += kRouteThreads) total[i] = cursor[i] = 0;
  __syncthreads();
  if (g.chunks == 1) {
    for (int p = tid; p < g.rows; p += kRouteThreads) atomicAdd(&total[lora_bucket(g, p)], 1);
  } else {
    const int32_t* counts = g.plan + g.plan_counts;
    for (int i = tid; i < buckets * g.chunks; i += kRouteThreads) {
      const int n = counts[i];
      if (n == 0) continue;
      const int c = i / buckets;
      const int b = i - c * buckets;
      atomicAdd(&total[b], n);
      if (c < (int)blockIdx.x) atomicAdd(&cursor[b], n);
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
    tiles += (n + kLoraTileRows - 1) / kLoraTileRows;
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
      for (int j = 0; j < n; j += kLoraTileRows)
        list[tile++] = LoraTile{slot, start + j, n - j < kLoraTileRows ? n - j : kLoraTileRows, 0};
    }
    start += n;
  }
  if (blockIdx.x == 0 && tid == kRouteThreads - 1) g.plan[0] = tile;
  __syncthreads();
  const int p0 = blockIdx.x * g.chunk;
  const int p1 = p0 + g.chunk < g.rows ? p0 + g.chunk : g.rows;
  int32_t* sorted = g.plan + kLoraPlanHeader;
  for (int p = p0 + tid; p < p1; p += kRouteThreads) sorted[atomicAdd(&cursor[lora_bucket(g, p)], 1)] = p;
}

// -------------------------------------------------------------------- host

static size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }

static long lora_tiles(int rows, int slots) {
  const long most = (long)rows / kLoraTileRows + slots + 2;  // a last tile of each bucket besides the whole ones
  return most < rows ? most : rows;
}

// Splits of k, chunks of the route and the places of everything in the
// workspace; its size.
size_t lora_layout(LoraArgs& g) {
  g.direct = g.rows <= kLoraDirectRows;
  size_t ints = 0;
  if (!g.direct) {
    const int buckets = g.slots + 2;
    g.chunks = kLoraCountWords / buckets;
    g.chunks = g.chunks < 1 ? 1 : g.chunks > 64 ? 64 : g.chunks;
    g.chunk = (g.rows + g.chunks - 1) / g.chunks;
    g.chunk = g.chunk < kLoraChunkMin ? kLoraChunkMin : g.chunk;
    if (g.rows <= kLoraOneChunk) g.chunk = g.rows;
    g.chunks = (g.rows + g.chunk - 1) / g.chunk;
    g.tiles = lora_tiles(g.rows, g.slots);
    g.plan_tiles = up(kLoraPlanHeader + (size_t)g.rows, 4);
    g.plan_counts = g.plan_tiles + 4 * (size_t)g.tiles;
    ints = g.plan_counts + (g.chunks > 1 ? (size_t)g.chunks * buckets : 0);
  }
  const size_t v0 = up(ints * 4, 256) / 4;  // in floats
  size_t at = v0;
  for (int i = 0; i < g.count; ++i) {
    LoraProblem& p = g.p[i];
    int splits;
    if (g.direct) {
      splits = (p.k + 511) / 512;
    } else {
      const long wgs = (long)(g.rows + kLoraTileRows - 1) / kLoraTileRows * ((p.rank + 63) / 64);
      splits = (int)((512 + wgs - 1) / wgs);
      if (splits > p.k / 512) splits = p.k / 512;
    }
    splits = splits < 1 ? 1 : splits > 8 ? 8 : splits;
    const int unit = g.direct ? 256 : 64;
    p.k_per_split = ((p.k + splits - 1) / splits + unit - 1) / unit * unit;
    p.splits = (p.k + p.k_per_split - 1) / p.k_per_split;
    p.rank_pad = (p.rank + 15) / 16 * 16;
    p.v_offset = at;
    at += up((size_t)p.splits * g.rows * p.rank_pad, 64);
  }
  return at * sizeof(float);
}

template <bool ROUTED>
static void launch_lora_products(const LoraArgs& g, hipStream_t st) {
  int shrink_y = 1, rank = 1, n = 1;
  for (int i = 0; i < g.count; ++i) {
    const LoraProblem& p = g.p[i];
    const int y = p.splits * ((p.rank + 63) / 64);
    shrink_y = y > shrink_y ? y : shrink_y;
    rank = p.rank > rank ? p.rank : rank;
    n = p.n > n ? p.n : n;
  }
  const unsigned tiles = (unsigned)(ROUTED ? g.tiles : g.rows);
  const dim3 block(kLoraThreads);
  const dim3 sg(tiles, shrink_y, g.count);
  if (rank <= 16) hipLaunchKernelGGL((lora_shrink_kernel<ROUTED, 1>), sg, block, 0, st, g);
  else if (rank <= 32) hipLaunchKernelGGL((lora_shrink_kernel<ROUTED, 2>), sg, block, 0, st, g);
  else hipLaunchKernelGGL((lora_shrink_kernel<ROUTED, 4>), sg, block, 0, st, g);
  constexpr int NT = ROUTED ? 4 : 1;
  const dim3 eg(tiles, (n + 64 * NT - 1) / (64 * NT), g.count);
  constexpr int C = ROUTED ? 4 : 1;
  if (rank <= 16) hipLaunchKernelGGL((lora_expand_kernel<ROUTED, 1, C, NT>), eg, block, 0, st, g);
  else if (rank <= 32) hipLaunchKernelGGL((lora_expand_kernel<ROUTED, 2, C, NT>), eg, block, 0, st, g);
  else if (rank <= 64) hipLaunchKernelGGL((lora_expand_kernel<ROUTED, 4, C, NT>), eg, block, 0, st, g);
  else if (rank <= 128) hipLaunchKernelGGL((lora_expand_kernel<ROUTED, 8, (C > 2 ? 2 : C), NT>), eg, block, 0, st, g);
  else hipLaunchKernelGGL((lora_expand_kernel<ROUTED, 16, 1, NT>), eg, block, 0, st, g);
}

hipError_t launch_lora(const LoraArgs& g, hipStream_t st) {
  if (g.direct) {
    launch_lora_products<false>(g, st);
    return hipGetLastError();
  }
  if (g.chunks > 1) hipLaunchKernelGGL(lora_count_kernel, dim3(g.chunks), dim3(kRouteThreads), 0, st, g);
  hipLaunchKernelGGL(lora_place_kernel, dim3(g.chunks), dim3(kRouteThreads), 0, st, g);
  launch_lora_products<true>(g, st);
  return hipGetLastError();
}

}  // namespace qmm
