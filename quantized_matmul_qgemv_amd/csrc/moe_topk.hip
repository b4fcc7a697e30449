// Routing to experts: from the router's logits l [T, E] the top_k experts of
// each token and their weights, which qmm_moe_route buckets and
// qmm_moe_combine applies.
//
//   s[e] = softmax(l)[e]  or  1 / (1 + exp(-l[e]))       the score
//   c[e] = s[e] + bias[e]                                what is chosen by
//   G[g] = sum of the group_top largest c of group g; the group_keep groups
//          with the largest G stay (ties: the lower group)
//   ids  = the top_k experts of the groups that stay, by c (ties: the lower
//          expert)
//   w[j] = scale * s[ids[j]] / (renormalize ? sum_j s[ids[j]] : 1)
//
// Without a bias and with groups judged by their best expert the scores only
// enter through their order, and both scores increase with the logit: the
// choice then compares the logits themselves and is exact.  Otherwise the
// choice is that of s and c in 64 bits, whatever the logits: formed so where a
// token has a whole wave; where it has sixteen lanes formed in fp32 first, and
// again in 64 bits where fp32 cannot tell two choices apart.  The weights are
// formed in 64 bits and rounded once.
#include "qmm_internal.h"

namespace qmm {

constexpr int kTopkWaves = 4;  // tokens per workgroup where a token has a whole wave

// The larger choice of two, the lower index where they are equal; index -1
// is no choice at all.
__device__ __forceinline__ bool better(double ca, int ea, double cb, int eb) {
  if (ea < 0 || eb < 0) return ea >= 0;
  return ca > cb || (ca == cb && ea < eb);
}

// A value of another lane: permutations within the rows of 16 lanes (all
// lanes read a valid one), and the last lane of one row or two rows before.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return __builtin_amdgcn_update_dpp(v, v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp_f(float v) {
  return __builtin_bit_cast(float, dpp<CTRL, ROWS>(__builtin_bit_cast(uint32_t, v)));
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp_d(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint64_t r = (uint64_t)dpp<CTRL, ROWS>((uint32_t)(u >> 32)) << 32 | dpp<CTRL, ROWS>((uint32_t)u);
  return __builtin_bit_cast(double, r);
}
// Exchanges that join ever larger blocks of equal lanes within a row of 16,
// then (the rows that receive are 1 and 3, then 2 and 3) whole rows up to
// lane 63.
constexpr int kNeighbour = 0xB1;  // quad_perm 1 0 3 2
constexpr int kPair = 0x4E;       // quad_perm 2 3 0 1
constexpr int kQuad = 0x141;      // row_half_mirror
constexpr int kHalf = 0x140;      // row_mirror
constexpr int kRow = 0x142;       // row_bcast:15
constexpr int kTwoRows = 0x143;   // row_bcast:31

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ void join_best(double& c, int& e) {
  const double oc = dpp_d<CTRL, ROWS>(c);
  const int oe = (int)dpp<CTRL, ROWS>((uint32_t)e);
  const bool take = better(oc, oe, c, e);
  c = take ? oc : c;
  e = take ? oe : e;
}
// The index of the wave's best choice (-1 if there is none), in all lanes.
__device__ __forceinline__ int wave_best(double c, int e) {
  join_best<kNeighbour>(c, e);
  join_best<kPair>(c, e);
  join_best<kQuad>(c, e);
  join_best<kHalf>(c, e);
  join_best<kRow, 0xA>(c, e);
  join_best<kTwoRows, 0xC>(c, e);
  return __builtin_amdgcn_readlane(e, 63);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}

// ---------------------------------------------------------------- exact row
// One token by a whole wave, in 64 bits: lane i holds experts i, i + 64, ...
// (V of them), and top_k rounds of a maximum over the wave pick the experts.
// Bound by its 64-bit exponentials and the latency of its rounds: 110 us for
// 32768 x 768 (top-8 by logit), 70 us for 32768 x 160 in 5 groups.
// `choices`: e doubles of LDS of this wave's own (used with groups).
template <int V>
__device__ void exact_row(const TopkArgs& a, long tok, double* choices) {
  const int lane = threadIdx.x & 63;
  const float* row = a.logits + tok * a.e;
  const bool by_logit = a.bias == nullptr && a.group_top == 1;

  float l[V];
  float top = -__builtin_inff();
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 64 + lane;
    l[i] = e < a.e ? row[e] : -__builtin_inff();
    bad |= l[i] != l[i] || (a.score == 0 && l[i] == __builtin_inff());
    top = fmaxf(top, l[i]);
  }
  top = wave_max(top);
  double total = 0.0;  // of the softmax
  if (a.score == 0 && (!by_logit || !a.renormalize)) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (l[i] > -__builtin_inff()) total += exp((double)l[i] - (double)top);
    total = wave_sum(total);
  }
  auto score = [&](float v) -> double {
    if (a.score != 0) return 1.0 / (1.0 + exp(-(double)v));
    return v > -__builtin_inff() ? exp((double)v - (double)top) / total : 0.0;
  };
  double c[V];
  unsigned alive = 0;  // bit i: expert i * 64 + lane may be chosen
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = i * 64 + lane;
    c[i] = 0.0;
    if (e >= a.e) continue;
    alive |= 1u << i;
    c[i] = by_logit ? (double)l[i] : score(l[i]) + (a.bias ? (double)a.bias[e] : 0.0);
    bad |= c[i] != c[i];
  }

  if (a.groups > 1) {
    const int size = a.e / a.groups;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * 64 + lane < a.e) choices[i * 64 + lane] = c[i];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();  // the wave's own LDS: writes before reads
    double g = 0.0;
    if (lane < a.groups) {
      double first = -__builtin_inf(), second = -__builtin_inf();
#pragma unroll 4
      for (int j = 0; j < size; ++j) {
        const double v = choices[lane * size + j];
        second = fmax(second, fmin(first, v));
        first = fmax(first, v);
        bad |= v != v;
      }
      g = a.group_top == 1 ? first : first + second;
      bad |= g != g;
    }
    __builtin_amdgcn_wave_barrier();
    int own = lane < a.groups ? lane : -1;
    uint64_t keep = 0;
    for (int j = 0; j < a.group_keep; ++j) {
      const int gi = wave_best(g, own);
      if (gi < 0) break;  // only where a row holds a NaN
      keep |= 1ull << gi;
      if (own == gi) own = -1;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 64 + lane;
      if (e < a.e && !((keep >> (e / size)) & 1)) alive &= ~(1u << i);
    }
  }
  bad = __any(bad);

  // lane j ends with the j-th chosen expert
  int id = lane;
  for (int j = 0; j < a.top_k && !bad; ++j) {
    double cb = 0.0;
    int eb = -1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 64 + lane;
      if (((alive >> i) & 1) && better(c[i], e, cb, eb)) {
        cb = c[i];
        eb = e;
      }
    }
    eb = wave_best(cb, eb);
    if (lane == j) id = eb;
    if ((eb & 63) == lane) alive &= ~(1u << (eb >> 6));
  }

  const bool mine = lane < a.top_k;
  const float v = mine && !bad ? row[id] : -__builtin_inff();
  double w;
  if (a.renormalize) {
    // softmax scores relative to the largest chosen one: the full sum cancels
    const float ref = wave_max(v);
    const double s = !mine ? 0.0 : a.score != 0 ? 1.0 / (1.0 + exp(-(double)v))
                   : v > -__builtin_inff() ? exp((double)v - (double)ref) : 0.0;
    const double sum = wave_sum(s);
    w = sum > 0.0 ? s / sum : 0.0;
  } else {
    w = mine ? score(v) : 0.0;
  }
  if (mine) {
    a.ids[tok * a.top_k + lane] = id;
    a.weights[tok * a.top_k + lane] = bad ? __builtin_nanf("") : (float)(w * (double)a.scale);
  }
}

template <int V>
__global__ __launch_bounds__(kTopkWaves * 64) void moe_topk_wave_kernel(TopkArgs a) {
  extern __shared__ double choices[];  // [kTopkWaves][e], with groups only
  const int wave = threadIdx.x >> 6;
  const long tok = (long)blockIdx.x * kTopkWaves + wave;
  if (tok < a.t) exact_row<V>(a, tok, choices + (size_t)wave * a.e);
}

// ------------------------------------------------------------- sixteen lanes
// One token by 16 lanes, four tokens a wave; lane i holds the `per` experts
// from i * per on.
//
// A choice and its expert are packed into one double that orders like the
// choice, so that comparing is v_max_f64 / v_min_f64.  Each lane sorts its
// experts down to a list of K (K >= top_k) with bitonic networks, and four
// exchanges along the DPP row (neighbours, pairs, quads, halves) merge the
// lists: max(a[i], b[K-1-i]) are the K largest of two sorted lists, one more
// bitonic pass sorts them.
//   By logit: a double in [1, 2) whose mantissa holds 32 bits that order like
//     the logit and below them 1023 - expert: equal logits order by the
//     lower expert.
//   SCORED: the fp32 choice as a double, its place (lane, element) in the 29
//     bits that are free.  By sigmoid the fp32 choice is off by at most
//     2^-21 + 2^-23 |c| (exp2 and rcp to one unit; the rounded argument's
//     part: |l| s (1 - s) < 0.28).  By softmax all scores of a row share the
//     error of the sum (36 additions, 2^-24 each; the exponentials' errors
//     weighted by their scores, below 9 * 2^-24; rcp), in all 50 * 2^-24 of the
//     difference of two scores, which is below 0.8 * 2^-18.  Choices that
//     matter and are nearer than kNear (twice that by softmax) + 2^-21 |c|,
//     which covers both errors of a pair, are formed again in 64 bits: the
//     groups' scores before any is dropped, and after the merge all experts
//     that are no further than that below the last chosen one, one for each lane.
// Rows with a NaN, an infinity or more than 16 such experts go to exact_row.
//
// Bound by vector instructions (about 1100 for four tokens where scores are
// compared, 700 by logit), small calls by latency.  Against a whole wave
// per token in 64 bits: 1 x 128 top-8 2.7 / 9.9 us, 2048 x 128 3.9 / 12.8,
// 32768 x 256 by logit 12.9, by sigmoid and bias 16.3, in 8 groups 21 / 147
// (1.6 TB/s of logits).  Sixteen lanes, as a row's exchanges are single DPP
// moves and four tokens share every instruction.
constexpr int kRowTokens = 16;  // tokens per workgroup of 256
constexpr float kNear = 0x1p-19f;

template <typename F>
__device__ __forceinline__ float row_all(float v, F f) {
  v = f(v, dpp_f<kNeighbour>(v));
  v = f(v, dpp_f<kPair>(v));
  v = f(v, dpp_f<kQuad>(v));
  return f(v, dpp_f<kHalf>(v));
}
__device__ __forceinline__ float add_f(float x, float y) { return x + y; }
__device__ __forceinline__ float max_f(float x, float y) { return fmaxf(x, y); }
__device__ __forceinline__ float min_f(float x, float y) { return fminf(x, y); }

__device__ __forceinline__ double row_sum(double v) {
  v += dpp_d<kNeighbour>(v);
  v += dpp_d<kPair>(v);
  v += dpp_d<kQuad>(v);
  return v + dpp_d<kHalf>(v);
}
__device__ __forceinline__ double row_max(double v) {
  v = fmax(v, dpp_d<kNeighbour>(v));
  v = fmax(v, dpp_d<kPair>(v));
  v = fmax(v, dpp_d<kQuad>(v));
  return fmax(v, dpp_d<kHalf>(v));
}

// How many of the other 15 lanes of the row hold a value that comes before
// (v, tie): a larger v, or an equal one with a lower tie.
template <int R = 1>
__device__ __forceinline__ int lanes_before(double v, int tie) {
  if constexpr (R == 16) {
    return 0;
  } else {
    const double o = dpp_d<0x120 + R>(v);  // row_ror:R
    const int t = (int)dpp<0x120 + R>((uint32_t)tie);
    return (o > v || (o == v && t < tie)) + lanes_before<R + 1>(v, tie);
  }
}

// How many groups of `lanes` lanes hold a larger value.
template <int R = 1>
__device__ __forceinline__ int groups_before(float v, int lanes) {
  if constexpr (R == 16) {
    return 0;
  } else {
    int n = groups_before<R + 1>(v, lanes);
    if ((R & (lanes - 1)) == 0) n += dpp_f<0x120 + R>(v) > v;  // row_ror:R
    return n;
  }
}

// 32 bits that order like the fp32 (both zeros equal), above 1023 - index.
__device__ __forceinline__ double packed(float f, int index) {
  const uint32_t u = __builtin_bit_cast(uint32_t, f + 0.0f);
  const uint32_t order = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  const uint32_t hi = 0x3FF00000u | (order >> 12), lo = order << 20 | (uint32_t)(1023 - index);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ uint32_t low_bits(double v) { return (uint32_t)__builtin_bit_cast(uint64_t, v); }

__device__ __forceinline__ void order_pair(double& x, double& y, bool down) {
  const double hi = fmax(x, y), lo = fmin(x, y);
  x = down ? hi : lo;
  y = down ? lo : hi;
}
// A bitonic list into descending order.
template <int K>
__device__ __forceinline__ void merge_down(double (&v)[K]) {
#pragma unroll
  for (int d = K / 2; d >= 1; d /= 2)
#pragma unroll
    for (int i = 0; i < K; ++i)
      if ((i & d) == 0) order_pair(v[i], v[i + d], true);
}
template <int K>
__device__ __forceinline__ void sort_down(double (&v)[K]) {
#pragma unroll
  for (int n = 2; n <= K; n *= 2)
#pragma unroll
    for (int d = n / 2; d >= 1; d /= 2)
#pragma unroll
      for (int i = 0; i < K; ++i)
        if ((i & d) == 0) order_pair(v[i], v[i + d], (i & n) == 0 || n == K);
}
template <int CTRL, int K>
__device__ __forceinline__ void join_lists(double (&v)[K]) {
  double o[K];
#pragma unroll
  for (int i = 0; i < K; ++i) o[i] = dpp_d<CTRL>(v[K - 1 - i]);
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = fmax(v[i], o[i]);
  merge_down(v);
}

// A lane's own values of one row: by 16 bytes where every lane has `per` of
// them and the rows are aligned; `rest` beyond them.
template <int V>
__device__ __forceinline__ void load_own(float (&v)[V], const float* p, int e0, int own, int e, int per, bool wide,
                                         float rest) {
  if (wide) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      float4 f = make_float4(rest, rest, rest, rest);
      if (i < per) f = *reinterpret_cast<const float4*>(p + e0 + i);
      v[i] = f.x;
      v[i + 1] = f.y;
      v[i + 2] = f.z;
      v[i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = p[e0 + i < e ? e0 + i : e - 1];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = i < own ? v[i] : rest;
  }
}

template <int V, int K, bool SCORED>
__global__ __launch_bounds__(256) void moe_topk_row_kernel(TopkArgs a) {
  extern __shared__ double choices[];  // [4][e], for exact_row with groups
  const int li = threadIdx.x & 15;
  const int wave = threadIdx.x >> 6;
  const long tok = (long)blockIdx.x * kRowTokens + (threadIdx.x >> 4);
  const float* row = a.logits + (tok < a.t ? tok : a.t - 1) * a.e;
  const int per = (a.e + 15) >> 4;
  const int e0 = li * per;
  const int own = per < a.e - e0 ? per : a.e - e0;  // experts of this lane (none: <= 0)
  const float inf = __builtin_inff();
  constexpr float kOut = -3.402823466e38f;  // SCORED: no choice (real ones stay within 1e38)

  float l[V];
  const bool whole = (per & 3) == 0 && a.e == per * 16;
  load_own<V>(l, row, e0, own, a.e, per, whole && ((uintptr_t)a.logits & 15) == 0, -inf);

  const float near_by = a.score == 0 ? 2 * kNear : kNear;
  bool slow = false;
  float c[V];  // choices
  float top = -inf;
  if (a.score == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
    top = row_all(top, max_f);
  }
  float finite = 0.0f;  // NaN if anything is not
  if constexpr (SCORED) {
    constexpr float log2e = 1.4426950408889634f;
    if (a.score == 0) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        c[i] = __builtin_amdgcn_exp2f((l[i] - top) * log2e);  // 0 beyond the lane's own
        sum += c[i];
      }
      const float r = __builtin_amdgcn_rcpf(row_all(sum, add_f));
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] *= r;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[i] * -log2e));
    }
    if (a.bias != nullptr) {
      float b[V];
      load_own<V>(b, a.bias, e0, own, a.e, per, whole && ((uintptr_t)a.bias & 15) == 0, 0.0f);
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] += b[i];
    }
    float big = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      finite = fmaf(c[i], 0.0f, finite);
      big = fmaxf(big, fabsf(c[i]));
    }
    slow = !(big < 1e38f);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = l[i];
#pragma unroll
    for (int i = 0; i < V; i += 2) slow |= __builtin_isunordered(l[i], l[i + 1]);
    slow |= a.score == 0 && top == inf;
  }
  slow |= finite != finite;

  // The choice in 64 bits, of logit v and bias index e; the softmax's sum.
  double total = 0.0;
  auto exact_total = [&]() {
    total = 0.0;
    if (a.score == 0) {
#pragma unroll 2
      for (int i = 0; i < own; ++i) total += exp((double)row[e0 + i] - (double)top);
      total = row_sum(total);
    }
  };
  auto exact_choice = [&](float v, int e) -> double {
    const double s = a.score != 0 ? 1.0 / (1.0 + exp(-(double)v)) : exp((double)v - (double)top) / total;
    return a.bias != nullptr ? s + (double)a.bias[e] : s;
  };

  bool kept = true;  // this lane's group (the host sends only groups of whole lanes here)
  if (a.groups > 1) {
    const int lanes = 16 / a.groups;
    float first = -inf, second = -inf;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float v = i < own ? c[i] : -inf;
      second = fmaxf(second, fminf(first, v));
      first = fmaxf(first, v);
    }
    auto join = [&](float f, float s) {
      second = fmaxf(fmaxf(second, s), fminf(first, f));
      first = fmaxf(first, f);
    };
    if (lanes > 1) join(dpp_f<kNeighbour>(first), dpp_f<kNeighbour>(second));
    if (lanes > 2) join(dpp_f<kPair>(first), dpp_f<kPair>(second));
    if (lanes > 4) join(dpp_f<kQuad>(first), dpp_f<kQuad>(second));
    const float g = (a.group_top == 1 ? first : first + second) + 0.0f;
    const int most = a.group_keep * lanes;
    if constexpr (!SCORED) {
      kept = lanes_before((double)g, li / lanes) < most;
    } else {
      kept = groups_before(g, lanes) * lanes < most;  // nearly equal ones are told apart below
      // of one group: half of what a pair of choices may differ by, for each choice in it
      const float err = a.group_top == 1 ? 0.5f * near_by + 0x1p-22f * fabsf(first)
                                         : near_by + 0x1p-22f * (fabsf(first) + fabsf(second));
      const uint32_t keeping = (uint32_t)(__ballot(kept) >> (threadIdx.x & 48)) & 0xFFFF;  // too many where some are equal
      const bool near = __popc(keeping) != most ||
                        !(row_all(kept ? g - err : inf, min_f) > row_all(kept ? -inf : g + err, max_f));
      if (__any(near && !slow)) {
        exact_total();
        double f1 = -__builtin_inf(), f2 = f1;
#pragma unroll 1
        for (int i = 0; i < own; ++i) {
          const double v = exact_choice(row[e0 + i], e0 + i);
          f2 = fmax(f2, fmin(f1, v));
          f1 = fmax(f1, v);
        }
        auto join64 = [&](double f, double s) {
          f2 = fmax(fmax(f2, s), fmin(f1, f));
          f1 = fmax(f1, f);
        };
        if (lanes > 1) join64(dpp_d<kNeighbour>(f1), dpp_d<kNeighbour>(f2));
        if (lanes > 2) join64(dpp_d<kPair>(f1), dpp_d<kPair>(f2));
        if (lanes > 4) join64(dpp_d<kQuad>(f1), dpp_d<kQuad>(f2));
        kept = lanes_before(a.group_top == 1 ? f1 : f1 + f2, li / lanes) < most;
      }
    }
  }

  const int mine_n = kept ? own : 0;  // of this lane's experts, those that may be chosen
  double best[K];
#pragma unroll
  for (int base = 0; base < V; base += K) {
    double part[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int at = base + i < V ? base + i : 0;
      if constexpr (SCORED) {
        if (base + i < V) c[at] = base + i < mine_n ? c[at] : kOut;
        const double d = base + i < V ? (double)c[at] : (double)kOut;
        part[i] = __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, d) | (uint64_t)(li << 5 | at));
      } else {
        part[i] = base + i < V && base + i < mine_n ? packed(c[at], e0 + at) : 0.0;
      }
    }
    sort_down(part);
    if (base == 0) {
#pragma unroll
      for (int i = 0; i < K; ++i) best[i] = part[i];
    } else {
#pragma unroll
      for (int i = 0; i < K; ++i) best[i] = fmax(best[i], part[K - 1 - i]);
      merge_down(best);
    }
  }
  join_lists<kNeighbour>(best);
  join_lists<kPair>(best);
  join_lists<kQuad>(best);
  join_lists<kHalf>(best);

  // lane j takes the j-th of the list
  double got = best[0];
#pragma unroll
  for (int j = 1; j < K; ++j) got = li == j ? best[j] : got;
  auto expert_of = [&](double v) {
    const int low = (int)low_bits(v);
    return SCORED ? ((low >> 5) & 15) * per + (low & 31) : 1023 - (low & 1023);
  };
  int id = expert_of(got);
  if constexpr (SCORED) {
    const float v = (float)got;
    const float err = near_by + 0x1p-21f * fabsf(v);
    // the lane before holds the next larger one (row_shr:1)
    const float before = dpp_f<0x111>(v);
    bool near = li > 0 && li < a.top_k && !(before - v > err);
    const float border = row_all(li < a.top_k ? v - err : inf, min_f);
    int n = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) n += c[i] >= border;
    const int count = (int)row_all((float)n, add_f);
    near |= count != a.top_k;
    slow |= count > 16;
    if (__any(near && !slow)) {
      exact_total();
      // experts beyond the list that are near, one after the other
      double below = best[K - 1];
#pragma unroll 1
      for (int j = K; j < 16 && __any(j < count && !slow); ++j) {
        double next = -__builtin_inf();
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float v = c[i];
          asm volatile("" : "+v"(v));  // formed here: 16 doubles held over the loop would cost 32 registers
          const double d = __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, (double)v) | (uint64_t)(li << 5 | i));
          if (d < below) next = fmax(next, d);
        }
        below = row_max(next);
        if (li == j) id = expert_of(below);
      }
      const bool in = li < count;
      const bool ok = in && id < a.e;
      const double e64 = ok ? exact_choice(row[id], id) : -__builtin_inf();
      // lanes without an expert keep their place behind the others
      const int to = (threadIdx.x & 48) + (in ? lanes_before(e64, ok ? id : 1024 + li) : li);
      id = __builtin_amdgcn_ds_permute(to << 2, id);
    }
  }

  // the weights: lane j has the j-th chosen expert
  const bool mine = li < a.top_k;
  const uint64_t again = __ballot(slow);  // lanes of all four tokens
  const float v = mine ? row[id < a.e ? id : 0] : -inf;
  double w;
  if (a.renormalize) {
    const float ref = row_all(v, max_f);
    const double s = !mine ? 0.0 : a.score != 0 ? 1.0 / (1.0 + exp(-(double)v))
                   : v > -inf ? exp((double)v - (double)ref) : 0.0;
    const double sum = row_sum(s);
    w = sum > 0.0 ? s / sum : 0.0;
  } else if (a.score != 0) {
    w = 1.0 / (1.0 + exp(-(double)v));
  } else {
    exact_total();
    w = v > -inf ? exp((double)v - (double)top) / total : 0.0;
  }
  const int part = (threadIdx.x >> 4) & 3;
  if (mine && tok < a.t && !((again >> (part * 16)) & 0xFFFF)) {
    a.ids[tok * a.top_k + li] = id;
    a.weights[tok * a.top_k + li] = (float)(w * (double)a.scale);
  }
  if (again == 0) return;
  for (int i = 0; i < 4; ++i) {
    const long other = (long)blockIdx.x * kRowTokens + wave * 4 + i;
    if (((again >> (i * 16)) & 0xFFFF) && other < a.t) exact_row<(V + 3) / 4>(a, other, choices + (size_t)wave * a.e);
  }
}

static_assert((kTopkTokens + kRowTokens - 1L) / kRowTokens * 256 < 1L << 32, "the threads of a launch");

template <int V, int K>
static void launch_row(const TopkArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(((long)a.t + kRowTokens - 1) / kRowTokens)), block(256);
  const size_t lds = a.groups > 1 ? (size_t)4 * a.e * sizeof(double) : 0;
  if (a.bias != nullptr || a.group_top == 2) hipLaunchKernelGGL((moe_topk_row_kernel<V, K, true>), grid, block, lds, st, a);
  else hipLaunchKernelGGL((moe_topk_row_kernel<V, K, false>), grid, block, lds, st, a);
}

// A launch has fewer than 2^32 threads, which the last tokens of the largest
// calls would make in whole workgroups: those take a launch of their own (a
// loop over tokens in the kernel instead: 163 registers for 78).
template <int V>
static void launch_wave(const TopkArgs& a, hipStream_t st) {
  constexpr int most = 0xFFFFFFFFu / (kTopkWaves * 64) * kTopkWaves;
  const dim3 block(kTopkWaves * 64);
  const size_t lds = a.groups > 1 ? (size_t)kTopkWaves * a.e * sizeof(double) : 0;
  for (int first = 0; first < a.t; first += most) {
    TopkArgs part = a;
    part.logits += (size_t)first * a.e;
    part.ids += (size_t)first * a.top_k;
    part.weights += (size_t)first * a.top_k;
    part.t = a.t - first < most ? a.t - first : most;
    const dim3 grid((unsigned)(((long)part.t + kTopkWaves - 1) / kTopkWaves));
    hipLaunchKernelGGL(moe_topk_wave_kernel<V>, grid, block, lds, st, part);
  }
}

// Sixteen lanes a token where a lane's experts fit its registers, the list of
// chosen ones its 16 lanes, and groups are made of whole lanes.
hipError_t launch_moe_topk(const TopkArgs& a, hipStream_t st) {
  const bool rows = a.e <= 512 && a.top_k <= 16 && (a.groups == 1 || (a.e % 16 == 0 && 16 % a.groups == 0));
  if (rows) {
    const int per = (a.e + 15) / 16;
    if (a.top_k <= 8) {
      if (per <= 4) launch_row<4, 8>(a, st);
      else if (per <= 8) launch_row<8, 8>(a, st);
      else if (per <= 16) launch_row<16, 8>(a, st);
      else launch_row<32, 8>(a, st);
    } else {
      if (per <= 4) launch_row<4, 16>(a, st);
      else if (per <= 8) launch_row<8, 16>(a, st);
      else if (per <= 16) launch_row<16, 16>(a, st);
      else launch_row<32, 16>(a, st);
    }
  } else {
    const int v = (a.e + 63) / 64;
    if (v <= 2) launch_wave<2>(a, st);
    else if (v <= 4) launch_wave<4>(a, st);
    else if (v <= 8) launch_wave<8>(a, st);
    else launch_wave<16>(a, st);
  }
  return hipGetLastError();
}

}  // namespace qmm
