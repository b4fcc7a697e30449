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
// choice then compares the logits themselves and is exact.  Otherwise s and c
// are formed in 64 bits, so that the choice is that of the formulas to 1e-15
// whatever the logits.  The weights are formed in 64 bits and rounded once.
#include "qmm_internal.h"

namespace qmm {

constexpr int kTopkWaves = 4;  // tokens per workgroup, one per wave

// The larger choice of two, the lower index where they are equal; index -1
// is no choice at all.
__device__ __forceinline__ bool better(double ca, int ea, double cb, int eb) {
  if (ea < 0 || eb < 0) return ea >= 0;
  return ca > cb || (ca == cb && ea < eb);
}

__device__ __forceinline__ void wave_best(double& c, int& e) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const double oc = __shfl_xor(c, d, 64);
    const int oe = __shfl_xor(e, d, 64);
    if (better(oc, oe, c, e)) {
      c = oc;
      e = oe;
    }
  }
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

// One wave per token; lane i holds experts i, i + 64, ... (V of them).
template <int V>
__global__ __launch_bounds__(kTopkWaves * 64) void moe_topk_kernel(TopkArgs a) {
  extern __shared__ double choices[];  // [kTopkWaves][e], with groups only
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const long tok = (long)blockIdx.x * kTopkWaves + wave;
  const bool live = tok < a.t;
  const float* row = a.logits + (live ? tok : 0) * a.e;
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
    if (e >= a.e) {
      c[i] = 0.0;
      continue;
    }
    alive |= 1u << i;
    c[i] = by_logit ? (double)l[i] : score(l[i]) + (a.bias ? (double)a.bias[e] : 0.0);
    bad |= c[i] != c[i];
  }

  if (a.groups > 1) {
    double* mine = choices + (size_t)wave * a.e;
    const int size = a.e / a.groups;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i * 64 + lane < a.e) mine[i * 64 + lane] = c[i];
    __syncthreads();
    double g = 0.0;
    if (lane < a.groups) {
      double first = -__builtin_inf(), second = -__builtin_inf();
      for (int j = 0; j < size; ++j) {
        const double v = mine[lane * size + j];
        if (v > first) {
          second = first;
          first = v;
        } else if (v > second) {
          second = v;
        }
      }
      g = a.group_top == 1 ? first : first + second;
      bad |= g != g;
    }
    int own = lane < a.groups ? lane : -1;
    uint64_t keep = 0;
    for (int j = 0; j < a.group_keep; ++j) {
      double gb = g;
      int gi = own;
      wave_best(gb, gi);
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
    wave_best(cb, eb);
    if (lane == j) id = eb;
    if ((eb & 63) == lane) alive &= ~(1u << (eb >> 6));
  }
  if (!live) return;

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

hipError_t launch_moe_topk(const TopkArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(((long)a.t + kTopkWaves - 1) / kTopkWaves)), block(kTopkWaves * 64);
  const size_t lds = a.groups > 1 ? (size_t)kTopkWaves * a.e * sizeof(double) : 0;
  const int v = (a.e + 63) / 64;
  if (v <= 1) hipLaunchKernelGGL(moe_topk_kernel<1>, grid, block, lds, st, a);
  else if (v <= 2) hipLaunchKernelGGL(moe_topk_kernel<2>, grid, block, lds, st, a);
  else if (v <= 4) hipLaunchKernelGGL(moe_topk_kernel<4>, grid, block, lds, st, a);
  else if (v <= 8) hipLaunchKernelGGL(moe_topk_kernel<8>, grid, block, lds, st, a);
  else hipLaunchKernelGGL(moe_topk_kernel<16>, grid, block, lds, st, a);
  return hipGetLastError();
}

}  // namespace qmm
