// route_kernel.hpp -- the expert router and its gradient.
//
//   s = softmax(l) or 1 / (1 + exp(-l));  the k experts with the largest s + b
//   w_j = c s_j, or c s_j / sum of the chosen s
//
// and, with g_j = c dw_j and q_j = s_j / sum (normalised) or s_j,
//   softmax, normalised   dl_j = q_j (g_j - sum g q)
//   sigmoid, normalised   dl_j = q_j (g_j - sum g q) (1 - s_j)
//   softmax               dl_i = s_i (g_i - sum g s) over all i (g_i = 0 where i is not chosen)
//   sigmoid               dl_j = g_j s_j (1 - s_j)
//
// A wave takes a token, a lane the experts lane, lane + 64, ...  Scores, what
// decides between experts, and sums are in 64 bits: the choice is then that of
// the formula wherever two experts differ by more than 1e-15, and the work is
// still small (a token's scores are read once; the kernels are bound by the
// latency of k rounds of finding the largest).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear_kernel.hpp"

namespace fg {

constexpr int kRouteWaves = 4;
constexpr int kMaxRouteExperts = 1024, kMaxRouteChoices = 64, kMaxRouteGroups = 64;

struct RouteParams {
  const void* logits;
  int64_t ld;  // elements
  const float* bias;
  int32_t* ids;
  float* w;
  int T, E, k, groups, top;
  bool sigmoid, normalize;
  float scale;
};

// In the place of a NaN where experts are compared: below every score, above "no candidate".
constexpr double kLast = -1e300;

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

// The largest and second largest of two such pairs.
__device__ __forceinline__ void merge_two(double& a, double& b, double c, double d) {
  const double low = a < c ? a : c;
  a = a < c ? c : a;
  b = b < d ? d : b;
  b = b < low ? low : b;
}

// SLOTS: experts of a lane.  SCORED: a bias or groups, so that scores decide; else the logits do.
template <typename L, int SLOTS, bool SCORED>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteParams p) {
  __shared__ double by_expert[SCORED ? kRouteWaves : 1][SCORED ? 64 * SLOTS : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  const double none = -__builtin_inf();
  if (t >= p.T) return;
  const L* row = (const L*)p.logits + t * p.ld;
  float l[SLOTS];
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    const int e = lane + 64 * s;
    l[s] = e < p.E ? to_f32(row[e]) : -__builtin_inff();
  }
  // softmax: the largest logit and the sum over all experts
  float top = 0.f;
  double sum = 1.0;
  if (!p.sigmoid) {
    top = l[0];
#pragma unroll
    for (int s = 1; s < SLOTS; ++s) top = fmaxf(top, l[s]);
    top = wave_max(top);
    if (top == -__builtin_inff()) top = 0.f;
    sum = 0.0;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
      if (lane + 64 * s < p.E) sum += exp((double)l[s] - (double)top);
    sum = wave_sum(sum);
  }
  auto score = [&](float x) {
    return p.sigmoid ? sigmoid64(x) : sum == 0.0 ? 0.0 : exp((double)x - (double)top) / sum;
  };
  double by[SLOTS];
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    const int e = lane + 64 * s;
    double v = l[s];
    if (SCORED && l[s] != -__builtin_inff()) {
      v = score(l[s]);
      if (p.bias) v += p.bias[e];
    }
    by[s] = v != v ? kLast : v;
  }
  if (SCORED && p.groups > 1) {
    // groups' sums of their two best: each group has a power of two of lanes
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) by_expert[wave][lane + 64 * s] = by[s];
    __builtin_amdgcn_wave_barrier();
    int per = 64;
    while (per * p.groups > 64) per >>= 1;
    const int size = p.E / p.groups, g = lane / per, l0 = lane - g * per;
    double a = none, b = none;
    if (g < p.groups)
      for (int i = l0; i < size; i += per) merge_two(a, b, by_expert[wave][g * size + i], none);
    for (int d = 1; d < per; d *= 2) {
      const double c = __shfl_xor(a, d), e = __shfl_xor(b, d);
      merge_two(a, b, c, e);
    }
    const double total = a == none ? none : a + (b == none ? 0.0 : b);
    int rank = 0;
    for (int o = 0; o < p.groups; ++o) {
      const double other = __shfl(total, o * per);
      rank += other > total || (other == total && o < g);
    }
    const unsigned long long kept = __ballot(g < p.groups && rank < p.top);
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int e = lane + 64 * s;
      if (e < p.E && !((kept >> (e / size * per)) & 1)) by[s] = none;
    }
  }
  // k rounds of finding the largest; equal ones go to the lowest expert
  int chosen = -1;
  float logit = 0.f;
  for (int j = 0; j < p.k; ++j) {
    double best = by[0];
    int at = lane;
    float x = l[0];
#pragma unroll
    for (int s = 1; s < SLOTS; ++s)
      if (by[s] > best) {
        best = by[s];
        at = lane + 64 * s;
        x = l[s];
      }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const double v = __shfl_xor(best, d);
      const int o = __shfl_xor(at, d);
      const bool take = v > best || (v == best && o < at);
      best = take ? v : best;
      at = take ? o : at;
    }
    if (best == none) break;  // no candidate is left
    const float won = __shfl(x, at & 63);
    if (lane == j) {
      chosen = at;
      logit = won;
    }
    if (lane == (at & 63)) {
#pragma unroll
      for (int s = 0; s < SLOTS; ++s)
        if (s == at >> 6) by[s] = none;
    }
  }
  double share = chosen >= 0 ? score(logit) : 0.0;
  if (p.normalize) {
    const double all = wave_sum(share);
    share = all == 0.0 ? 0.0 : share / all;
  }
  if (lane < p.k) {
    p.ids[t * p.k + lane] = chosen;
    p.w[t * p.k + lane] = chosen < 0 ? 0.f : (float)(p.scale * share);
  }
}

struct RouteGradParams {
  const float* dw;
  const void* logits;
  int64_t ld;
  const int32_t* ids;
  void* dl;
  int64_t ld_dl;
  int T, E, k;
  bool sigmoid, normalize;
  float scale;
};

__device__ __forceinline__ void store_as(float* p, double v) { *p = (float)v; }
__device__ __forceinline__ void store_as(uint16_t* p, double v) { *p = bf16_bits((float)v); }

template <typename L, int SLOTS>
__global__ __launch_bounds__(64 * kRouteWaves) void route_backward_kernel(RouteGradParams p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (t >= p.T) return;
  const L* row = (const L*)p.logits + t * p.ld;
  const int id = lane < p.k ? p.ids[t * p.k + lane] : -1;
  const bool there = (unsigned)id < (unsigned)p.E;
  const double g = there ? (double)p.dw[t * p.k + lane] * p.scale : 0.0;
  const float x = there ? to_f32(row[id]) : 0.f;
  float l[SLOTS];
  float top = 0.f;
  double sum = 1.0;
  const bool dense = !p.sigmoid && !p.normalize;
  if (!p.sigmoid) {
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int e = lane + 64 * s;
      l[s] = e < p.E ? to_f32(row[e]) : -__builtin_inff();
      top = s == 0 ? l[0] : fmaxf(top, l[s]);
    }
    top = wave_max(top);
    if (top == -__builtin_inff()) top = 0.f;
    sum = 0.0;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
      if (lane + 64 * s < p.E) sum += exp((double)l[s] - (double)top);
    sum = wave_sum(sum);
  }
  auto score = [&](float v) {
    return p.sigmoid ? sigmoid64(v) : sum == 0.0 ? 0.0 : exp((double)v - (double)top) / sum;
  };
  const double s_j = there ? score(x) : 0.0;
  double q = s_j;
  if (p.normalize) {
    const double all = wave_sum(s_j);
    q = all == 0.0 ? 0.0 : s_j / all;
  }
  const double mean = p.sigmoid && !p.normalize ? 0.0 : wave_sum(g * q);
  // what place j sends to its expert; dense: the part - s_i mean reaches every expert
  double d = dense ? g * q : q * (g - mean);
  if (p.sigmoid) d *= 1.0 - s_j;
  L* out = (L*)p.dl + t * p.ld_dl;
  double dl[SLOTS];
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) dl[s] = dense && lane + 64 * s < p.E ? -score(l[s]) * mean : 0.0;
  for (int j = 0; j < p.k; ++j) {
    const int e = __shfl(id, j);
    const double v = __shfl(d, j);
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
      if (e == lane + 64 * s) dl[s] += v;
  }
#pragma unroll
  for (int s = 0; s < SLOTS; ++s)
    if (lane + 64 * s < p.E) store_as(out + lane + 64 * s, dl[s]);
}

}  // namespace fg
