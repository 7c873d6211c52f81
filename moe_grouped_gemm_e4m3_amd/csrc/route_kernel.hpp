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
// still small (a token's scores are read once).  A few tokens are bound by latency:
// two loads, an exponential in 64 bits, the groups and k rounds of finding the
// largest (8 of 256 experts in 8 groups: 5.6 us for one token, of which a launch is
// about 2).  Thousands are bound by the vector instructions of a token's wave (the
// same, 4096 tokens: 9.6 us; 940 of them, 59% of the SIMDs' cycles at four each and
// more for those on 64 bits).  Without bias and groups the logits decide, and a sum that the division
// by the chosen scores' sum cancels is not computed (8192 x 128, not normalised,
// forward and backward: 14 us).
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

// Reductions over the wave's lanes by data-parallel moves: lanes of a row, then
// rows, into lane 63 (an exchange through LDS costs five times as much).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t lane_move(uint32_t v, uint32_t none) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double lane_move(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = lane_move<CTRL, ROWS>((uint32_t)b, 0u), hi = lane_move<CTRL, ROWS>((uint32_t)(b >> 32), 0u);
  return __builtin_bit_cast(double, lo | hi << 32);
}
__device__ __forceinline__ uint32_t from_lane(uint32_t v, int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); }
__device__ __forceinline__ double from_lane(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t lo = from_lane((uint32_t)b, lane), hi = from_lane((uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, lo | hi << 32);
}
__device__ __forceinline__ double wave_sum(double v) {
  v += lane_move<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8
  v += lane_move<0x112, 0xf>(v);
  v += lane_move<0x114, 0xf>(v);
  v += lane_move<0x118, 0xf>(v);
  v += lane_move<0x142, 0xa>(v);  // the last lane of rows 0 and 2 to the next row
  v += lane_move<0x143, 0xc>(v);  // lane 31 to rows 2 and 3
  return from_lane(v, 63);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, lane_move<0x111, 0xf>(v, 0u));
  v = max(v, lane_move<0x112, 0xf>(v, 0u));
  v = max(v, lane_move<0x114, 0xf>(v, 0u));
  v = max(v, lane_move<0x118, 0xf>(v, 0u));
  v = max(v, lane_move<0x142, 0xa>(v, 0u));
  v = max(v, lane_move<0x143, 0xc>(v, 0u));
  return from_lane(v, 63);
}

// The value of lane ^ D's group of D lanes, in which all lanes hold the same.
template <int D>
__device__ __forceinline__ double other_group(double v) {
  if (D == 1) return lane_move<0xb1, 0xf>(v);   // quad_perm 1 0 3 2
  if (D == 2) return lane_move<0x4e, 0xf>(v);   // quad_perm 2 3 0 1
  if (D == 4) return lane_move<0x141, 0xf>(v);  // mirrored halves of a row
  if (D == 8) return lane_move<0x140, 0xf>(v);  // mirrored row
  return __shfl_xor(v, D);
}

// Integers that order as the numbers do, above 0; a NaN stands in the place of
// -infinity, below all numbers.  -0 + 0 is +0: both zeros are one number.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return v != v ? 0x007fffffu : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_of(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return b >> 63 ? ~b : b | (uint64_t)1 << 63;
}
__device__ __forceinline__ float wave_max_logit(float v) {
  const uint32_t b = wave_max(order_of(v));
  return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}
__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

// The largest and second largest of two such pairs.
__device__ __forceinline__ void merge_two(double& a, double& b, double c, double d) {
  const double low = a < c ? a : c;
  a = a < c ? c : a;
  b = b < d ? d : b;
  b = b < low ? low : b;
}

template <int D>
__device__ __forceinline__ void merge_groups(double& a, double& b) {
  const double c = other_group<D>(a), d = other_group<D>(b);
  merge_two(a, b, c, d);
}

// SLOTS: experts of a lane.  SCORED: a bias or groups, so that scores decide
// (in 64 bits); else the logits do.
template <typename L, int SLOTS, bool SCORED>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteParams p) {
  __shared__ double by_expert[SCORED ? kRouteWaves : 1][SCORED ? 64 * SLOTS : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
  const double none = -__builtin_inf();
  if (t >= p.T) return;
  const L* row = (const L*)p.logits + t * p.ld;
  float l[SLOTS], bias[SLOTS];
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    const int e = lane + 64 * s;
    l[s] = e < p.E ? to_f32(row[e]) : -__builtin_inff();
    bias[s] = SCORED && p.bias && e < p.E ? p.bias[e] : 0.f;
  }
  // softmax: the largest logit and the sum over all experts, which cancels where
  // the chosen scores are divided by their sum (but for a NaN)
  float top = 0.f;
  double scale = 1.0;
  if (!p.sigmoid) {
    top = l[0];
    bool nan = l[0] != l[0];
#pragma unroll
    for (int s = 1; s < SLOTS; ++s) {
      top = fmaxf(top, l[s]);
      nan |= l[s] != l[s];
    }
    top = wave_max_logit(top);
    if (top == -__builtin_inff()) top = 0.f;
    if (__any(nan)) {
      scale = __builtin_nan("");
    } else if (SCORED || !p.normalize) {
      double sum = 0.0;
#pragma unroll
      for (int s = 0; s < SLOTS; ++s)
        if (lane + 64 * s < p.E) sum += exp((double)l[s] - (double)top);
      sum = wave_sum(sum);
      scale = sum == 0.0 ? 0.0 : 1.0 / sum;
    }
  }
  auto score = [&](float x) { return p.sigmoid ? sigmoid64(x) : exp((double)x - (double)top) * scale; };
  // what experts are compared by: 32 bits, and where these are equal 32 more;
  // 0: no candidate (every candidate's upper bits are above 0)
  uint32_t key[SLOTS], low[SCORED ? SLOTS : 1];
  double sc[SCORED ? SLOTS : 1];
  if constexpr (SCORED) {
    double by[SLOTS];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      sc[s] = 0.0;
      by[s] = none;
      if (l[s] != -__builtin_inff()) {
        sc[s] = score(l[s]);
        by[s] = p.bias ? sc[s] + bias[s] : sc[s];
      }
      if (by[s] != by[s]) by[s] = kLast;
    }
    if (p.groups > 1) {
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
      if (per > 1) merge_groups<1>(a, b);
      if (per > 2) merge_groups<2>(a, b);
      if (per > 4) merge_groups<4>(a, b);
      if (per > 8) merge_groups<8>(a, b);
      if (per > 16) merge_groups<16>(a, b);
      if (per > 32) merge_groups<32>(a, b);
      const double total = a == none ? none : a + (b == none ? 0.0 : b);
      int rank = 0;
      for (int o = 0; o < p.groups; ++o) {
        const double other = from_lane(total, o * per);
        rank += other > total || (other == total && o < g);
      }
      const unsigned long long kept = __ballot(g < p.groups && rank < p.top);
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        const int e = lane + 64 * s;
        if (e < p.E && !((kept >> (e / size * per)) & 1)) by[s] = none;
      }
    }
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const uint64_t o = by[s] == none ? 0 : order_of(by[s]);
      key[s] = (uint32_t)(o >> 32);
      low[s] = (uint32_t)o;
      by_expert[wave][lane + 64 * s] = sc[s];
    }
    __builtin_amdgcn_wave_barrier();
  } else {
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) key[s] = l[s] == -__builtin_inff() ? 0 : order_of(l[s]);
  }
  // k rounds of finding the largest; equal ones go to the lowest expert
  int chosen = -1;
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int s = 1; s < SLOTS; ++s) best = max(best, key[s]);
    best = wave_max(best);
    if (best == 0) break;  // no candidate is left
    // the lanes and slots that hold it: usually one
    unsigned long long held[SLOTS];
    int count = 0;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      held[s] = __ballot(key[s] == best);
      count += __builtin_popcountll(held[s]);
    }
    if (SCORED && count > 1) {
      uint32_t lo = 0;
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) lo = key[s] == best ? max(lo, low[s]) : lo;
      lo = wave_max(lo);
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) held[s] = __ballot(key[s] == best && low[s] == lo);
    }
    int e = 0;
#pragma unroll
    for (int s = SLOTS - 1; s >= 0; --s)
      if (held[s]) e = 64 * s + __builtin_ctzll(held[s]);
    if (lane == j) chosen = e;
    const int mine = e - lane;  // 64 s for the lane and slot that hold it
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) key[s] = mine == 64 * s ? 0 : key[s];
  }
  double share = 0.0;
  if (chosen >= 0) {
    if constexpr (SCORED)
      share = by_expert[wave][chosen];
    else
      share = score(to_f32(row[chosen]));
  }
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

// Every logit's gradient is written once; what the chosen experts get on top is
// added in the order of their places.  Bound by latency for a few tokens, by vector
// instructions for many (8192 x 128: 430 a token, 66% of the SIMDs' cycles).
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
  // softmax: the largest logit and the sum over all experts; normalised, the sum
  // cancels (but for a NaN, which a NaN or +infinity among the logits makes of all scores)
  double e[SLOTS];
  float top = 0.f;
  double scale = 1.0;
  const bool dense = !p.sigmoid && !p.normalize;
  if (!p.sigmoid) {
    float l[SLOTS];
    bool nan = false;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      l[s] = lane + 64 * s < p.E ? to_f32(row[lane + 64 * s]) : -__builtin_inff();
      top = s == 0 ? l[0] : fmaxf(top, l[s]);
      nan |= !(l[s] < __builtin_inff());
    }
    top = wave_max_logit(top);
    if (top == -__builtin_inff()) top = 0.f;
    if (__any(nan)) scale = __builtin_nan("");
    if (dense) {
      double sum = 0.0;
#pragma unroll
      for (int s = 0; s < SLOTS; ++s) {
        e[s] = lane + 64 * s < p.E ? exp((double)l[s] - (double)top) : 0.0;
        sum += e[s];
      }
      sum = wave_sum(sum);
      scale = sum == 0.0 ? 0.0 : 1.0 / sum;
    }
  }
  // sigmoid: 1 - s_j without the difference, which cancels (from a logit of 37 on to 0)
  double s_j = 0.0, rest = 1.0;
  if (there) {
    const double u = exp(p.sigmoid ? -(double)x : (double)x - (double)top);
    s_j = p.sigmoid ? 1.0 / (1.0 + u) : u * scale;
    rest = x > 0.f ? u * s_j : 1.0 - s_j;
  }
  double q = s_j;
  if (p.normalize) {
    const double all = wave_sum(s_j);
    q = all == 0.0 ? 0.0 : s_j / all;
  }
  const double mean = p.sigmoid && !p.normalize ? 0.0 : wave_sum(g * q);
  // what place j sends to its expert; dense: the part - s_i mean reaches every expert
  double d = dense ? g * q : q * (g - mean);
  if (p.sigmoid) d *= rest;
  L* out = (L*)p.dl + t * p.ld_dl;
  double dl[SLOTS];
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) dl[s] = dense ? -(e[s] * scale) * mean : p.sigmoid ? 0.0 : 0.0 * scale;
  for (int j = 0; j < p.k; ++j) {
    const int to = (int)from_lane((uint32_t)id, j) - lane;
    const double v = from_lane(d, j);
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
      if (to == 64 * s) dl[s] += v;
  }
#pragma unroll
  for (int s = 0; s < SLOTS; ++s)
    if (lane + 64 * s < p.E) store_as(out + lane + 64 * s, dl[s]);
}

}  // namespace fg
