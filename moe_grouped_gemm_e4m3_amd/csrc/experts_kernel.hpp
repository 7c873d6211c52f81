// experts_kernel.hpp -- a whole expert layer for a few tokens, in two kernels.
//
//   up    g = W1[e][0:F] x_t, u = W1[e][F:2F] x_t, h = act(g) u      for every pair (t, j) with e = ids[t, j]
//   down  D[t] = bf16( sum_j w[t, j] W2[e] h_(t, j) )
//
// Every active expert's weights are read once for each 64 tokens
// (weight_stream.hpp); that read is the time.  `up` has a workgroup for each
// expert and 16 hidden units; its tokens are the rows of the matrix product.
// `down` has a workgroup for each 16 or 32 outputs, which goes through all active
// experts, so that the sum over experts never leaves it: its waves share out the
// chunks of all experts' hidden units, evenly, each adds into sums of its own
// (one for each token and output, in LDS), and these are added in wave order.
// No sum depends on the order in which workgroups run.
//
// h passes through the workspace as the sum of two bf16 (16 significant bits):
// as one its rounding would add as much error as the output's own, and both
// products of a weight tile cost less than the tile's load.
//
// A token that names an expert twice has one product with the sum of both
// weights, at the first of the two places.
#pragma once

#include "weight_stream.hpp"

namespace fg {

constexpr int kLayerTokens = 64;    // tokens a pass over the weights serves: a lane each
constexpr int kMaxExperts = 1024;   // `down` keeps a set of tokens for each in LDS
constexpr int kMaxChoices = 32;

struct ExpertParams {
  const uint16_t* X;
  int64_t ldx;  // elements
  const uint8_t *W1, *W2;
  const void *s1, *s2;      // e4m3: fp32 factors of blocks; 4-bit: bf16 scales of groups
  const uint8_t *z1, *z2;   // 4-bit: zero points or NULL
  const int32_t* ids;
  const float* w;
  uint16_t* D;
  int64_t ldd;
  uint16_t* H;  // [T k][2][F]: both parts of every pair's h
  int T, k, E, F, K, act;
  int group;
  int row1, row2;        // bytes of a weight row
  int groups1, groups2;  // scale groups (e4m3: block columns) of a row
  bool wide1, wide2;
  bool by_pair;  // up: blockIdx.y is a pair (fewer pairs than experts), else an expert
};

// Rows [row0, row0 + 16 PER) of rows x cols weights of expert e in region r of src.
template <class S>
__device__ __forceinline__ void set_weights(Sources<S>& src, int r, const uint8_t* W, const void* s, const uint8_t* z,
                                            int e, int rows, int row0, int row_bytes, int groups) {
  const int l16 = threadIdx.x & 15;
  const int64_t at = (int64_t)e * rows + row0;
  src.q[r] = make_rsrc(W + at * row_bytes, (int64_t)(rows - row0) * row_bytes);
  src.q_off = l16 * row_bytes;
  src.q_tile = 16 * row_bytes;
  if constexpr (S::FP8) {
    src.fs[r] = (const float*)s + ((int64_t)e * ((rows + 127) >> 7) + (row0 >> 7)) * groups;
  } else {
    src.s[r] = make_rsrc((const uint16_t*)s + at * groups, (int64_t)(rows - row0) * groups * 2);
    src.z[r] = make_rsrc(z ? z + at * groups : nullptr, z ? (int64_t)(rows - row0) * groups : 0);
    src.has_z = z != nullptr;
    src.s_off = l16 * groups * 2; src.s_tile = 32 * groups;
    src.z_off = l16 * groups; src.z_tile = 16 * groups;
  }
}

template <class S>
__device__ __forceinline__ void clear(f32x4 (&acc)[S::MT][S::CF]) {
#pragma unroll
  for (int t = 0; t < S::MT; ++t)
#pragma unroll
    for (int c = 0; c < S::CF; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};
}

constexpr int kUpWaves = 4;

// One tile of 16 MT member tokens, from member `base` on, and 16 hidden units.
template <int FMT, int GPC, int MT, int DEPTH>
__device__ __forceinline__ void up_tile(const ExpertParams& p, int e, int t0, int f0, int base, int members,
                                        const int* list, f32x4 (*red)[4][64]) {
  using S = Stream<FMT, GPC, MT, 2, 2, 1, DEPTH>;
  const int lane = threadIdx.x & 63, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Sources<S> src;
  src.K = p.K;
  src.group = p.group;
  src.wide = p.wide1;
  set_weights(src, 0, p.W1, p.s1, p.z1, e, 2 * p.F, f0, p.row1, p.groups1);
  set_weights(src, 1, p.W1, p.s1, p.z1, e, 2 * p.F, p.F + f0, p.row1, p.groups1);
  const int T = min(kLayerTokens, p.T - t0);
  src.x = make_rsrc(p.X + (int64_t)t0 * p.ldx, ((int64_t)(T - 1) * p.ldx + p.K) * 2);
#pragma unroll
  for (int t = 0; t < MT; ++t) src.x_off[t] = (list[min(base + 16 * t + l16, members - 1)] & 63) * (int)(2 * p.ldx);
  src.x_part = 0;

  f32x4 acc[MT][2];
  clear<S>(acc);
  stream_chunks<S>(acc, src, wave, (p.K + 127) >> 7, kUpWaves);
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    red[wave][2 * t][lane] = acc[t][0];
    red[wave][2 * t + 1][lane] = acc[t][1];
  }
  __syncthreads();
#pragma unroll
  for (int x = threadIdx.x; x < MT * 256; x += 64 * kUpWaves) {
    const int col = x & 15, row = (x >> 4) & 15, t = x >> 8;
    const int at = (row >> 2) * 16 + col, i = row & 3;
    float g = red[0][2 * t][at][i], u = red[0][2 * t + 1][at][i];
#pragma unroll
    for (int w = 1; w < kUpWaves; ++w) {
      g += red[w][2 * t][at][i];
      u += red[w][2 * t + 1][at][i];
    }
    const int m = base + 16 * t + row;
    if (m < members) {
      const int pair = list[m];
      const float h = p.act == kActSilu ? gated_value<kActSilu>(g, u) : gated_value<kActGeluTanh>(g, u);
      const uint16_t top = bf16_bits(h);
      // the rest of an infinity or a NaN would be a NaN
      const float rest = (top & 0x7f80) == 0x7f80 ? 0.f : h - to_f32(top);
      uint16_t* dst = p.H + ((int64_t)(t0 + (pair & 63)) * p.k + (pair >> 6)) * 2 * p.F + f0 + col;
      dst[0] = top;
      dst[p.F] = bf16_bits(rest);
    }
  }
}

// Grid: tiles of 16 hidden units, pairs or experts, passes of 64 tokens.
template <int FMT, int GPC>
__global__ __launch_bounds__(64 * kUpWaves) void experts_up_kernel(ExpertParams p) {
  __shared__ f32x4 red[kUpWaves][4][64];
  __shared__ int list[kLayerTokens];
  const int lane = threadIdx.x & 63;
  const int t0 = blockIdx.z * kLayerTokens, T = min(kLayerTokens, p.T - t0);
  const int32_t* ids = p.ids + (int64_t)t0 * p.k;
  int e = blockIdx.y;
  if (p.by_pair) {
    if ((int)blockIdx.y >= T * p.k) return;
    e = load_invariant(ids + blockIdx.y);
    if ((unsigned)e >= (unsigned)p.E) return;
  }
  // the first of this lane's token's places that name e
  int place = -1;
  if (lane < T)
    for (int j = p.k - 1; j >= 0; --j)
      if (ids[lane * p.k + j] == e) place = j;
  const unsigned long long mask = __ballot(place >= 0);
  if (mask == 0) return;
  if (p.by_pair) {
    // the first pair of an expert stands for all of them
    const int first = __builtin_ctzll(mask);
    if (first * p.k + __builtin_amdgcn_readlane(place, first) != (int)blockIdx.y) return;
  }
  const int members = __builtin_popcountll(mask);
  if (threadIdx.x < 64 && place >= 0) list[__builtin_popcountll(mask & ((1ull << lane) - 1))] = lane | place << 6;
  __syncthreads();
  const int f0 = blockIdx.x * 16;
  for (int base = 0; base < members; base += 32) {
    if (base) __syncthreads();  // red is read
    if (members - base <= 16)
      up_tile<FMT, GPC, 1, 2>(p, e, t0, f0, base, members, list, red);
    else
      up_tile<FMT, GPC, 2, 2>(p, e, t0, f0, base, members, list, red);
  }
}

template <int FMT_, int GPC_, int MT_, int CF_, int WAVES_, int DEPTH_>
struct DownTile {
  using S = Stream<FMT_, GPC_, MT_, CF_, 1, 2, DEPTH_>;
  static constexpr int WAVES = WAVES_, THREADS = 64 * WAVES, COLS = 16 * CF_, ROWS = 16 * MT_;
  static int lds_bytes(int T) { return WAVES * (T < kLayerTokens ? T : kLayerTokens) * COLS * 4; }
};

// Grid: tiles of COLS outputs, passes of 64 tokens.
template <class C>
__global__ __launch_bounds__(C::THREADS) void experts_down_kernel(ExpertParams p) {
  using S = typename C::S;
  extern __shared__ float sums[];  // [WAVES][T][COLS]
  __shared__ unsigned long long tokens[kMaxExperts];  // that go to an expert
  // experts with their tiles of ROWS tokens, and how many
  __shared__ uint16_t items[kMaxExperts * (kLayerTokens / C::ROWS)];
  __shared__ int item_count;
  __shared__ int pair_of[C::WAVES][C::ROWS], token_of[C::WAVES][C::ROWS];
  __shared__ float weight_of[C::WAVES][C::ROWS];
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, quarter = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t0 = blockIdx.y * kLayerTokens, T = min(kLayerTokens, p.T - t0);
  const int32_t* ids = p.ids + (int64_t)t0 * p.k;
  const float* weights = p.w + (int64_t)t0 * p.k;
  const int n0 = blockIdx.x * C::COLS;

  for (int i = tid; i < p.E; i += C::THREADS) tokens[i] = 0;
  for (int i = tid; i < C::WAVES * T * C::COLS; i += C::THREADS) sums[i] = 0.f;
  __syncthreads();
  for (int i = tid; i < T * p.k; i += C::THREADS) {
    const int e = ids[i];
    if ((unsigned)e < (unsigned)p.E) atomicOr(&tokens[e], 1ull << (i / p.k));
  }
  __syncthreads();
  if (wave == 0) {
    int n = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      const int e = e0 + lane;
      const int members = e < p.E ? __builtin_popcountll(tokens[e]) : 0;
#pragma unroll
      for (int sub = 0; sub < kLayerTokens / C::ROWS; ++sub) {
        const unsigned long long any = __ballot(members > sub * C::ROWS);
        if (members > sub * C::ROWS) items[n + __builtin_popcountll(any & ((1ull << lane) - 1))] = (uint16_t)(e | sub << 10);
        n += __builtin_popcountll(any);
      }
    }
    if (lane == 0) item_count = n;
  }
  __syncthreads();

  const int chunks = (p.F + 127) >> 7;
  const int total = item_count * chunks;
  int at = (int)((int64_t)total * wave / C::WAVES);
  const int end = (int)((int64_t)total * (wave + 1) / C::WAVES);
  float* mine = sums + wave * T * C::COLS;
  Sources<S> src;
  src.K = p.F;
  src.group = p.group;
  src.wide = p.wide2;
  src.x = make_rsrc(p.H + (int64_t)t0 * p.k * 2 * p.F, (int64_t)T * p.k * 4 * p.F);
  src.x_part = 2 * p.F;
  while (at < end) {
    const int item = __builtin_amdgcn_readfirstlane(at / chunks), c0 = at - item * chunks;
    const int c1 = min(chunks, c0 + end - at);
    at += c1 - c0;
    const int what = __builtin_amdgcn_readfirstlane(items[item]);
    const int e = what & 1023, base = (what >> 10) * C::ROWS;
    const unsigned long long mask = tokens[e];
    const int rows = min(C::ROWS, __builtin_popcountll(mask) - base);
    const int rank = __builtin_popcountll(mask & ((1ull << lane) - 1)) - base;
    if (((mask >> lane) & 1) && rank >= 0 && rank < C::ROWS) {
      int place = -1;
      float w = 0.f;
      for (int j = 0; j < p.k; ++j)
        if (ids[lane * p.k + j] == e) {
          w = place < 0 ? weights[lane * p.k + j] : w + weights[lane * p.k + j];
          if (place < 0) place = j;
        }
      pair_of[wave][rank] = lane * p.k + place;
      token_of[wave][rank] = lane;
      weight_of[wave][rank] = w;
    }
    // a wave's own LDS accesses are in order; the compiler keeps them so
    __builtin_amdgcn_wave_barrier();
    set_weights(src, 0, p.W2, p.s2, p.z2, e, p.K, n0, p.row2, p.groups2);
#pragma unroll
    for (int t = 0; t < S::MT; ++t) src.x_off[t] = pair_of[wave][min(16 * t + l16, rows - 1)] * 4 * p.F;
    f32x4 acc[S::MT][S::CF];
    clear<S>(acc);
    stream_chunks<S>(acc, src, c0, c1, 1);
#pragma unroll
    for (int t = 0; t < S::MT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 16 * t + 4 * quarter + i;
        if (r < rows) {
          const float w = weight_of[wave][r];
          float* row = mine + token_of[wave][r] * C::COLS + l16;
#pragma unroll
          for (int c = 0; c < S::CF; ++c) row[16 * c] += w * acc[t][c][i];
        }
      }
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  for (int i = tid; i < T * C::COLS; i += C::THREADS) {
    const int t = i / C::COLS, n = n0 + (i & (C::COLS - 1));
    float v = sums[i];
#pragma unroll
    for (int w = 1; w < C::WAVES; ++w) v += sums[w * T * C::COLS + i];
    if (n < p.K) p.D[(int64_t)(t0 + t) * p.ldd + n] = bf16_bits(v);
  }
}

}  // namespace fg
