// experts_kernel.hpp -- a whole expert layer for a few tokens, in two kernels.
//
//   up    g = W1[e][0:F] x_t, u = W1[e][F:2F] x_t, h = act(g) u      for every pair (t, j) with e = ids[t, j]
//   down  D[t] = bf16( sum_j w[t, j] W2[e] h_(t, j) )
//
// Every active expert's weights are read once for each 64 tokens
// (weight_stream.hpp); that read is the time where they are many (one token, 8
// experts of 2048 x 7168 in e4m3: 352 MB in 67.7 us, 5.2 TB/s, a little more than a
// copy's reads and writes together; 64 tokens over 16 of them: 706 MB in 162 us, 4.4
// TB/s).  `up` has workgroups for
// each expert and tile of hidden units; an expert's tokens are the rows of the
// matrix product.  `down` has workgroups for tiles of outputs, which go through
// all active experts, so that the sum over experts stays inside: sums of its own
// for each token and output, in LDS.  Both come in two organisations.
//
//   split  a tile is 16 units (or 16 or 32 outputs), and its waves share out the
//          reduction, each with an LDS ring of its own, and are added in wave
//          order: many independent small streams, for few tokens, where latency
//          counts (one token, 6 experts of 704 x 2048 in 4 bits: 16.0 us)
//   wide   a tile is 64 or 128 units (128 outputs), and its waves have rows of
//          their own and share one copy of the tokens' columns, with a barrier a
//          chunk: fewer bytes through LDS for a weight.  `down` then splits all
//          experts' chunks over workgroups, whose sums a third kernel adds in
//          their order (39 tokens, 2 of 64 experts of 2048 x 1024 each in 4 bits: 67
//          us; in one part 558)
//
// A kernel takes so many tokens of an expert at a time: `up` 2, 4 or 16 (split) and
// 16 or 32 (wide), `down` 1 or 4 and 16, 24 or 32.  For more of them it streams the
// expert's weights again, one time after the other, from cache where they fit.  The
// plan goes by the average, so that ids which crowd on one expert cost more (16
// tokens, one of 16 4-bit experts of 1024 x 2048 each, spread 30 us, all on one 43).
//
// No sum depends on the order in which workgroups run, and there are no atomics
// on results.
//
// h is held in 32 bits: it passes through the workspace as fp32, and `down` makes
// three bf16 of it in LDS whose sum it is exactly, three products of a weight tile
// in the place of one.
//
// A token that names an expert twice has one product with the sum of both
// weights, at the first of the two places.
#pragma once

#include "decode_plan.hpp"
#include "weight_stream.hpp"

namespace fg {

static_assert(kLayerTokens == 64, "a lane for each token");
constexpr int kMaxExperts = 1024, kMaxChoices = 32;  // `down` keeps them in LDS (Pairs): 25 KiB at most

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
  float* H;  // [T k][F]: every pair's h
  int T, k, E, F, K, act;
  int group;
  int row1, row2;        // bytes of a weight row
  int groups1, groups2;  // scale groups (e4m3: block columns) of a row
  bool by_pair;  // up: blockIdx.y is a pair (fewer pairs than experts), else an expert
};

// Rows [row0, row0 + 16 PER) of rows x cols weights of expert e in region r of src.
template <class S>
__device__ __forceinline__ void set_weights(Sources<S>& src, int r, const uint8_t* W, const void* s, const uint8_t* z,
                                            int e, int rows, int row0, int row_bytes, int groups) {
  const int64_t at = (int64_t)e * rows + row0;
  src.q[r] = make_rsrc(W + at * row_bytes, (int64_t)(rows - row0) * row_bytes);
  src.row_bytes = row_bytes;
  src.groups = groups;
  if constexpr (S::FP8) {
    // a tile of 16 rows lies in one block row; rows past the matrix follow its last
    const int blocks = (rows + 127) >> 7;
#pragma unroll
    for (int i = 0; i < S::PER; ++i)
      src.fs[r * S::PER + i] = (const float*)s + ((int64_t)e * blocks + min((row0 + 16 * i) >> 7, blocks - 1)) * groups;
  } else {
    src.s[r] = make_rsrc((const uint16_t*)s + at * groups, (int64_t)(rows - row0) * groups * 2);
    src.z[r] = make_rsrc(z ? z + at * groups : nullptr, z ? (int64_t)(rows - row0) * groups : 0);
  }
}

template <class S>
__device__ __forceinline__ void clear(f32x4 (&acc)[S::MT][S::CF]) {
#pragma unroll
  for (int t = 0; t < S::MT; ++t)
#pragma unroll
    for (int c = 0; c < S::CF; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// h of token t's place j and hidden unit f.
__device__ __forceinline__ void store_hidden(const ExpertParams& p, int t, int j, int f, float g, float u) {
  p.H[((int64_t)t * p.k + j) * p.F + f] =
      p.act == kActSilu ? gated_value<kActSilu>(g, u) : gated_value<kActGeluTanh>(g, u);
}

// PER: tiles of 16 hidden units.  MOST: tokens of an expert in one go (2, 4 or 16).
template <class Fmt_, int PER_, int WAVES_, int DEPTH_, int MOST_>
struct UpTile {
  using Fmt = Fmt_;
  static constexpr bool WIDE = false;
  static constexpr int PER = PER_, WAVES = WAVES_, MOST = MOST_;
  static constexpr int RING = DEPTH_ * (2 * PER * 2048 + x_kib(Fmt::FP8, MOST) * 1024);
  static constexpr int MT = MOST > 16 ? 2 : 1, THREADS = 64 * WAVES, UNITS = 16 * PER;
  static constexpr int WAVE_LDS = RING + scale_lds<Fmt, 2 * PER>();
  static constexpr int BLOCKS = 2 * PER * MT;  // 16 x 16 sums of a wave
  static_assert(BLOCKS * 1024 <= WAVE_LDS, "LDS");
};

// Up to ROWS member tokens, from member `base` on, and C::UNITS hidden units.
template <class C, int ROWS>
__device__ __forceinline__ void up_tile(const ExpertParams& p, int e, int t0, int f0, int base, int members,
                                        const int* list, uint8_t* lds) {
  constexpr int MT = ROWS > 16 ? 2 : 1;
  using S = Stream<typename C::Fmt, MT, x_kib(C::Fmt::FP8, ROWS), 2 * C::PER, 2, 0, C::RING>;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Sources<S> src;
  src.K = p.K;
  set_group(src, p.group);
  set_weights(src, 0, p.W1, p.s1, p.z1, e, 2 * p.F, f0, p.row1, p.groups1);
  set_weights(src, 1, p.W1, p.s1, p.z1, e, 2 * p.F, p.F + f0, p.row1, p.groups1);
  const int T = min(kLayerTokens, p.T - t0);
  src.x = make_rsrc(p.X + (int64_t)t0 * p.ldx, ((int64_t)(T - 1) * p.ldx + p.K) * 2);
#pragma unroll
  for (int i = 0; i < S::X_LOADS; ++i) src.x_off[i] = (list[min(base + x_row_of<S>(i), members - 1)] & 63) * (int)(2 * p.ldx);

  f32x4 acc[MT][2 * C::PER];
  clear<S>(acc);
  uint8_t* mine = lds + wave * C::WAVE_LDS;
  const int chunks = (p.K + S::COLS - 1) / S::COLS;
  stream_chunks<S>(acc, src, mine, nullptr, (uint32_t*)(mine + C::RING), chunks * wave / C::WAVES, chunks * (wave + 1) / C::WAVES,
                   5 * blockIdx.x);
  f32x4* sums = (f32x4*)mine;
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int c = 0; c < 2 * C::PER; ++c) sums[(2 * C::PER * t + c) * 64 + lane] = acc[t][c];
  __syncthreads();
  for (int x = threadIdx.x; x < MT * C::PER * 256; x += C::THREADS) {
    const int col = x & 15, row = (x >> 4) & 15, b = x >> 8, t = b / C::PER, c = b - t * C::PER;
    const int at = ((2 * C::PER * t + c) * 64 + (row >> 2) * 16 + col) * 4 + (row & 3);
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int w = 0; w < C::WAVES; ++w) {
      const float* part = (const float*)(lds + w * C::WAVE_LDS);
      g += part[at];
      u += part[at + C::PER * 256];
    }
    const int m = base + 16 * t + row, f = f0 + 16 * c + col;
    if (m < members && f < p.F && 16 * t + row < ROWS) {
      const int pair = list[m];
      store_hidden(p, t0 + (pair & 63), pair >> 6, f, g, u);
    }
  }
}

// The expert of a workgroup of `up`, and its tokens in `list` (t | place << 6,
// the first place that names it).  -> how many; 0: nothing to do.
__device__ __forceinline__ int expert_tokens(const ExpertParams& p, int t0, int& e, int* list) {
  const int lane = threadIdx.x & 63, T = min(kLayerTokens, p.T - t0);
  const int32_t* ids = p.ids + (int64_t)t0 * p.k;
  e = blockIdx.y;
  if (p.by_pair) {
    if ((int)blockIdx.y >= T * p.k) return 0;
    e = load_invariant(ids + blockIdx.y);
    if ((unsigned)e >= (unsigned)p.E) return 0;
  }
  // the first of this lane's token's places that name e; ids come eight at a time
  int place = -1;
  if (lane < T)
    for (int j0 = (p.k - 1) & ~7; j0 >= 0; j0 -= 8) {
      int id[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) id[j] = ids[lane * p.k + min(j0 + j, p.k - 1)];
#pragma unroll
      for (int j = 7; j >= 0; --j)
        if (id[j] == e) place = min(j0 + j, p.k - 1);
    }
  const unsigned long long mask = __ballot(place >= 0);
  if (mask == 0) return 0;
  if (p.by_pair) {
    // the first pair of an expert stands for all of them
    const int first = __builtin_ctzll(mask);
    if (first * p.k + __builtin_amdgcn_readlane(place, first) != (int)blockIdx.y) return 0;
  }
  if (threadIdx.x < 64 && place >= 0) list[__builtin_popcountll(mask & ((1ull << lane) - 1))] = lane | place << 6;
  __syncthreads();
  return __builtin_popcountll(mask);
}

// Grid: tiles of C::UNITS hidden units, pairs or experts, passes of 64 tokens.
template <class C>
__global__ __launch_bounds__(C::THREADS) void experts_up_kernel(ExpertParams p) {
  // one object: with two, the compiler waits for all loads into LDS before a read of it
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::WAVES * C::WAVE_LDS + kLayerTokens * 4];
  int* list = (int*)(lds + C::WAVES * C::WAVE_LDS);
  const int t0 = blockIdx.z * kLayerTokens, f0 = blockIdx.x * C::UNITS;
  int e;
  const int members = expert_tokens(p, t0, e, list);
  for (int base = 0; base < members; base += C::MOST) {
    if (base) __syncthreads();  // the sums are read
    const int left = members - base;
    if (C::MOST <= 4 || left <= 4)
      up_tile<C, C::MOST < 4 ? C::MOST : 4>(p, e, t0, f0, base, members, list, lds);
    else
      up_tile<C, C::MOST>(p, e, t0, f0, base, members, list, lds);
  }
}

// ---- wide: the waves of a workgroup share the tokens' columns ----

// PER: tiles of 16 hidden units of a wave.  MOST: tokens of an expert in one go.

template <class Fmt_, int PER_, int WAVES_, int DEPTH_, int MOST_>
struct WideUp {
  using Fmt = Fmt_;
  static constexpr bool WIDE = true;
  static constexpr int PER = PER_, WAVES = WAVES_, THREADS = 64 * WAVES, UNITS = 16 * PER * WAVES, MOST = MOST_;
  static constexpr int SCALES = Fmt::GPC == 4 ? 64 : 32;
  static constexpr int RING = DEPTH_ * (WAVES * PER * 4096 + x_kib(Fmt::FP8, MOST) * 1024);
  static constexpr int SCALE_LDS = scale_lds<Fmt, 2 * PER, SCALES>();  // of a wave
  static constexpr int LDS = RING + WAVES * SCALE_LDS;
};

template <class C, int ROWS>
__device__ __forceinline__ void wide_up_tile(const ExpertParams& p, int e, int t0, int f0, int base, int members,
                                             const int* list, uint8_t* ring, uint8_t* scales) {
  constexpr int MT = ROWS > 16 ? 2 : 1;
  using S = Stream<typename C::Fmt, MT, x_kib(C::Fmt::FP8, ROWS), 2 * C::PER, 2, 0, C::RING, C::WAVES, C::SCALES>;
  const int lane = threadIdx.x & 63, l16 = lane & 15, quarter = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Sources<S> src;
  src.K = p.K;
  set_group(src, p.group);
  const int f = f0 + 16 * C::PER * wave;  // past F: some rows that are there, for nothing
  set_weights(src, 0, p.W1, p.s1, p.z1, e, 2 * p.F, min(f, p.F - 16), p.row1, p.groups1);
  set_weights(src, 1, p.W1, p.s1, p.z1, e, 2 * p.F, p.F + min(f, p.F - 16), p.row1, p.groups1);
  const int T = min(kLayerTokens, p.T - t0);
  src.x = make_rsrc(p.X + (int64_t)t0 * p.ldx, ((int64_t)(T - 1) * p.ldx + p.K) * 2);
#pragma unroll
  for (int i = 0; i < S::X_LOADS; ++i) src.x_off[i] = (list[min(base + x_row_of<S>(i), members - 1)] & 63) * (int)(2 * p.ldx);
  f32x4 acc[MT][2 * C::PER];
  clear<S>(acc);
  stream_chunks<S>(acc, src, ring, nullptr, (uint32_t*)(scales + wave * C::SCALE_LDS), 0, (p.K + S::COLS - 1) / S::COLS,
                   5 * blockIdx.x);
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = base + 16 * t + 4 * quarter + i;
      if (m >= members || 16 * t + 4 * quarter + i >= ROWS) continue;
      const int pair = list[m];
#pragma unroll
      for (int c = 0; c < C::PER; ++c)
        if (f + 16 * c + l16 < p.F)
          store_hidden(p, t0 + (pair & 63), pair >> 6, f + 16 * c + l16, acc[t][c][i], acc[t][C::PER + c][i]);
    }
}

template <class C>
__global__ __launch_bounds__(C::THREADS) void experts_wide_up_kernel(ExpertParams p) {
  __shared__ __attribute__((aligned(1024))) uint8_t ring[C::LDS + kLayerTokens * 4];
  uint8_t* scales = ring + C::RING;
  int* list = (int*)(ring + C::LDS);
  const int t0 = blockIdx.z * kLayerTokens, f0 = blockIdx.x * C::UNITS;
  int e;
  const int members = expert_tokens(p, t0, e, list);
  for (int base = 0; base < members; base += C::MOST) {
    if (C::MOST == 16 || members - base <= 16)
      wide_up_tile<C, 16>(p, e, t0, f0, base, members, list, ring, scales);
    else
      wide_up_tile<C, C::MOST>(p, e, t0, f0, base, members, list, ring, scales);
  }
}

// CF: tiles of 16 outputs.  MOST: tokens of an expert in one go (1 or 4).  Two
// tiles halve the activations' loads for a weight, and the workgroups.  LDS sizes
// are those of down_lds.
template <class Fmt_, DownKind KIND_>
struct DownTile {
  using Fmt = Fmt_;
  static constexpr DownShape SHAPE = down_shape(Fmt::FP8, KIND_);
  static constexpr int CF = SHAPE.tiles, WAVES = SHAPE.waves, MOST = SHAPE.rows;
  static constexpr int RING = down_ring(Fmt::FP8, KIND_), X_BYTES = down_x(Fmt::FP8, KIND_);
  static constexpr int THREADS = 64 * WAVES, COLS = 16 * CF;
  static constexpr int WAVE_LDS = RING + X_BYTES + scale_lds<Fmt, CF>();
};

// What `down` knows of the pairs, in dynamic LDS: the experts with tokens, and
// for each its tokens in order, with the first place that names it and the
// weights of all such places.
struct Pairs {
  unsigned long long* tokens;  // [E] that go to an expert
  float* weight;               // [T k]
  int* items;                  // [1] experts with tokens
  uint16_t *expert;            // [min(E, T k)] of an item
  uint16_t *start;             // [E] of its tokens in `weight` and `pair`
  uint16_t *pair;              // [T k]: t k + j
};
__device__ __forceinline__ Pairs pairs_at(uint8_t* lds, int E, int n) {
  Pairs s;
  s.tokens = (unsigned long long*)lds;
  s.weight = (float*)(s.tokens + E);
  s.items = (int*)(s.weight + n);
  s.expert = (uint16_t*)(s.items + 1);
  s.start = s.expert + E;
  s.pair = s.start + E;
  return s;
}

__device__ __forceinline__ void sort_pairs(const Pairs& s, const ExpertParams& p, int t0, int T) {
  const int tid = threadIdx.x, lane = tid & 63, n = T * p.k;
  const int32_t* ids = p.ids + (int64_t)t0 * p.k;
  const float* weights = p.w + (int64_t)t0 * p.k;
  for (int i = tid; i < p.E; i += blockDim.x) s.tokens[i] = 0;
  if (tid == 0) *s.items = 0;
  __syncthreads();
  bool twice = false;
  for (int i = tid; i < n; i += blockDim.x) {
    const int e = ids[i];
    const unsigned long long bit = 1ull << (i / p.k);
    if ((unsigned)e < (unsigned)p.E) twice |= (atomicOr(&s.tokens[e], bit) & bit) != 0;
  }
  if (twice) *s.items = 1;  // some token names an expert twice
  __syncthreads();
  twice = *s.items != 0;
  __syncthreads();
  if (tid < 64) {
    int count = 0, start = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      const int e = e0 + lane;
      const int members = e < p.E ? __builtin_popcountll(s.tokens[e]) : 0;
      const unsigned long long any = __ballot(members > 0);
      if (any == 0) continue;
      int before = members;  // inclusive sum over the lanes
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(before, d);
        if (lane >= d) before += o;
      }
      if (members > 0) {
        s.expert[count + __builtin_popcountll(any & ((1ull << lane) - 1))] = (uint16_t)e;
        s.start[e] = (uint16_t)(start + before - members);
      }
      count += __builtin_popcountll(any);
      start += __builtin_amdgcn_readlane(before, 63);
    }
    if (lane == 0) *s.items = count;
  }
  __syncthreads();
  for (int i = tid; i < n; i += blockDim.x) {
    const int e = ids[i], t = i / p.k;
    if ((unsigned)e >= (unsigned)p.E) continue;
    float w = weights[i];
    if (twice) {
      bool first = true;
      for (int j = t * p.k; j < i; ++j) first &= ids[j] != e;
      if (!first) continue;
      for (int j = i + 1; j < (t + 1) * p.k; ++j)
        if (ids[j] == e) w += weights[j];
    }
    const int at = s.start[e] + __builtin_popcountll(s.tokens[e] & ((1ull << t) - 1));
    s.pair[at] = (uint16_t)i;
    s.weight[at] = w;
  }
  __syncthreads();
}

// Token r of an item.
struct Member {
  int token, pair;
  float w;
};
__device__ __forceinline__ Member member(const ExpertParams& p, const Pairs& s, int e, int r) {
  const int at = s.start[e] + r;
  return Member{s.pair[at] / p.k, s.pair[at], s.weight[at]};
}

// Grid: tiles of COLS outputs, passes of 64 tokens.
template <class C>
__global__ __launch_bounds__(C::THREADS) __attribute__((amdgpu_waves_per_eu(2, 4))) void experts_down_kernel(ExpertParams p) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, quarter = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t0 = blockIdx.y * kLayerTokens, T = min(kLayerTokens, p.T - t0);
  const int n0 = blockIdx.x * C::COLS;
  float* sums = (float*)(lds + C::WAVES * C::WAVE_LDS);  // [WAVES][T][COLS]
  const Pairs pairs = pairs_at((uint8_t*)(sums + C::WAVES * T * C::COLS), p.E, T * p.k);
  for (int i = tid; i < C::WAVES * T * C::COLS; i += C::THREADS) sums[i] = 0.f;
  sort_pairs(pairs, p, t0, T);

  using S = Stream<typename C::Fmt, 1, 0, C::CF, 1, C::MOST, C::RING>;
  static_assert(S::X_BYTES == C::X_BYTES, "LDS");
  const int chunks = (p.F + S::COLS - 1) / S::COLS;
  const int items = __builtin_amdgcn_readfirstlane(*pairs.items), total = items * chunks;
  int at = (int)((int64_t)total * wave / C::WAVES), end = (int)((int64_t)total * (wave + 1) / C::WAVES);
  if (items <= C::WAVES) {
    // every wave inside an item: a second one would cost another wait for its first weights
    const int each = items > 0 ? C::WAVES / items : 1, item = wave / each, part = wave - item * each;
    at = item < items ? item * chunks + chunks * part / each : 0;
    end = item < items ? item * chunks + chunks * (part + 1) / each : 0;
  }
  float* mine = sums + wave * T * C::COLS;
  uint8_t* ring = lds + wave * C::WAVE_LDS;
  while (at < end) {
    const int item = __builtin_amdgcn_readfirstlane(at / chunks), c0 = at - item * chunks;
    const int c1 = min(chunks, c0 + end - at);
    at += c1 - c0;
    const int e = __builtin_amdgcn_readfirstlane(pairs.expert[item]);
    const int members = __builtin_amdgcn_readfirstlane(__builtin_popcountll(pairs.tokens[e]));
    for (int base = 0; base < members; base += C::MOST) {
      const int rows = min(C::MOST, members - base);
      const Member me = member(p, pairs, e, base + min(l16, rows - 1));
      Sources<S> src;
      src.K = p.F;
      set_group(src, p.group);
      src.x = make_rsrc(p.H + (int64_t)t0 * p.k * p.F, (int64_t)T * p.k * 4 * p.F);
      set_weights(src, 0, p.W2, p.s2, p.z2, e, p.K, n0, p.row2, p.groups2);
#pragma unroll
      for (int i = 0; i < S::X_LOADS; ++i) {
        const int r = min(x_row_of<S>(i), rows - 1);
        src.x_off[i] = __shfl(me.pair, r) * 4 * p.F;
      }
      f32x4 acc[S::MT][S::CF];
      clear<S>(acc);
      stream_chunks<S>(acc, src, ring, ring + C::RING, (uint32_t*)(ring + C::RING + C::X_BYTES), c0, c1, 5 * blockIdx.x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * quarter + i;
        const float wr = __shfl(me.w, r);
        const int tr = __shfl(me.token, r);
        if (r < rows) {
          float* row = mine + tr * C::COLS + l16;
#pragma unroll
          for (int c = 0; c < S::CF; ++c) row[16 * c] += wr * acc[0][c][i];
        }
      }
    }
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

// Waves share an item's hidden units; a workgroup does a part of all items'
// chunks for COLS outputs and, with more than one part, leaves its sums to
// join_parts_kernel.
template <class Fmt_, DownKind KIND_>
struct WideDown {
  using Fmt = Fmt_;
  static constexpr DownShape SHAPE = down_shape(Fmt::FP8, KIND_);
  static constexpr int CF = SHAPE.tiles, WAVES = SHAPE.waves, COLS = 16 * CF * WAVES, MOST = SHAPE.rows;
  static constexpr int THREADS = 128 * WAVES;  // waves that multiply, then as many that split hidden units
  static constexpr int RING = down_ring(Fmt::FP8, KIND_), X_BYTES = down_x(Fmt::FP8, KIND_);
  static constexpr int EU_WAVES = Fmt::FP8 && MOST == 16 ? 4 : 2;  // that LDS leaves room for, at most
  static constexpr int SCALE_LDS = scale_lds<Fmt, CF>();
  static constexpr int TOKENS_AT = RING + X_BYTES + WAVES * SCALE_LDS;
};

template <class C, int ROWS>
__device__ __forceinline__ void wide_down_item(const ExpertParams& p, const Pairs& pairs, int t0, int T, int e, int base,
                                               int members, int n0, int c0, int c1, uint8_t* ring, uint8_t* scales,
                                               float* sums) {
  constexpr int MT = ROWS > 16 ? 2 : 1;
  using S = Stream<typename C::Fmt, MT, 0, C::CF, 1, ROWS, C::RING, C::WAVES>;
  static_assert(2 * S::X_BYTES <= C::X_BYTES, "LDS");
  const int lane = threadIdx.x & 63, l16 = lane & 15, quarter = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rows = min(ROWS, members - base);
  const Member me = member(p, pairs, e, base + min(lane & (16 * MT - 1), rows - 1));
  Sources<S> src;
  src.K = p.F;
  set_group(src, p.group);
  src.x = make_rsrc(p.H + (int64_t)t0 * p.k * p.F, (int64_t)T * p.k * 4 * p.F);
  set_weights(src, 0, p.W2, p.s2, p.z2, e, p.K, min(n0 + 16 * C::CF * wave, p.K - 16), p.row2,
              p.groups2);  // past K: some rows that are there, for nothing
#pragma unroll
  for (int i = 0; i < S::X_LOADS; ++i) {
    const int r = min(x_row_of<S>(i), rows - 1);
    src.x_off[i] = __shfl(me.pair, r) * 4 * p.F;
  }
  if (wave >= C::WAVES) return split_chunks<S>(src, ring + C::RING, c0, c1, 5 * blockIdx.x);
  f32x4 acc[MT][C::CF];
  clear<S>(acc);
  stream_chunks<S>(acc, src, ring, ring + C::RING, (uint32_t*)(scales + wave * C::SCALE_LDS), c0, c1, 5 * blockIdx.x);
  float* mine = sums + 16 * C::CF * wave + l16;
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * t + 4 * quarter + i;
      const float w = __shfl(me.w, r);
      const int token = __shfl(me.token, r);
      if (r < rows) {
#pragma unroll
        for (int c = 0; c < C::CF; ++c) mine[token * C::COLS + 16 * c] += w * acc[t][c][i];
      }
    }
}

// Grid: tiles of COLS outputs, parts.  One pass of tokens from t0 on.
template <class C>
__global__ __launch_bounds__(C::THREADS) __attribute__((amdgpu_waves_per_eu(2, C::EU_WAVES))) void experts_wide_down_kernel(ExpertParams p, int t0, float* partial) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
  const int tid = threadIdx.x;
  const int T = min(kLayerTokens, p.T - t0);
  const int n0 = blockIdx.x * C::COLS;
  uint8_t* scales = lds + C::RING + C::X_BYTES;
  float* sums = (float*)(lds + C::TOKENS_AT);  // [T][COLS]
  const Pairs pairs = pairs_at((uint8_t*)(sums + T * C::COLS), p.E, T * p.k);
  for (int i = tid; i < T * C::COLS; i += C::THREADS) sums[i] = 0.f;
  sort_pairs(pairs, p, t0, T);
  constexpr int COLS = C::Fmt::FP8 ? 128 : 256;
  const int chunks = (p.F + COLS - 1) / COLS;
  const int total = __builtin_amdgcn_readfirstlane(*pairs.items) * chunks;
  int at = (int)((int64_t)total * blockIdx.y / gridDim.y);
  const int end = (int)((int64_t)total * (blockIdx.y + 1) / gridDim.y);
  while (at < end) {
    const int item = __builtin_amdgcn_readfirstlane(at / chunks), c0 = at - item * chunks;
    const int c1 = min(chunks, c0 + end - at);
    at += c1 - c0;
    const int e = __builtin_amdgcn_readfirstlane(pairs.expert[item]);
    const int members = __builtin_amdgcn_readfirstlane(__builtin_popcountll(pairs.tokens[e]));
    for (int base = 0; base < members; base += C::MOST) {
      if (C::MOST == 16 || members - base <= 16)
        wide_down_item<C, 16>(p, pairs, t0, T, e, base, members, n0, c0, c1, lds, scales, sums);
      else
        wide_down_item<C, C::MOST>(p, pairs, t0, T, e, base, members, n0, c0, c1, lds, scales, sums);
    }
  }
  __syncthreads();
  for (int i = tid; i < T * C::COLS; i += C::THREADS) {
    const int t = i / C::COLS, n = n0 + (i & (C::COLS - 1));
    if (n >= p.K) continue;
    if (gridDim.y == 1)
      p.D[(int64_t)(t0 + t) * p.ldd + n] = bf16_bits(sums[i]);
    else
      partial[((int64_t)blockIdx.y * T + t) * p.K + n] = sums[i];
  }
}

}  // namespace fg
