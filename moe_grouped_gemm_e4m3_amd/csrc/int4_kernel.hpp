// int4_kernel.hpp -- the cast to 4-bit codes and the product of a few bf16 rows
// with them.
//
//   cast     symmetric:  s = bf16(max(amax, 1e-20) / 7),   z = 8
//            zero point: s = bf16(max(hi - lo, 1e-20) / 15), z = rint(-lo / s)     lo <= 0 <= hi
//            q = clamp(rint(x / s) + z, 0, 15)
//   product  D[m, n] = bf16( sum_k A[m, k] s[n, k/g] (B[n, k] - z[n, k/g]) )
#pragma once

#include "weight_stream.hpp"

namespace fg {

constexpr int kInt4Chunk = 64;  // bytes of 128 codes

// Byte offset in a row of the word that holds columns 8 word .. 8 word + 7.
__device__ __forceinline__ int64_t int4_word_at(int word) {
  const int in = word & 15;
  return (int64_t)(word >> 4) * kInt4Chunk + ((in & 3) * 4 + (in >> 2)) * 4;
}

struct Int4CastParams {
  const void* x;
  int64_t ldx;  // elements
  uint8_t* q;
  uint16_t* s;
  uint8_t* z;  // NULL: symmetric
  int N, K, group;
  int groups, words;  // of a row: scale groups; words with the padding ones
  int64_t units;      // rows x unit groups
  int per_row;        // unit groups of a row
};

template <typename T>
__device__ __forceinline__ void int4_load8(const T* x, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const f32x4 a = *(const f32x4_at4*)x, b = *(const f32x4_at4*)(x + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
    const i32x4 a = *(const i32x4_at2*)x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float((uint32_t)a[i] << 16);
      v[2 * i + 1] = __uint_as_float((uint32_t)a[i] & 0xffff0000u);
    }
  }
}

// LANES lanes share a group and take its words in turn (groups of up to 128:
// a word each, and the row is read once; longer ones are read twice, the second
// time from cache).  fp32 is bound by HBM, 4.5 bytes for each weight (7168 x 16384:
// 113 to 121 us, 4.4 to 4.7 TB/s), bf16 by the division and the rounding of each (93
// to 104 us, 2.8 to 3.2 TB/s).
template <typename T, int LANES>
__global__ __launch_bounds__(256) void int4_cast_kernel(Int4CastParams p) {
  constexpr int UNITS = 256 / LANES;
  const int l = threadIdx.x % LANES;
  const int group_words = p.group / 8, k_words = p.K / 8;
  for (int64_t u0 = (int64_t)blockIdx.x * UNITS; u0 < p.units; u0 += (int64_t)gridDim.x * UNITS) {
    // lanes past the last unit follow it, for the exchanges, and store nothing
    const int64_t u = min(u0 + threadIdx.x / LANES, p.units - 1);
    const bool live = u0 + threadIdx.x / LANES < p.units;
    const int64_t n = u / p.per_row;
    const int g = (int)(u - n * p.per_row);
    const T* row = (const T*)p.x + n * p.ldx;
    const int w0 = g * group_words, w1 = min(w0 + group_words, k_words);
    float lo = 0.f, hi = 0.f, v[8];
    for (int w = w0 + l; w < w1; w += LANES) {
      int4_load8(row + 8 * w, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
      }
    }
#pragma unroll
    for (int d = 1; d < LANES; d *= 2) {
      lo = fminf(lo, __shfl_xor(lo, d));
      hi = fmaxf(hi, __shfl_xor(hi, d));
    }
    // half the span over 7.5: the same bits as the span over 15, and no overflow
    const float span = p.z ? (0.5f * hi - 0.5f * lo) / 7.5f : fmaxf(hi, -lo) / 7.f;
    const uint16_t sb = bf16_bits(fmaxf(span, p.z ? 1e-20f / 15.f : 1e-20f / 7.f));
    const float s = to_f32(sb);
    const float z = p.z ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 8.f;
    if (live && l == 0 && g < p.groups) {
      p.s[n * p.groups + g] = sb;
      if (p.z) p.z[n * p.groups + g] = (uint8_t)z;
    }
    // the last group's lanes write the row's padding words too
    const int end = g == p.per_row - 1 ? p.words : w0 + group_words;
    for (int w = w0 + l; w < end; w += LANES) {
      uint32_t word = 0;
      if (w < w1) {
        if (group_words > LANES || g == p.per_row - 1) int4_load8(row + 8 * w, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t c = (uint32_t)fminf(fmaxf(rintf(v[i] / s) + z, 0.f), 15.f);
          word |= c << (8 * (i & 3) + 4 * (i >> 2));
        }
      }
      if (live) *(uint32_t*)(p.q + n * (int64_t)p.words * 4 + int4_word_at(w)) = word;
    }
  }
}

struct Int4Params {
  const uint16_t* A;
  int64_t lda;  // elements
  const uint8_t* B;
  const uint16_t* s;
  const uint8_t* z;  // NULL: 8
  uint16_t* D;
  int64_t ldd;
  int M, N, K, group, groups;
  int row_bytes;  // of B
  int parts;      // row parts
};

// The weights and activations of a tile: rows [m0, m0 + rows) of A, weight rows
// from n0 on.
template <class S>
__device__ __forceinline__ void set_tile(Sources<S>& src, const Int4Params& p, int m0, int rows, int n0) {
  src.K = p.K;
  set_group(src, p.group);
  // rows past N are outside the ranges and read as zeros
  src.q[0] = make_rsrc(p.B + (int64_t)n0 * p.row_bytes, (int64_t)(p.N - n0) * p.row_bytes);
  src.s[0] = make_rsrc(p.s + (int64_t)n0 * p.groups, (int64_t)(p.N - n0) * p.groups * 2);
  src.z[0] = make_rsrc(p.z ? p.z + (int64_t)n0 * p.groups : nullptr, p.z ? (int64_t)(p.N - n0) * p.groups : 0);
  src.row_bytes = p.row_bytes;
  src.groups = p.groups;
  src.x = make_rsrc(p.A + (int64_t)m0 * p.lda, ((int64_t)(rows - 1) * p.lda + p.K) * 2);
#pragma unroll
  for (int i = 0; i < S::X_LOADS; ++i) src.x_off[i] = min(x_row_of<S>(i), rows - 1) * (int)(2 * p.lda);
}

// A tile of ROWS rows and 16 CF columns; the waves share out its chunks of K, each
// through a ring of its own ("split").  For tiles that all fit on the CUs at once:
// then a call is the latency of a launch, a first load and a wave's few chunks (1 x
// 7168 x 2048: 4.0 us, 7.7 MB; 16 x 2112 x 7168: 7.9 us; 1 x 24576 x 1536, 20 MB in
// six rounds of workgroups: 7.4 us, 2.7 TB/s).
template <class Fmt, int ROWS_, int CF_, int WAVES_, int DEPTH_>
struct Int4Tile {
  static constexpr int MT = (ROWS_ + 15) / 16, CF = CF_, WAVES = WAVES_;
  static constexpr int NX = ROWS_ > 2 ? ROWS_ / 2 : 1;
  static constexpr int RING = DEPTH_ * (CF * 2048 + NX * 1024);
  using S = Stream<Fmt, MT, NX, CF, 1, 0, RING>;
  static constexpr int THREADS = 64 * WAVES, ROWS = ROWS_, COLS = 16 * CF;
  static constexpr int BLOCKS = MT * CF;
  static constexpr int WAVE_LDS = RING + scale_lds<Fmt, CF>();
  static_assert(BLOCKS * 1024 <= WAVE_LDS, "LDS");
};

// Grid: column tiles x row parts, parts fastest.  The waves' partials are added
// in wave order.
template <class C>
__global__ __launch_bounds__(C::THREADS) void int4_product_kernel(Int4Params p) {
  using S = typename C::S;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::WAVES * C::WAVE_LDS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile = blockIdx.x / p.parts;
  const int m0 = (blockIdx.x - tile * p.parts) * C::ROWS, n0 = tile * C::COLS;
  const int rows = min(C::ROWS, p.M - m0);
  Sources<S> src;
  set_tile(src, p, m0, rows, n0);

  f32x4 acc[S::MT][S::CF];
#pragma unroll
  for (int t = 0; t < S::MT; ++t)
#pragma unroll
    for (int c = 0; c < S::CF; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint8_t* mine = lds + wave * C::WAVE_LDS;
  const int chunks = (p.K + S::COLS - 1) / S::COLS;
  stream_chunks<S>(acc, src, mine, nullptr, (uint32_t*)(mine + C::RING), chunks * wave / C::WAVES, chunks * (wave + 1) / C::WAVES,
                   5 * tile);
  f32x4* sums = (f32x4*)mine;
#pragma unroll
  for (int t = 0; t < S::MT; ++t)
#pragma unroll
    for (int c = 0; c < S::CF; ++c) sums[(t * S::CF + c) * 64 + lane] = acc[t][c];
  __syncthreads();
  for (int x = threadIdx.x; x < C::BLOCKS * 256; x += C::THREADS) {
    const int col = x & (C::COLS - 1), row = x / C::COLS;
    const int at = (((row >> 4) * S::CF + (col >> 4)) * 64 + ((row & 15) >> 2) * 16 + (col & 15)) * 4 + (row & 3);
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < C::WAVES; ++w) v += ((const float*)(lds + w * C::WAVE_LDS))[at];
    if (row < rows && n0 + col < p.N) p.D[(int64_t)(m0 + row) * p.ldd + n0 + col] = bf16_bits(v);
  }
}

// A tile of ROWS rows and 16 CF WAVES columns and a part of K; the waves share
// the activations' columns ("wide"): a workgroup's X is read once for 128 columns
// instead of 16.  64 x 7168 x 16384 takes 35.4 us (64 MB; 424 TFLOP/s) for 78 or
// more of the split tiles: a chunk costs its 1.9 us of products, widening and LDS
// reads, which is what bounds it, not the 13 us of its weights.
template <class Fmt_, int ROWS_, int CF_, int WAVES_, int DEPTH_>
struct Int4Wide {
  using Fmt = Fmt_;
  static constexpr int MT = ROWS_ / 16, CF = CF_, WAVES = WAVES_, ROWS = ROWS_;
  static constexpr int RING = DEPTH_ * (WAVES * CF * 2048 + ROWS * 512);
  using S = Stream<Fmt, MT, ROWS / 2, CF, 1, 0, RING, WAVES>;
  static constexpr int THREADS = 64 * WAVES, COLS = 16 * CF * WAVES;
  static constexpr int SCALE_LDS = scale_lds<Fmt, CF>(), LDS = RING + WAVES * SCALE_LDS;
};

// Grid: column tiles, row parts, parts of K.
template <class C>
__global__ __launch_bounds__(C::THREADS) void int4_wide_kernel(Int4Params p, float* partial) {
  using S = typename C::S;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::LDS];
  const int lane = threadIdx.x & 63, l16 = lane & 15, quarter = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m0 = blockIdx.y * C::ROWS, n0 = blockIdx.x * C::COLS + 16 * C::CF * wave;
  const int rows = min(C::ROWS, p.M - m0);
  Sources<S> src;
  set_tile(src, p, m0, rows, min(n0, p.N - 1));  // past N: some rows that are there, for nothing
  f32x4 acc[S::MT][S::CF];
#pragma unroll
  for (int t = 0; t < S::MT; ++t)
#pragma unroll
    for (int c = 0; c < S::CF; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int chunks = (p.K + S::COLS - 1) / S::COLS;
  const int first = (int)((int64_t)chunks * blockIdx.z / gridDim.z), end = (int)((int64_t)chunks * (blockIdx.z + 1) / gridDim.z);
  stream_chunks<S>(acc, src, lds, nullptr, (uint32_t*)(lds + C::RING + wave * C::SCALE_LDS), first, end, 5 * blockIdx.x);
#pragma unroll
  for (int t = 0; t < S::MT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 16 * t + 4 * quarter + i;
      if (row >= rows) continue;
#pragma unroll
      for (int c = 0; c < S::CF; ++c) {
        const int n = n0 + 16 * c + l16;
        if (n >= p.N) continue;
        if (gridDim.z == 1)
          p.D[(int64_t)(m0 + row) * p.ldd + n] = bf16_bits(acc[t][c][i]);
        else
          partial[((int64_t)blockIdx.z * p.M + m0 + row) * p.N + n] = acc[t][c][i];
      }
    }
}

}  // namespace fg
