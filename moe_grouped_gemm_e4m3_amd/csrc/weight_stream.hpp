// weight_stream.hpp -- products of a few bf16 rows with e4m3 or 4-bit weights,
// streamed from HBM once: the inner loop of the 4-bit product (int4.hip) and of
// the few-token expert layers (experts.hip).
//
//   P[m, n] = sum_k X[m, k] Q[n, k]   over one scale group, on the matrix cores
//   e4m3:   acc[m, n] += s[n / 128, k / 128] P[m, n]
//   4 bits: acc[m, n] += s[n, k / g] (P[m, n] - z[n, k / g] sum_k X[m, k])
//
// A weight code becomes bf16 exactly (an e4m3 value and an integer of 0..15 have
// at most 4 significant bits), so products are exact and only fp32 sums round.
// A nibble in a byte read as e4m3 is its value times 2^-9 (codes 0..15 are the
// subnormals and the first binade), so the same conversion instruction serves
// both formats.  The zero point leaves the sum because it is constant in a
// group: the sum of X comes from the matrix cores too, as a product with ones.
//
// Weights go from global memory to registers in 16-byte loads, without LDS: a
// wave's 16 weight rows are the columns of a 16x16x32 MFMA, whose order of k is
// free as long as X's follows it.  A wave takes chunks of 128 columns and keeps
// DEPTH of them in flight.
#pragma once

#include "linear_kernel.hpp"

namespace fg {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

enum WeightFormat { kFp8Block, kInt4Group };

// GPC: scale groups in a chunk (4-bit: 4, 2 or 1 for groups of 32, 64 and any
// multiple of 128).  MT: row tiles of 16.  CF: weight tiles of 16 rows.  REGIONS:
// the weight tiles lie in so many places of the matrix (2: gate and up rows).
// PARTS: X is the sum of so many bf16 matrices.
template <int FMT_, int GPC_, int MT_, int CF_, int REGIONS_, int PARTS_, int DEPTH_>
struct Stream {
  static constexpr int FMT = FMT_, GPC = GPC_, MT = MT_, CF = CF_, REGIONS = REGIONS_, PARTS = PARTS_, DEPTH = DEPTH_;
  static constexpr bool FP8 = FMT == kFp8Block;
  static constexpr int WL = FP8 ? 2 : 1;      // 16-byte loads of a weight row's chunk and lane
  static constexpr int PER = CF / REGIONS;    // weight tiles of a region
  static_assert(CF % REGIONS == 0, "tiles");
};

// Where a wave's weights and activations are.  Offsets are a lane's, in bytes.
template <class S>
struct Sources {
  __amdgpu_buffer_rsrc_t q[S::REGIONS], s[S::REGIONS], z[S::REGIONS];
  int q_off, s_off, z_off;    // this lane's row of a region's first tile
  int q_tile, s_tile, z_tile;  // from one tile of a region to the next
  const float* fs[S::REGIONS];  // e4m3: the block row's factors
  __amdgpu_buffer_rsrc_t x;
  int x_off[S::MT];  // this lane's row of every row tile
  int x_part;        // from one part of X to the next
  int K, group;
  bool has_z, wide;  // wide: the scales of a chunk are one aligned load
};

template <class S>
struct Chunk {
  i32x4 w[S::CF][S::WL];
  i32x4 x[S::PARTS][S::MT][4];
  float fs[S::REGIONS];
  uint32_t s[S::CF][S::GPC], z[S::CF][S::GPC];
};

// Column of X (from the chunk's first) of a lane's piece m of 8, as the weights' loads have it.
template <bool FP8>
__device__ __forceinline__ int piece_col(int m, int quarter) {
  return FP8 ? (m >> 1) * 64 + quarter * 16 + (m & 1) * 8 : m * 32 + quarter * 8;
}

template <class S, bool TAIL>
__device__ __forceinline__ void load_chunk(Chunk<S>& c, const Sources<S>& src, int chunk) {
  const int quarter = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int r = 0; r < S::REGIONS; ++r) {
    if constexpr (S::FP8) c.fs[r] = *(const __attribute__((address_space(4))) float*)(src.fs[r] + chunk);
#pragma unroll
    for (int i = 0; i < S::PER; ++i) {
      const int cf = r * S::PER + i;
#pragma unroll
      for (int j = 0; j < S::WL; ++j) {
        int v = src.q_off + i * src.q_tile + (S::FP8 ? j * 64 + quarter * 16 : quarter * 16);
        if (S::FP8 && TAIL && chunk * 128 + j * 64 + quarter * 16 >= src.K) v = kOobOffset;
        c.w[cf][j] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(src.q[r], v, chunk * (S::FP8 ? 128 : 64), 0));
      }
      if constexpr (!S::FP8) {
        const int g = S::GPC == 1 ? chunk * 128 / src.group : chunk * S::GPC;
        const int sv = src.s_off + i * src.s_tile, zv = src.z_off + i * src.z_tile;
        if (S::GPC > 1 && src.wide) {
          if constexpr (S::GPC == 4) {
            const u32x2 t = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(src.s[r], sv, 2 * g, 0));
            c.s[cf][0] = t.x << 16; c.s[cf][1] = t.x & 0xffff0000u;
            c.s[cf][2] = t.y << 16; c.s[cf][3] = t.y & 0xffff0000u;
          } else if constexpr (S::GPC == 2) {
            const uint32_t t = __builtin_amdgcn_raw_buffer_load_b32(src.s[r], sv, 2 * g, 0);
            c.s[cf][0] = t << 16; c.s[cf][1] = t & 0xffff0000u;
          }
          if (src.has_z) {
            uint32_t t = 0;
            if constexpr (S::GPC == 4) t = __builtin_amdgcn_raw_buffer_load_b32(src.z[r], zv, g, 0);
            if constexpr (S::GPC == 2) t = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(src.z[r], zv, g, 0);
#pragma unroll
            for (int h = 0; h < S::GPC; ++h) c.z[cf][h] = (t >> (8 * h)) & 255u;
          }
        } else {
#pragma unroll
          for (int h = 0; h < S::GPC; ++h) {
            if (TAIL && h > 0 && chunk * 128 + h * (128 / S::GPC) >= src.K) continue;
            c.s[cf][h] = (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(src.s[r], sv, 2 * (g + h), 0) << 16;
            if (src.has_z) c.z[cf][h] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(src.z[r], zv, g + h, 0);
          }
        }
        if (!src.has_z) {
#pragma unroll
          for (int h = 0; h < S::GPC; ++h) c.z[cf][h] = 8;
        }
      }
    }
  }
#pragma unroll
  for (int p = 0; p < S::PARTS; ++p)
#pragma unroll
    for (int t = 0; t < S::MT; ++t)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int col = piece_col<S::FP8>(m, quarter);
        int v = src.x_off[t] + p * src.x_part + 2 * col;
        if (TAIL && chunk * 128 + col >= src.K) v = kOobOffset;
        c.x[p][t][m] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(src.x, v, chunk * 256, 0));
      }
}

// Eight weights as bf16: e4m3 bytes, or the eight codes of a 4-bit word.
__device__ __forceinline__ bf16x8 widen_fp8(int lo, int hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
__device__ __forceinline__ bf16x8 widen_int4(int w) {
  const int lo = w & 0x0f0f0f0f, hi = (int)((uint32_t)w >> 4) & 0x0f0f0f0f;
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.f, true);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

template <class S, bool TAIL>
__device__ __forceinline__ void add_chunk(f32x4 (&acc)[S::MT][S::CF], const Chunk<S>& c, const Sources<S>& src, int chunk) {
  if constexpr (S::FP8) {
#pragma unroll
    for (int cf = 0; cf < S::CF; ++cf) {
      f32x4 P[S::MT];
#pragma unroll
      for (int t = 0; t < S::MT; ++t) P[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const bf16x8 b = widen_fp8(c.w[cf][m >> 1][2 * (m & 1)], c.w[cf][m >> 1][2 * (m & 1) + 1]);
#pragma unroll
        for (int t = 0; t < S::MT; ++t)
#pragma unroll
          for (int p = 0; p < S::PARTS; ++p)
            P[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, c.x[p][t][m]), b, P[t], 0, 0, 0);
      }
      const float s = c.fs[cf / S::PER];
#pragma unroll
      for (int t = 0; t < S::MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][cf][i] = __builtin_fmaf(s, P[t][i], acc[t][cf][i]);
    }
  } else {
    constexpr int MPG = 4 / S::GPC;
    const __bf16 one = (__bf16)1.f;
    const bf16x8 ones = bf16x8{one, one, one, one, one, one, one, one};
#pragma unroll
    for (int g = 0; g < S::GPC; ++g) {
      if (TAIL && g > 0 && chunk * 128 + g * (128 / S::GPC) >= src.K) continue;  // groups past the row's last
      f32x4 sum[S::MT];
#pragma unroll
      for (int t = 0; t < S::MT; ++t) {
        sum[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = g * MPG; m < (g + 1) * MPG; ++m)
#pragma unroll
          for (int p = 0; p < S::PARTS; ++p)
            sum[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, c.x[p][t][m]), ones, sum[t], 0, 0, 0);
      }
#pragma unroll
      for (int cf = 0; cf < S::CF; ++cf) {
        f32x4 P[S::MT];
#pragma unroll
        for (int t = 0; t < S::MT; ++t) P[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = g * MPG; m < (g + 1) * MPG; ++m) {
          const bf16x8 b = widen_int4(c.w[cf][0][m]);
#pragma unroll
          for (int t = 0; t < S::MT; ++t)
#pragma unroll
            for (int p = 0; p < S::PARTS; ++p)
              P[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, c.x[p][t][m]), b, P[t], 0, 0, 0);
        }
        const float s = __uint_as_float(c.s[cf][g]), z = (float)c.z[cf][g];
#pragma unroll
        for (int t = 0; t < S::MT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[t][cf][i] = __builtin_fmaf(s, __builtin_fmaf(-z, sum[t][i], P[t][i]), acc[t][cf][i]);
      }
    }
  }
}

// acc += the products of chunks first, first + step, ... below `end`; the
// chunk that holds column K's group end, if partial, is chunk K / 128.
template <class S>
__device__ __forceinline__ void stream_chunks(f32x4 (&acc)[S::MT][S::CF], const Sources<S>& src, int first, int end,
                                              int step) {
  const int whole = min(end, src.K >> 7);  // chunks without a tail
  const int n = first < whole ? (whole - first + step - 1) / step : 0;
  Chunk<S> c[S::DEPTH];
#pragma unroll
  for (int d = 0; d < S::DEPTH; ++d)
    if (d < n) load_chunk<S, false>(c[d], src, first + d * step);
  int i = 0;
  for (; i + S::DEPTH <= n; i += S::DEPTH) {
#pragma unroll
    for (int d = 0; d < S::DEPTH; ++d) {
      add_chunk<S, false>(acc, c[d], src, first + (i + d) * step);
      if (i + d + S::DEPTH < n) load_chunk<S, false>(c[d], src, first + (i + d + S::DEPTH) * step);
    }
  }
#pragma unroll
  for (int d = 0; d < S::DEPTH; ++d)
    if (i + d < n) add_chunk<S, false>(acc, c[d], src, first + (i + d) * step);
  const int last = src.K >> 7;  // the partial chunk
  if ((src.K & 127) && last < end && last >= first && (last - first) % step == 0) {
    load_chunk<S, true>(c[0], src, last);
    add_chunk<S, true>(acc, c[0], src, last);
  }
}

}  // namespace fg
