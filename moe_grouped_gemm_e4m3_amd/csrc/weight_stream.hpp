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
// A wave streams chunks of 128 bytes of its weight rows (128 e4m3 or 256 4-bit
// columns) through an LDS ring that it alone uses, DEPTH - 1 of them in flight,
// with the same columns of X next to them.  fp32 rows of X are the sums of three
// bf16, made while the chunk before is multiplied.
//
// Weights loaded into registers in the matrix cores' layout (16 rows by 16 bytes)
// cost an access of the vector cache for every lane, 64 for 1 KiB, and that rate,
// about one a clock, bounded the 4-bit layers at 2.3 TB/s; whole rows of 128 bytes
// cost a quarter of them.
#pragma once

#include "decode_plan.hpp"
#include "linear_fewrow.hpp"

namespace fg {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Formats.  GPC: scale groups in 128 columns (4, 2 or 1 for groups of 32, 64 and
// any multiple of 128).  Z: with zero points (else 8).
struct Fp8Block {
  static constexpr bool FP8 = true, Z = false;
  static constexpr int GPC = 1;
};
template <int GPC_, bool Z_>
struct Int4Group {
  static constexpr bool FP8 = false, Z = Z_;
  static constexpr int GPC = GPC_;
};

// MT: row tiles of 16.  NX: KiB of X in a chunk (so X_ROWS rows are there).  CF:
// weight tiles of 16 rows, in REGIONS places of the matrix (2: gate and up
// rows).  ROWS32: 0, or rows of an fp32 X, which comes through registers (NX 0).
// RING: bytes of the ring.
// SHARE: waves that work on the same columns, with one copy of X, a ring and a
// barrier for each chunk; 1: a wave on its own.  SCALES: 4-bit groups of each
// weight row whose scales wait in LDS.
template <class Fmt_, int MT_, int NX_, int CF_, int REGIONS_, int ROWS32_, int RING_, int SHARE_ = 1, int SCALES_ = 32>
struct Stream {
  using Fmt = Fmt_;
  static constexpr int MT = MT_, NX = NX_, CF = CF_, REGIONS = REGIONS_;
  static constexpr bool WIDE_X = ROWS32_ > 0;
  static constexpr int PARTS = WIDE_X ? 3 : 1;       // bf16 matrices whose sum X is
  static constexpr bool FP8 = Fmt::FP8, Z = Fmt::Z;
  static constexpr int GPC = Fmt::GPC;
  static constexpr int PER = CF / REGIONS;           // weight tiles of a region
  static constexpr int HALVES = FP8 ? 1 : 2;         // pieces of 128 columns in a chunk
  static constexpr int COLS = 128 * HALVES;          // columns of a chunk
  static constexpr int X_PART = 2 * COLS;            // bytes of one row and part of X
  static constexpr int X_ROW = X_PART * PARTS;
  static constexpr int X_ROWS = WIDE_X ? ROWS32_ : NX * 1024 / X_ROW;
  static constexpr int SHARE = SHARE_;
  static constexpr int X_BYTES = X_ROWS * X_ROW;     // of all parts
  // WIDE_X: a lane loads and splits pieces of 8 columns, or where a wave has fewer than 64 of them, of 2 or 4
  static constexpr int LANE_COLS = WIDE_X ? X_ROWS / SHARE * COLS / 64 : 8;
  static constexpr int PIECE = LANE_COLS < 8 ? LANE_COLS : 8;
  static constexpr int SLOT = SHARE * CF * 2048 + NX * 1024;  // X, then every wave's weights
  static constexpr int X_LOADS = WIDE_X ? LANE_COLS / PIECE : NX > SHARE ? NX / SHARE : 1;  // of a wave: of 16 bytes, or pieces
  static constexpr int LOADS = CF * 2 + (WIDE_X ? 0 : X_LOADS);  // into LDS
  static constexpr int FIT = RING_ / SLOT, MOST = 63 / LOADS + 1;
  static constexpr int DEPTH = FIT < MOST ? FIT : MOST;
  static constexpr int SCALES = SCALES_;
  static constexpr int SCALE_LD = SCALES + 1;        // words; odd, so that rows lie in different banks
  static_assert(CF % REGIONS == 0 && DEPTH >= 2 && X_ROWS <= 16 * MT, "stream");
  static constexpr int X_REGS = WIDE_X ? X_LOADS * (PIECE == 8 ? 2 : 1) : 0;  // loads of a wave's pieces
  static_assert(WIDE_X ? NX == 0 && X_ROWS % SHARE == 0 && LANE_COLS >= 2 && X_LOADS * PIECE == LANE_COLS &&
                             (DEPTH - 1) * LOADS + X_REGS < 64
                       : (NX & (NX - 1)) == 0, "X");
};
// LDS bytes of a wave's scales.
template <class Fmt, int CF, int SCALES = 32>
constexpr int scale_lds() {
  return scale_bytes(Fmt::FP8, CF, SCALES);
}

// Where a wave's weights and activations are.
template <class S>
struct Sources {
  __amdgpu_buffer_rsrc_t q[S::REGIONS], s[S::REGIONS], z[S::REGIONS];
  const float* fs[S::CF];  // e4m3: the factors of every tile's block row
  int row_bytes, groups;   // of a weight row
  __amdgpu_buffer_rsrc_t x;
  int x_off[S::X_LOADS];   // this lane's row of X in every load, bytes
  int K;
  int group_chunks, group_shift;  // GPC 1: multiples of 128 in a group, and their logarithm (-1: no power of two)
};

template <class S>
__device__ __forceinline__ void set_group(Sources<S>& src, int group) {
  src.group_chunks = group >> 7;
  src.group_shift = (src.group_chunks & (src.group_chunks - 1)) ? -1 : 31 - __builtin_clz(src.group_chunks | 1);
}
// Scale group of the 128 columns `half` and part g of them.
template <class S>
__device__ __forceinline__ int group_of(const Sources<S>& src, int half, int g) {
  return S::GPC > 1 ? half * S::GPC + g : src.group_shift >= 0 ? half >> src.group_shift : half / src.group_chunks;
}

// A lane's place in load i of X: lanes are pieces of 16 bytes of rows.  A piece's place in its 8 is exchanged by the row, and so are
// two eights, and e4m3's even pieces stand before the odd ones: the 16 lanes that
// read at the same time then read from all 64 banks (4 bits, 64 x 7168 x 16384:
// LDS cycles 4.1 for 7.8 million, 35.4 us for 36.8).
// Load i of a wave is KiB x_kib_of(i) of X: the waves share them out (where
// there are fewer KiB than waves, some load the same).
template <class S>
__device__ __forceinline__ int x_kib_of(int i) {
  if (S::SHARE == 1) return i;
  return (__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * S::X_LOADS + i) & (S::NX - 1);
}
// fp32 rows are shared out whole, in pieces: the first column of lane's piece i
// among all of its wave's.
template <class S>
__device__ __forceinline__ int x_col_of(int i) {
  return (i * 64 + (int)(threadIdx.x & 63)) * S::PIECE;
}
template <class S>
__device__ __forceinline__ int x_first_row() {
  return S::SHARE == 1 ? 0 : (__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & (S::SHARE - 1)) * (S::X_ROWS / S::SHARE);
}
template <class S>
__device__ __forceinline__ int x_row_of(int i) {
  if (S::WIDE_X) return x_first_row<S>() + x_col_of<S>(i) / S::COLS;
  return (x_kib_of<S>(i) * 1024 + (threadIdx.x & 63) * 16) / S::X_ROW;
}

// This wave's weights in a slot.
template <class S>
__device__ __forceinline__ int weights_at() {
  return S::NX * 1024 + (S::SHARE == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * S::CF * 2048);
}

// Loads chunk c into a slot.  Past column K, and where it is not wanted, zeros,
// without touching memory (but counted as loads).  The scalar offset counts against the
// range's end and must not pass it: every range holds a row at least.
template <class S>
__device__ __forceinline__ void load_chunk(const Sources<S>& src, uint8_t* slot, int c, bool want) {
  typedef __attribute__((address_space(3))) void* Lds;
  const int lane = threadIdx.x & 63;
  const int r8 = lane >> 3, byte = ((lane & 7) ^ r8) * 16;
  const bool in = byte < (want ? (S::FP8 ? src.K : src.row_bytes) - c * 128 : 0);
  uint8_t* mine = slot + weights_at<S>();
#pragma unroll
  for (int t = 0; t < S::CF; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int v = ((t % S::PER) * 16 + h * 8 + r8) * src.row_bytes + byte;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(src.q[t / S::PER], (Lds)(mine + t * 2048 + h * 1024), 16,
                                               in ? v : kOobOffset, c * 128, 0, 0);
    }
  if (S::WIDE_X) return;
  const int cols_left = want ? src.K - c * S::COLS : 0;
#pragma unroll
  for (int i = 0; i < S::X_LOADS; ++i) {
    const int row = x_row_of<S>(i), at = ((lane * 16) & (S::X_PART - 1)) ^ ((row & 7) << 4) ^ ((row & 1) << 7);
    const int pos = (at >> 4) & 7, in8 = S::FP8 ? (pos & 3) << 1 | pos >> 2 : pos;
    const int col = ((at & ~127) + in8 * 16) >> 1;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src.x, (Lds)(slot + x_kib_of<S>(i) * 1024), 16,
                                             col < cols_left ? src.x_off[i] + 2 * col : kOobOffset,
                                             c * (2 * S::COLS), 0, 0);
  }
}

// This wave's LDS accesses are done.
__device__ __forceinline__ void wait_lds() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// A barrier of the workgroup, which no access of memory is moved across; it waits
// for none.
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// fp32 X of a chunk, on its way to LDS as bf16 parts.
template <class S>
struct XLoads {
  uint32_t v[S::X_LOADS][S::PIECE];

  // Chunk c; past column K, and where it is not wanted, zeros.
  __device__ __forceinline__ void load(const Sources<S>& src, int c, bool want) {
    const int cols_left = want ? src.K - c * S::COLS : 0, from = c * (4 * S::COLS);
#pragma unroll
    for (int i = 0; i < S::X_LOADS; ++i) {
      const int col = x_col_of<S>(i) % S::COLS, at = src.x_off[i] + 4 * col;
      if constexpr (S::PIECE == 2) {
        const auto w = __builtin_amdgcn_raw_buffer_load_b64(src.x, col < cols_left ? at : kOobOffset, from, 0);
#pragma unroll
        for (int j = 0; j < 2; ++j) v[i][j] = w[j];
      } else {
#pragma unroll
        for (int h = 0; h < S::PIECE / 4; ++h) {
          const auto w = __builtin_amdgcn_raw_buffer_load_b128(src.x, col < cols_left ? at + 16 * h : kOobOffset, from, 0);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][4 * h + j] = w[j];
        }
      }
    }
  }

  // To x: three bf16 whose sum is the number, exactly but for bits under 2^-126: its
  // upper 8 significant bits, the next 8, the rest.  What is left of an infinity is
  // finite and has its sign, so that its products are those of an infinity.
  __device__ __forceinline__ void store(uint8_t* x) const {
    typedef uint32_t Words __attribute__((ext_vector_type(S::PIECE / 2)));
#pragma unroll
    for (int i = 0; i < S::X_LOADS; ++i) {
      const int row = x_row_of<S>(i), col = x_col_of<S>(i) % S::COLS, eight = col >> 6, in = (col >> 3) & 7;
      const int pos = S::FP8 ? (in & 1) << 2 | in >> 1 : in;
      uint8_t* to = x + row * S::X_ROW + (eight >> 1) * 256 +
                    (((pos ^ (row & 7)) << 4) ^ ((row & 1) << 7) ^ ((eight & 1) << 7)) + 2 * (col & 7);
      float r[S::PIECE];
#pragma unroll
      for (int j = 0; j < S::PIECE; ++j) r[j] = __uint_as_float(v[i][j]);
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        Words w;
#pragma unroll
        for (int j = 0; j < S::PIECE / 2; ++j)
          w[j] = __builtin_amdgcn_perm(__float_as_uint(r[2 * j + 1]), __float_as_uint(r[2 * j]), 0x07060302u);
        *(Words*)(to + p * S::X_PART) = w;
        if (p == 2) break;
#pragma unroll
        for (int j = 0; j < S::PIECE; ++j) {
          if (p == 0) r[j] = __builtin_amdgcn_fmed3f(r[j], -__FLT_MAX__, __FLT_MAX__);
          r[j] -= __uint_as_float(__float_as_uint(r[j]) & 0xffff0000u);
        }
      }
    }
  }
};

// Scales and zero points of 16 groups from g on of the wave's rows, on their way
// to LDS: one word each, bf16 scale above, zero point below.  Groups from g_end
// on (of the last chunk, that the row does not have) get scales of zero: what
// stands behind a row's last scale may be anything, and 0 NaN is not 0.
template <class S>
struct ScaleLoads {
  uint32_t s[S::CF][2][2], z[S::CF][2][2];

  __device__ __forceinline__ void load(const Sources<S>& src, int g, int g_end) {
    const int lane = threadIdx.x & 63, r8 = lane >> 3;
#pragma unroll
    for (int t = 0; t < S::CF; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int x = min(g + 8 * y + (lane & 7), g_end - 1), row = (t % S::PER) * 16 + h * 8 + r8;
          const int at = row * src.groups + x;
          s[t][h][y] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(src.s[t / S::PER], 2 * at, 0, 0);
          if (S::Z) z[t][h][y] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(src.z[t / S::PER], at, 0, 0);
        }
  }
  // scales: of a row's group g
  __device__ __forceinline__ void store(uint32_t* scales, int g, int g_end) const {
    const int lane = threadIdx.x & 63, r8 = lane >> 3;
#pragma unroll
    for (int t = 0; t < S::CF; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          scales[(t * 16 + h * 8 + r8) * S::SCALE_LD + 8 * y + (lane & 7)] =
              g + 8 * y + (lane & 7) < g_end ? s[t][h][y] << 16 | (S::Z ? z[t][h][y] : 8u) : 0u;
  }
};

// Eight weights as bf16: e4m3 bytes, or the eight codes of a 4-bit word.
__device__ __forceinline__ bf16x8 widen_bytes(int lo, int hi, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
__device__ __forceinline__ bf16x8 widen_int4(int w) {
  return widen_bytes(w & 0x0f0f0f0f, (int)((uint32_t)w >> 4) & 0x0f0f0f0f, 512.f);
}

__device__ __forceinline__ f32x4 mfma_bf16(i32x4 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), b, c, 0, 0, 0);
}

// A lane's 8 columns of X for matrix product m of 128 columns `half` of a slot,
// in the order of its weights: e4m3, 16 bytes of each 64, 8 at a time; 4 bits,
// word m of piece `quarter`.  Pieces are exchanged inside groups of 8 and of two
// groups, so an address is one of a few lane constants and an immediate.
template <class S>
__device__ __forceinline__ i32x4 x_piece(const uint8_t* x, int t, int part, int half, int m) {
  const int lane = threadIdx.x & 63, quarter = lane >> 4;
  // rows past X's are never looked at again
  constexpr bool pow2 = (S::X_ROWS & (S::X_ROWS - 1)) == 0;
  const int row = pow2 ? (16 * t + (lane & 15)) & (S::X_ROWS - 1) : min(16 * t + (lane & 15), S::X_ROWS - 1);
  const int in8 = (m & 1) * 4 + quarter;
  const int eight = S::FP8 ? m >> 1 : half * 2 + (m >> 1);
  return *(const i32x4*)(x + (row * S::X_ROW + (((in8 ^ (row & 7)) << 4) ^ ((row & 1) << 7) ^ ((eight & 1) << 7))) +
                         part * S::X_PART + (eight >> 1) * 256);
}
// 16 bytes of a lane's weight row in tile t: piece 4 j + quarter of 8.
template <class S>
__device__ __forceinline__ i32x4 w_piece(const uint8_t* slot, int t, int j) {
  const int lane = threadIdx.x & 63, l16 = lane & 15;
  return *(const i32x4*)(slot + weights_at<S>() + (l16 * 128 + (((4 * j + (lane >> 4)) ^ (l16 & 7)) << 4)) + t * 2048);
}

// A lane's X for matrix products of 32 columns, one after the other (4 or 8 a
// chunk).  The parts of fp32 rows are asked for a product ahead, which the
// compiler does not do by itself, and a read of LDS takes as long as several
// products (the layer above: 171 us for 162).
template <class S>
struct XPieces {
  const uint8_t* xs;
  i32x4 x[2][S::PARTS][S::MT];

  __device__ __forceinline__ void load(int step) {
    if (S::WIDE_X && step < 4 * S::HALVES)
#pragma unroll
      for (int p = 0; p < S::PARTS; ++p)
#pragma unroll
        for (int t = 0; t < S::MT; ++t) x[step & 1][p][t] = x_piece<S>(xs, t, p, step >> 2, step & 3);
  }
  // Before the products of a step.
  __device__ __forceinline__ void next(int step) {
    load(step + 1);
    if (S::WIDE_X) __builtin_amdgcn_sched_barrier(0);
  }
  __device__ __forceinline__ i32x4 at(int step, int p, int t) const {
    return S::WIDE_X ? x[step & 1][p][t] : x_piece<S>(xs, t, p, step >> 2, step & 3);
  }
};

// acc += the slot's products.  Products that follow each other are of different
// tiles, and a group's sums are scaled while the matrix cores work on the next
// group's: with a wave or two on a SIMD, what waits for a result is not hidden
// by other waves.
template <class S>
__device__ __forceinline__ void add_chunk(f32x4 (&acc)[S::MT][S::CF], const Sources<S>& src, const uint8_t* slot,
                                          const uint8_t* xs, const float (&fs)[S::CF], const uint32_t* scales, int chunk,
                                          int g0) {
  const f32x4 zero = f32x4{0.f, 0.f, 0.f, 0.f};
  XPieces<S> pieces;
  pieces.xs = xs;
  pieces.load(0);
  if constexpr (S::FP8) {
    f32x4 P[S::MT][S::CF];
#pragma unroll
    for (int t = 0; t < S::MT; ++t)
#pragma unroll
      for (int cf = 0; cf < S::CF; ++cf) P[t][cf] = zero;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      i32x4 w[S::CF];
#pragma unroll
      for (int cf = 0; cf < S::CF; ++cf) w[cf] = w_piece<S>(slot, cf, j);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int step = 2 * j + h;
        pieces.next(step);
        bf16x8 b[S::CF];
#pragma unroll
        for (int cf = 0; cf < S::CF; ++cf) b[cf] = widen_bytes(w[cf][2 * h], w[cf][2 * h + 1], 1.f);
#pragma unroll
        for (int p = 0; p < S::PARTS; ++p)
#pragma unroll
          for (int t = 0; t < S::MT; ++t) {
            const i32x4 x = pieces.at(step, p, t);
#pragma unroll
            for (int cf = 0; cf < S::CF; ++cf) P[t][cf] = mfma_bf16(x, b[cf], P[t][cf]);
          }
      }
    }
#pragma unroll
    for (int t = 0; t < S::MT; ++t)
#pragma unroll
      for (int cf = 0; cf < S::CF; ++cf)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][cf][i] = __builtin_fmaf(fs[cf], P[t][cf][i], acc[t][cf][i]);
  } else {
    constexpr int MPG = 4 / S::GPC, GROUPS = 2 * S::GPC;
    const __bf16 one = (__bf16)1.f;
    const bf16x8 ones = bf16x8{one, one, one, one, one, one, one, one};
    const int l16 = threadIdx.x & 15;
    f32x4 sum[2][S::MT], P[2][S::MT][S::CF];
    uint32_t sz[2][S::CF];
    i32x4 w[S::CF];
#pragma unroll
    for (int g = 0; g <= GROUPS; ++g) {
      const int now = g & 1, last = 1 - now;
      if (g < GROUPS) {
        const int half = g / S::GPC, in = g % S::GPC;
        if (in == 0) {
#pragma unroll
          for (int cf = 0; cf < S::CF; ++cf) w[cf] = w_piece<S>(slot, cf, half);
        }
        const int at = group_of(src, chunk * 2 + half, in) - g0;
#pragma unroll
        for (int cf = 0; cf < S::CF; ++cf) {
          sz[now][cf] = scales[(cf * 16 + l16) * S::SCALE_LD + at];
#pragma unroll
          for (int t = 0; t < S::MT; ++t) P[now][t][cf] = zero;
        }
#pragma unroll
        for (int t = 0; t < S::MT; ++t) sum[now][t] = zero;
#pragma unroll
        for (int m = in * MPG; m < (in + 1) * MPG; ++m) {
          const int step = 4 * half + m;
          pieces.next(step);
          bf16x8 b[S::CF];
#pragma unroll
          for (int cf = 0; cf < S::CF; ++cf) b[cf] = widen_int4(w[cf][m]);
#pragma unroll
          for (int p = 0; p < S::PARTS; ++p)
#pragma unroll
            for (int t = 0; t < S::MT; ++t) {
              const i32x4 x = pieces.at(step, p, t);
              sum[now][t] = mfma_bf16(x, ones, sum[now][t]);
#pragma unroll
              for (int cf = 0; cf < S::CF; ++cf) P[now][t][cf] = mfma_bf16(x, b[cf], P[now][t][cf]);
            }
        }
      }
      if (g > 0) {
#pragma unroll
        for (int cf = 0; cf < S::CF; ++cf) {
          const float s = __uint_as_float(sz[last][cf] & 0xffff0000u), z = S::Z ? (float)(uint8_t)sz[last][cf] : 8.f;
#pragma unroll
          for (int t = 0; t < S::MT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[t][cf][i] = __builtin_fmaf(s, __builtin_fmaf(-z, sum[last][t][i], P[last][t][cf][i]), acc[t][cf][i]);
        }
      }
    }
  }
}

// The fp32 X of stream_chunks, by SHARE further waves, so that every SIMD has a
// wave that multiplies and one that splits: one barrier a chunk, behind which the
// chunk's parts are there and the place of the chunk before is free.  (Beside the
// products, in the one wave of a SIMD, all of the splitting shows: 64 tokens, 8 of
// 16 e4m3 experts of 2048 x 7168, half of the places, 188 us for 171.)
template <class S>
__device__ __forceinline__ void split_chunks(const Sources<S>& src, uint8_t* x, int first, int end, unsigned turn) {
  if (first >= end) return;
  const int n = end - first;
  int c = first + (int)(turn % (unsigned)n);
  auto next_of = [&](int x) { return x + 1 == end ? first : x + 1; };
  XLoads<S> now, next;
  now.load(src, c, true);
  c = next_of(c);
  next.load(src, c, 1 < n);
  now.store(x);
#pragma unroll 1
  for (int i = 1; i <= n; ++i) {
    wait_lds();
    meet();
    if (i == n) break;
    next.store(x + (i & 1 ? S::X_BYTES : 0));
    c = next_of(c);
    next.load(src, c, i + 1 < n);
  }
  wait_loads<0>();
  meet();
}

// acc += the products of chunks [first, end), from the `turn`-th on and around.
// ring: this wave's LDS, or the sharing waves' (which all call with the same
// chunks).  x: WIDE_X: X_BYTES, which this wave fills; where waves share, two times
// as many, which others fill (split_chunks, called with the same chunks).  No load
// is outstanding when it returns.
//
// The turn is the tile's, so that tiles which run side by side read different
// columns: rows a power of two of bytes apart have the same columns in the same
// memory channels.
template <class S>
__device__ __forceinline__ void stream_chunks(f32x4 (&acc)[S::MT][S::CF], const Sources<S>& src, uint8_t* ring, uint8_t* x,
                                              uint32_t* scales, int first, int end, unsigned turn) {
  if (first >= end) return;
  constexpr bool SPLIT = S::WIDE_X && S::SHARE == 1;  // of X, here
  int ahead = first + (int)(turn % (unsigned)(end - first));  // the next chunk to load
  int c = ahead;
  auto next_of = [&](int x) { return x + 1 == end ? first : x + 1; };
  const int n = end - first;
  // 4 bits: scales of groups [g0, g0 + SCALES) wait in LDS.  The first 16 are on
  // their way before the ring's loads, which waits for them would include.
  int g0 = 0, g_all = 0, g_last = 0;
  if constexpr (!S::FP8) {
    g_last = group_of(src, 2 * end - 1, S::GPC - 1);  // of the last chunk, whether the row has it or not
    const int g_first = group_of(src, 2 * first, 0);
    g0 = g_last - g_first < S::SCALES ? g_first : group_of(src, 2 * c, 0);
    g_all = min(src.groups, g_last + 1);
  }
  typename std::conditional<S::FP8, int, ScaleLoads<S>>::type loads;
  if constexpr (!S::FP8) loads.load(src, g0, g_all);
  // the first chunk's X, and the second's, which stays in registers for a turn
  typename std::conditional<SPLIT, XLoads<S>, int>::type x_first, x_next;
  if constexpr (SPLIT) {
    x_first.load(src, c, true);
    x_next.load(src, next_of(c), 1 < n);
  }
#pragma unroll
  for (int d = 0; d < S::DEPTH - 1; ++d) {
    load_chunk<S>(src, ring + d * S::SLOT, ahead, d < n);
    ahead = next_of(ahead);
  }
  typedef const __attribute__((address_space(4))) float* Scalar;
  int slot = 0;
  auto load_scales = [&](bool first_are_here) {
    if constexpr (!S::FP8) {
      const int all = min(S::SCALES, g_last + 1 - g0);
      for (int g = 0; g < all; g += 16) {
        if (g > 0 || !first_are_here) loads.load(src, g0 + g, g_all);
        loads.store(scales + g, g0 + g, g_all);
      }
    }
  };
  load_scales(true);
  if constexpr (SPLIT) {
    x_first.store(x);
    wait_lds();
  }
  float next[S::CF];
  if constexpr (S::FP8) {
#pragma unroll
    for (int t = 0; t < S::CF; ++t) next[t] = *(Scalar)(src.fs[t] + c);
  }
  int i = 0;
  auto chunk = [&](bool last) __attribute__((always_inline)) {
    float fs[S::CF];
    if constexpr (S::FP8) {
#pragma unroll
      for (int t = 0; t < S::CF; ++t) {
        fs[t] = next[t];
        next[t] = *(Scalar)(src.fs[t] + next_of(c));
      }
    } else {
      const int lo = group_of(src, 2 * c, 0);
      if (lo < g0 || group_of(src, 2 * c + 1, S::GPC - 1) >= g0 + S::SCALES) {
        // the next groups' scales: the ring fills meanwhile
        g0 = lo;
        load_scales(false);
      }
    }
    const int into = slot == 0 ? S::DEPTH - 1 : slot - 1;  // the slot read in the last turn
    if constexpr (S::SHARE > 1) {
      // every wave's loads of this chunk are done, and its reads of the last
      wait_loads<(S::DEPTH - 2) * S::LOADS>();
      meet();
    }
    load_chunk<S>(src, ring + into * S::SLOT, ahead, i + S::DEPTH - 1 < n);
    ahead = next_of(ahead);
    if constexpr (S::SHARE == 1) {
      // from the second turn on, the X asked for in the last may be outstanding too
      if (!SPLIT || i == 0)
        wait_loads<(S::DEPTH - 1) * S::LOADS>();
      else
        wait_loads<(S::DEPTH - 1) * S::LOADS + S::X_REGS>();
    }
    const uint8_t* here = ring + slot * S::SLOT;
    add_chunk<S>(acc, src, here, !S::WIDE_X ? here : SPLIT || (i & 1) == 0 ? x : x + S::X_BYTES, fs, scales, c, g0);
    c = next_of(c);
    if constexpr (SPLIT) {
      if (!last) {
        // behind the products that read what it takes the place of: a wave's LDS accesses keep their order
        x_next.store(x);
        x_next.load(src, next_of(c), i + 2 < n);
      }
    }
    // the slot is loaded again in the next turn: its reads are done
    wait_lds();
    slot = slot == S::DEPTH - 1 ? 0 : slot + 1;
  };
  if constexpr (SPLIT) {
#pragma unroll 1
    for (; i < n - 1; ++i) chunk(false);
    chunk(true);
  } else {
#pragma unroll 1
    for (; i < n; ++i) chunk(false);
  }
  wait_loads<0>();
  if constexpr (S::SHARE > 1) {
    meet();
  }
}

// D = bf16(sums of parts, added in their order); partial: [parts][M][N].
static __global__ __launch_bounds__(256) void join_parts_kernel(const float* partial, int parts, uint16_t* D, int64_t ldd,
                                                                int M, int N) {
  const int64_t all = (int64_t)M * N, step = (int64_t)gridDim.x * 1024;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < all; i += step) {
    const int64_t m = i / N;
    const int n = (int)(i - m * N);
    if (n + 4 <= N) {
      f32x4 v = *(const f32x4_at4*)(partial + i);
#pragma unroll 8
      for (int s = 1; s < parts; ++s) v += *(const f32x4_at4*)(partial + s * all + i);
      *(u32x2_at2*)(D + m * ldd + n) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    } else {
      for (int64_t j = i; j < i + 4 && j < all; ++j) {
        float v = partial[j];
        for (int s = 1; s < parts; ++s) v += partial[s * all + j];
        D[j / N * ldd + j % N] = bf16_bits(v);
      }
    }
  }
}

}  // namespace fg
