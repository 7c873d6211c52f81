// linear_tile.hpp -- the large-tile kernel of the 8-bit-integer and bf16
// products (operations and epilogues: linear_kernel.hpp).
//
// Times in this file and in linear_plan.hpp are of one call among others in a
// HIP graph, on operands that stay the same (other operands in every call and
// kernel traces: up to 10 % more).
//
// A slice of a 256 x 256 tile is 2048 MFMA cycles for 64 KiB of loads; the
// chip's power limits the tiles of 256 rows (2.0 GHz): int8 4096 x 7168 x 16384
// on 256 x 224 tiles 345 us, 2790 TOP/s; gated bf16 4096 x 2048 x 7168 on 256 x
// 256 164 us, 1460 TFLOP/s; dX and dW at 4096 x 7168 x 4096 on 256 x 224 199
// and 203 us in a trace, 1210 and 1190 TFLOP/s, their transposing fragment
// reads twice as many.  Smaller tiles take two to three times their MFMAs' time
// for a slice: its loads and LDS reads and the barrier (128 x 128: 62 GB/s of
// loads a CU).  K-major rows that do not lie a multiple of 128 bytes apart cost
// up to 30 % more (half a line off: 4 to 16 %): a slice of such a row takes
// parts of two cache lines.
#pragma once

#include "linear_kernel.hpp"

namespace fg {

// A BM x BN output tile (gated: BN / 2 hidden units, gate and up columns) per
// workgroup of KG groups of WAVES_M x WAVES_N waves.  A slice is 128 bytes of
// the reduction: 64 bf16 or 128 int8.  The main loop takes KG slices a step,
// one for each group; the groups' sums are added at the end of a tile.
template <int E_, int BM_, int BN_, int WAVES_M_, int WAVES_N_, int KG_, int STAGES_, bool TA_ = false,
          bool TB_ = false>
struct LinearTile {
  static constexpr int E = E_, BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
  static constexpr int KG = KG_, STAGES = STAGES_;  // slices of a step, steps in LDS
  static constexpr bool TA = TA_, TB = TB_;
  static constexpr bool INT8 = epi_int8(E), GATED = epi_gated(E);
  static constexpr int ES = INT8 ? 1 : 2;
  static constexpr int GW = WAVES_M * WAVES_N, NW = GW * KG, THREADS = NW * 64;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, SM = WM / 16, SN = WN / 16;
  // B rows of a stage: BN rounded up to whole loads of every wave (MN-major:
  // to a power of two); what lies past BN loads as zeros without touching
  // memory and is not read
  static constexpr int BROWS = TB ? (BN > 128 ? 256 : BN) : (BN + 8 * GW - 1) / (8 * GW) * (8 * GW);
  // a stage: for each slice its A rows, then its B rows
  static constexpr int A_BYTES = BM * 128, SLICE = (BM + BROWS) * 128, STAGE = KG * SLICE;
  static constexpr int SUMS = (KG - 1) * BM * BN * 4;  // the further groups' accumulators
  static constexpr int LDS_BYTES = STAGES * STAGE + SUMS;
  static constexpr int LA = BM / 8 / GW, LB = BROWS / 8 / GW;  // 1 KiB loads per wave and step
  static constexpr int OUT_N = GATED ? BN / 2 : BN;         // output columns of a tile
  // two workgroups share a CU where LDS and registers allow it
  static constexpr int OCC = 2 * LDS_BYTES <= 160 * 1024 ? 2 : 1;
  static_assert(BM % (8 * GW) == 0 && BROWS % (8 * GW) == 0, "loads");
  static_assert(LDS_BYTES <= 160 * 1024 && STAGES >= 2 && (STAGES - 1) * (LA + LB) < 64, "stages");
  static_assert(WM % 16 == 0 && WN % 16 == 0 && BN % WAVES_N == 0, "wave tile");
  static_assert(!GATED || SN % 2 == 0, "gate and up blocks come in pairs");
  static_assert(!INT8 || (!TA && !TB), "bytes are staged K-major");
};

// One output tile: its place, and its slices of the reduction.
struct LinearWork {
  int w;  // tile id, < 0: none
  int m0, n0;
  int kb0, kb1;
};

template <class C>
__device__ __forceinline__ LinearWork linear_work(const LinearParams& p, int w) {
  LinearWork t;
  t.w = -1;
  t.m0 = t.n0 = t.kb0 = 0;
  t.kb1 = p.nk;
  if (w < p.num_tiles) {
    t.w = w;
    if (epi_partial(C::E)) {  // every tile of one split, then the next split's
      const int tiles = p.tiles_m * p.tiles_n, split = w / tiles;
      w -= split * tiles;
      t.kb0 = split * p.split_nk;
      t.kb1 = min(p.nk, t.kb0 + p.split_nk);
    }
    int tm, tn;
    raster(w, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    t.m0 = tm * C::BM;
    t.n0 = tn * C::OUT_N;
  }
  return t;
}

// 16-byte chunk swizzle of MN-major stage rows (one row per reduction index,
// CH chunks of 8 columns): a transposing fragment read takes, for each half of
// the wave, rows 8 q + j (j < 4, two q) at one pair of chunks.  Moving the pair
// by j and q lays those eight 32-byte pieces in different banks; a row of 8
// chunks is half the banks, so its own parity already parts neighbours.
template <int CH>
__device__ __forceinline__ int mn_swz(int r) {
  if (CH == 8) return (r & 2) | ((r >> 1) & 4);
  return (((r & 3) | ((r >> 1) & 12)) << 1) & (CH - 1);
}

// 16-byte chunk swizzle of K-major stage rows.  A 128-bit LDS read is served
// 16 lanes at a time, lanes 0-3, 12-15, 20-23 and 24-27 together: with the
// row's low 3 bits those lanes' chunks lie in 16 different bank groups
// (measured: no conflicts; an XOR with bit 3 as well has two on every read).
__device__ __forceinline__ int lin_swz(int row) {
  return row & 7;
}

// The loads of one operand's slices into the LDS stages: 1 KiB each, straight
// into LDS, shared out over the waves.
template <class C, bool IS_A>
struct Loader {
  static constexpr bool MN = IS_A ? C::TA : C::TB;
  static constexpr bool PAIRED = !IS_A && C::GATED;  // gate and up rows
  static constexpr int N = IS_A ? C::LA : C::LB;     // loads per wave
  static constexpr int ROWS = IS_A ? C::BM : C::BN, COLS = IS_A ? C::BM : C::BROWS;
  // the ranges read (K-major: the tile's rows; MN-major: each slice's
  // reduction rows)
  __amdgpu_buffer_rsrc_t rs[MN ? C::KG : 1];
  const uint8_t *gate, *up;  // gated: the tile's gate and up rows
  int bytes;
  int cols;   // rows (MN-major: columns) of the operand from the tile's first on
  bool empty; // nothing to read: every offset is out of range
  const uint8_t* from;  // MN-major: the operand at the tile's first column
  const uint8_t* at;    // MN-major: the first slice's first row

  static __device__ __forceinline__ int64_t ld(const LinearParams& p) { return IS_A ? p.lda : p.ldb; }

  // The ranges of tile t.
  __device__ __forceinline__ void tile(const LinearParams& p, const LinearWork& t) {
    const uint8_t* base = IS_A ? p.A : p.B;
    const int first = IS_A ? t.m0 : t.n0;
    cols = (IS_A ? p.M : p.N) - first;
    // no tile, or one of a gradient pair's padding columns alone
    empty = t.w < 0 || cols <= 0;
    if constexpr (MN) {
      from = empty ? base : base + (int64_t)first * 2;
    } else {
      bytes = empty ? 0 : (int)min((int64_t)(cols - 1) * ld(p) + p.K * C::ES, (int64_t)0x7fffffff);
      gate = base + (int64_t)first * ld(p);
      if (PAIRED)
        up = base + (int64_t)(p.N + first) * ld(p);
      else
        rs[0] = rows(gate, bytes);
    }
  }
  // MN-major: the rows of the step at slice kb; of W they are the hidden units
  // of one half of the gradient pair.  Returns how many steps from this one on
  // are whole slices of rows that follow each other.
  __device__ __forceinline__ int slices(const LinearParams& p, int kb) {
    int whole = 0;
    const int pitch = (int)ld(p);  // at most 4 MiB
#pragma unroll
    for (int g = C::KG - 1; g >= 0; --g) {
      int row = (kb + g) * 64, left = p.K - row;
      if (!IS_A && !C::TA && p.F > 0) {
        const bool up = row >= p.half;
        left = up ? p.F + p.half - row : p.F - row;
        row = up ? row - p.half + p.F : row;
      }
      const bool none = empty || left <= 0;
      at = from + (none ? 0 : (int64_t)row * pitch);
      rs[g] = rows(at, none ? 0 : (min(left, 64) - 1) * pitch + cols * 2);
      whole = left / (64 * C::KG);
    }
    return empty ? 1 : whole;
  }
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(const uint8_t* first, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(first), (short)0, bytes, 0x00020000);
  }
  // MN-major: the next step's slices, where they are whole and follow.
  __device__ __forceinline__ void next(const LinearParams& p) {
    if constexpr (MN) {
      at += ld(p) * (64 * C::KG);
#pragma unroll
      for (int g = 0; g < C::KG; ++g) rs[g] = rows(at + ld(p) * (64 * g), (int)ld(p) * 63 + cols * 2);
    }
  }
  // Load j of this wave's N of the step at slice kb, into its stage.
  __device__ __forceinline__ void issue(const LinearParams& p, uint8_t* stage, int kb, int j, int wave, int lane) const {
    constexpr int PIECES = COLS / 8;  // 1 KiB pieces of a slice
    const int g = C::KG == 1 ? 0 : (wave * N + j) / PIECES, q = wave * N + j - g * PIECES;
    __amdgpu_buffer_rsrc_t r;
    int v, k = 0;
    if constexpr (MN) {  // whole stage rows of COLS columns
      r = C::KG > 1 && g == 1 ? rs[C::KG - 1] : rs[0];
      constexpr int CH = COLS / 8;  // chunks per row
      const int row = q * (64 / CH) + lane / CH;
      const int c = (lane % CH) ^ mn_swz<CH>(row);
      v = c * 8 < cols && (ROWS == COLS || c * 8 < ROWS) ? row * (int)ld(p) + c * 16 : kOobOffset;
    } else {  // 8 stage rows of 128 bytes
      int row = q * 8;
      if constexpr (PAIRED) {  // stage rows: 16 gate rows, 16 up rows of the same hidden units, ...
        row = (q >> 2) * 16 + (q & 1) * 8;
        r = rows((q >> 1) & 1 ? up : gate, bytes);
      } else {
        r = rs[0];
      }
      const int r8 = lane >> 3, c = ((lane & 7) ^ lin_swz(r8)) * 16;
      const int slice = kb + g;
      v = ROWS == COLS || q * 8 < ROWS ? k_clip((row + r8) * (int)ld(p) + c, slice * 128 + c, p.K * C::ES) : kOobOffset;
      // the scalar offset counts against the range's end and must not pass
      // it: 0 where nothing is read
      k = empty || (C::KG > 1 && slice >= p.nk) ? 0 : slice * 128;
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, (__attribute__((address_space(3))) void*)(stage + g * C::SLICE + q * 1024), 16, v, k, 0, 0);
  }
};

// Both operands' loads, step after step and tile after tile.  Past the
// workgroup's last tile they load zeros and touch no memory: every step issues
// the same number of loads, which the main loop's waits count on.
template <class C>
struct Loads {
  LinearWork t;
  int kb;   // first slice of the step in tile t
  int dst;  // LDS offset of its stage
  int run;  // steps until the ranges have to be worked out anew
  Loader<C, true> a;
  Loader<C, false> b;

  __device__ __forceinline__ Loads(const LinearParams& p, const LinearWork& first) : t(first), kb(first.kb0), dst(0) {
    a.tile(p, t);
    b.tile(p, t);
    slices(p);
  }
  __device__ __forceinline__ void slices(const LinearParams& p) {
    run = C::KG == 1 ? t.kb1 - kb : (t.kb1 - kb + C::KG - 1) / C::KG;
    if (C::TA) run = min(run, a.slices(p, kb));
    if (C::TB) run = min(run, b.slices(p, kb));
    run = max(run, 1);
  }
  __device__ __forceinline__ void advance(const LinearParams& p, int grid) {
    dst = dst == (C::STAGES - 1) * C::STAGE ? 0 : dst + C::STAGE;
    kb += C::KG;
    a.next(p);
    b.next(p);
    // out of line: the main loop's straight path has no other branch
    if (__builtin_expect(--run == 0, 0)) {
      if (kb >= t.kb1) {
        if (t.w >= 0) t = linear_work<C>(p, t.w + grid);
        kb = t.kb0;
        a.tile(p, t);
        b.tile(p, t);
      }
      slices(p);
    }
  }
};

// Fragments of half h (64 bytes of the reduction) of a slice: lane l holds
// row l % 16, bytes [16 (l / 16), +16) of the half.
template <int COLS, bool MN, int N>
struct FragReader {
  int off;   // K-major: byte offset of the first fragment's chunk for half 0
  int row0;  // MN-major: first column block of the wave
  __device__ __forceinline__ FragReader(int first_row, int lane) {
    const int l16 = lane & 15, q = lane >> 4;
    if (MN) {
      // lane i of group q reads reduction rows 8 q + i / 4 (and 4 further),
      // columns 4 (i % 4) .. +3 of the block; the transposing read hands it
      // column i of the four rows
      off = (8 * q + (l16 >> 2)) * COLS * 2 + (l16 & 1) * 8;
      row0 = (first_row >> 4) * 2 + ((l16 >> 1) & 1);
    } else {
      const int r = first_row + l16;
      off = r * 128 + ((q ^ lin_swz(r)) << 4);
      row0 = 0;
    }
  }
  // Fragment i of half h of the slice in stage st.
  __device__ __forceinline__ void read(const uint8_t* st, int h, int lane, int i, i32x4 (&f)[N]) const {
    if constexpr (MN) {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef short s16x8 __attribute__((ext_vector_type(8)));
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const int r = 8 * (lane >> 4) + ((lane & 15) >> 2);  // row within the half
      const int chunk = ((row0 + 2 * i) ^ mn_swz<COLS / 8>(r)) << 4;
      const uint8_t* a = st + off + h * 32 * COLS * 2 + chunk;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)a);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a + 4 * COLS * 2));
      f[i] = __builtin_bit_cast(i32x4, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      f[i] = *(const i32x4*)(st + (off ^ (h * 64)) + i * 2048);
    }
  }
};

template <class C>
struct LinearAcc {
  typedef typename std::conditional<C::INT8, i32x4, f32x4>::type V;
  V v[C::SM][C::SN];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < C::SM; ++i)
#pragma unroll
      for (int j = 0; j < C::SN; ++j) v[i][j] = V{0, 0, 0, 0};
  }
  // column block j with every row block
  __device__ __forceinline__ void mma(const i32x4 (&a)[C::SM], const i32x4 (&b)[C::SN], int j) {
#pragma unroll
      for (int i = 0; i < C::SM; ++i) {
        if constexpr (C::INT8)
          v[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[j], a[i], v[i][j], 0, 0, 0);
        else
          v[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b[j]),
                                                            __builtin_bit_cast(bf16x8, a[i]), v[i][j], 0, 0, 0);
      }
  }
};

// Four consecutive fp32 (zeros at and past column n_end).
__device__ __forceinline__ f32x4 load_f32x4(const float* src, int n, int n_end) {
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
  if (n + 4 <= n_end) {
    x = *(const f32x4_at4*)(src + n);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < n_end) x[r] = src[n + r];
  }
  return x;
}

// Columns of two neighbouring 16-column blocks of an output row (first column
// n0), four of each per lane: a0, a1 and b0, b1.  The lanes of quarters kq and
// kq ^ 1 trade halves, so that an even lane holds eight columns of the first
// block and an odd lane eight of the second: 16-byte stores.
template <bool FULL>
__device__ __forceinline__ void store_pair(uint16_t* row, int n0, int n_end, bool ok, int lane, uint32_t a0,
                                           uint32_t a1, uint32_t b0, uint32_t b1) {
  const int kq = lane >> 4;
  const auto x = __builtin_amdgcn_permlane16_swap(a0, b0, false, false);
  const auto y = __builtin_amdgcn_permlane16_swap(a1, b1, false, false);
  const i32x4 w = {(int)x[0], (int)y[0], (int)x[1], (int)y[1]};
  const int n = n0 + (kq & 1 ? 16 + 4 * (kq - 1) : 4 * kq);
  if (FULL || (ok && n + 8 <= n_end)) {
    *(i32x4_at2*)(row + n) = w;
  } else if (ok) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (n + e < n_end) row[n + e] = (uint16_t)((uint32_t)w[e >> 1] >> ((e & 1) * 16));
  }
}

// Columns [n, n + 4) of an output row.
template <bool FULL>
__device__ __forceinline__ void store_quad(uint16_t* row, int n, int n_end, bool ok, uint32_t a0, uint32_t a1) {
  if (FULL || (ok && n + 4 <= n_end)) {
    *(u32x2_at2*)(row + n) = u32x2{a0, a1};
  } else if (ok) {
    const uint32_t w[2] = {a0, a1};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < n_end) row[n + e] = (uint16_t)(w[e >> 1] >> ((e & 1) * 16));
  }
}

// The finished tile, straight from the accumulators.  Lane (l16, kq) holds
// row l16 and columns [4 kq, +4) of every 16 x 16 block.  FULL: the whole tile
// lies inside the output, so nothing is tested
// (gated with kept pre-activations, 4096 x 2048 x 7168: 192 us with the tests,
// 175 without).
template <class C, int ACT, bool FULL>
__device__ __forceinline__ void store_blocks(const LinearParams& p, const LinearWork& t, const LinearAcc<C>& acc,
                                             int wm, int wn, int lane) {
  const int l16 = lane & 15, kq = lane >> 4;
  constexpr bool GRAD = C::E == kEpiGatedGrad;
  constexpr int STEP = C::GATED ? 2 : 1;       // accumulator blocks per output block
  constexpr int NB = C::SN / STEP;             // output blocks of the wave
  const int nw = t.n0 + wn * NB * 16;          // the wave's first output column
  const int n_end = GRAD || C::E == kEpiGatedPartial ? p.half : p.N;
  f32x4 sb[C::INT8 ? C::SN : 1];
  if constexpr (C::INT8) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int n = nw + j * 16 + 4 * kq;
      sb[j * STEP] = load_f32x4(p.sb, n, p.N);
      if (C::GATED) sb[j * STEP + 1] = load_f32x4(p.sb + p.N, n, p.N);
    }
  }
  if constexpr (epi_partial(C::E)) {
    const int cols = C::GATED ? 2 * p.half : p.N;
    float* part = p.P + (int64_t)(t.kb0 / p.split_nk) * p.M * cols;
#pragma unroll
    for (int i = 0; i < C::SM; ++i) {
      const int m = t.m0 + wm * C::WM + i * 16 + l16;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int n = nw + j * 16 + 4 * kq;  // N is a multiple of 4
        float* dst = part + (int64_t)m * cols + n;
        if (FULL || (m < p.M && n < n_end)) {
          *(f32x4*)dst = __builtin_bit_cast(f32x4, acc.v[i][j * STEP]);
          if constexpr (C::GATED) *(f32x4*)(dst + p.half) = acc.v[i][j * STEP + 1];
        }
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < C::SM; ++i) {
    const int m = t.m0 + wm * C::WM + i * 16 + l16;
    bool ok = FULL || m < p.M;
    int64_t drow = m;
    if (C::TA && p.F > 0 && ok) {  // dW: rows of the gradient pair
      drow = pair_row(p, m);
      ok = FULL || drow >= 0;
    }
    uint16_t* row = p.D + drow * p.ldd;
    float sa = 0.f;
    if (C::INT8 && ok) sa = p.sa[m];
    // the wave's 16 rows of P (full tiles: all of them inside)
    __amdgpu_buffer_rsrc_t prs;
    if constexpr (C::E == kEpiGatedKeep && FULL)
      prs = make_rsrc(p.P + (int64_t)(t.m0 + wm * C::WM + i * 16) * p.ldp + nw, 0x7fffffff);
    uint32_t lo[NB], hi[NB], lo2[GRAD ? NB : 1], hi2[GRAD ? NB : 1];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int n = nw + j * 16 + 4 * kq;
      float a[4], b[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        a[r] = (float)acc.v[i][j * STEP][r];
        if (C::GATED) b[r] = (float)acc.v[i][j * STEP + STEP - 1][r];
        if constexpr (C::INT8) {
          a[r] = a[r] * sa * sb[j * STEP][r];
          if (C::GATED) b[r] = b[r] * sa * sb[j * STEP + STEP - 1][r];
        }
      }
      if constexpr (C::E == kEpiGatedKeep) {
        if constexpr (FULL) {
          const int at = l16 * (int)p.ldp * 4 + kq * 16;
          const i32x4 g = {__float_as_int(a[0]), __float_as_int(a[1]), __float_as_int(a[2]), __float_as_int(a[3])};
          const i32x4 u = {__float_as_int(b[0]), __float_as_int(b[1]), __float_as_int(b[2]), __float_as_int(b[3])};
          __builtin_amdgcn_raw_buffer_store_b128(g, prs, at, j * 64, 0);
          __builtin_amdgcn_raw_buffer_store_b128(u, prs, at, j * 64 + p.N * 4, 0);
        } else if (ok) {
          float* prow = p.P + (int64_t)m * p.ldp;
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n + r < p.N) {
              prow[n + r] = a[r];
              prow[p.N + n + r] = b[r];
            }
        }
      }
      if constexpr (GRAD) {
        uint32_t h[2] = {0, 0};
        if (ok) {
          const uint16_t* hrow = p.dH + (int64_t)m * p.lddh;
          if (FULL || n + 4 <= p.N) {
            const u32x2 u = *(const u32x2_at2*)(hrow + n);
            h[0] = u.x;
            h[1] = u.y;
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (n + r < p.N) h[r >> 1] |= (uint32_t)hrow[n + r] << (16 * (r & 1));
          }
        }
        float dg[4], du[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float dh = to_f32((uint16_t)(h[r >> 1] >> (16 * (r & 1))));
          gated_grad<ACT>(dh, a[r], b[r], dg[r], du[r]);
          if (!FULL && n + r >= p.N) dg[r] = du[r] = 0.f;
        }
        lo2[j] = pack_bf16x2(du[0], du[1]);
        hi2[j] = pack_bf16x2(du[2], du[3]);
#pragma unroll
        for (int r = 0; r < 4; ++r) a[r] = dg[r];
      } else if constexpr (C::GATED) {
#pragma unroll
        for (int r = 0; r < 4; ++r) a[r] = gated_value<ACT>(a[r], b[r]);
      }
      lo[j] = pack_bf16x2(a[0], a[1]);
      hi[j] = pack_bf16x2(a[2], a[3]);
      // one block at a time: interleaved, the blocks' temporaries do not fit
      // beside the accumulators and the next tile's fragments
      if (C::GATED) __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j + 1 < NB; j += 2) {
      store_pair<FULL>(row, nw + j * 16, n_end, ok, lane, lo[j], hi[j], lo[j + 1], hi[j + 1]);
      if constexpr (GRAD)
        store_pair<FULL>(row + p.half, nw + j * 16, n_end, ok, lane, lo2[j], hi2[j], lo2[j + 1], hi2[j + 1]);
    }
    if constexpr (NB % 2 == 1) {  // the last block alone: 8 bytes a lane
      store_quad<FULL>(row, nw + (NB - 1) * 16 + 4 * kq, n_end, ok, lo[NB - 1], hi[NB - 1]);
      if constexpr (GRAD)
        store_quad<FULL>(row + p.half, nw + (NB - 1) * 16 + 4 * kq, n_end, ok, lo2[NB - 1], hi2[NB - 1]);
    }
  }
}

// Stores a finished tile.
template <class C>
__device__ __forceinline__ void store_linear(const LinearParams& p, const LinearWork& t, const LinearAcc<C>& acc,
                                             int wm, int wn, int lane) {
  bool full = t.n0 + C::OUT_N <= p.N;
  if (C::TA && p.F > 0)
    full = full && (t.m0 >= p.half ? t.m0 - p.half : t.m0) + C::BM <= p.F;
  else
    full = full && t.m0 + C::BM <= p.M;
  if (C::E == kEpiGatedKeep) full = full && p.ldp <= 1 << 24;  // 32-bit offsets within 16 rows of P
  if constexpr (C::GATED && !epi_partial(C::E)) {
    if (p.act == kActSilu) {
      if (full)
        store_blocks<C, kActSilu, true>(p, t, acc, wm, wn, lane);
      else
        store_blocks<C, kActSilu, false>(p, t, acc, wm, wn, lane);
    } else {
      if (full)
        store_blocks<C, kActGeluTanh, true>(p, t, acc, wm, wn, lane);
      else
        store_blocks<C, kActGeluTanh, false>(p, t, acc, wm, wn, lane);
    }
  } else {
    if (full)
      store_blocks<C, 0, true>(p, t, acc, wm, wn, lane);
    else
      store_blocks<C, 0, false>(p, t, acc, wm, wn, lane);
  }
}

// Wait until this wave's LDS reads are done and at most N of its vector
// memory operations are outstanding (they complete in issue order), then meet
// the other waves.
template <int N>
__device__ __forceinline__ void linear_sync() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// One half of a slice: the MFMAs on fragments (a, b), and between them the
// reads of the next half's fragments (na, nb) from stages st_a and st_b and
// LOAD, the loads of a later slice into ld_a and ld_b, spread evenly: issued
// together they would fill the memory pipe's queue and hold up the MFMAs
// behind them.  No two of the four stages overlap here, and the compiler is
// told so: it would otherwise wait for the loads before it reads.
template <class C, int H, bool LOAD>
__device__ __forceinline__ void linear_half(const LinearParams& p, LinearAcc<C>& acc, const i32x4 (&a)[C::SM],
                                            const i32x4 (&b)[C::SN], i32x4 (&na)[C::SM], i32x4 (&nb)[C::SN],
                                            const FragReader<C::BM, C::TA, C::SM>& ra,
                                            const FragReader<C::BROWS, C::TB, C::SN>& rb, const uint8_t* __restrict st_a,
                                            const uint8_t* __restrict st_b, const Loads<C>& ld,
                                            uint8_t* __restrict ld_a, uint8_t* __restrict ld_b, int wave, int lane) {
  constexpr int READS = (C::SM + C::SN + C::SN - 1) / C::SN;
  constexpr int LOADS = C::LA + C::LB;
#pragma unroll
  for (int j = 0; j < C::SN; ++j) {
#pragma unroll
    for (int i = j * READS; i < (j + 1) * READS && i < C::SM + C::SN; ++i) {
      if (i < C::SM)
        ra.read(st_a, H, lane, i, na);
      else
        rb.read(st_b, H, lane, i - C::SM, nb);
    }
#pragma unroll
    for (int r = 0; r < LOADS; ++r) {
      if (!LOAD || r * C::SN / LOADS != j) continue;
      if (r < C::LB)
        ld.b.issue(p, ld_b, ld.kb, r, wave, lane);
      else
        ld.a.issue(p, ld_a, ld.kb, r - C::LB, wave, lane);
    }
    __builtin_amdgcn_sched_barrier(0);
    acc.mma(a, b, j);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// The reduction runs in 128-byte slices through STAGES LDS stages.  A slice's
// fragments are read in halves, each one half ahead of the MFMAs that use it,
// so no MFMA waits for an LDS read that was just issued; one barrier a slice
// lies between the two halves, where every wave has read all of the current
// stage and the next slice has landed.  The loads run STAGES slices ahead
// (into the workgroup's next tile too) and are issued in the half after the
// barrier that frees their stage.
//
// Workgroup `block` of `grid`, with C::LDS_BYTES at lds.
template <class C>
__device__ __forceinline__ void linear_tiles(const LinearParams& p, uint8_t* lds, int block, int grid) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = C::KG == 1 ? 0 : wave / C::GW, gwave = wave - group * C::GW;
  const int wm = gwave / C::WAVES_N, wn = gwave % C::WAVES_N;
  const int slice = group * C::SLICE;  // the group's slice in a stage

  LinearWork cur = linear_work<C>(p, xcd_local_id(block, grid));
  if (cur.w < 0) return;
  Loads<C> ld(p, cur);

  const FragReader<C::BM, C::TA, C::SM> ra(wm * C::WM, lane);
  const FragReader<C::BROWS, C::TB, C::SN> rb(wn * C::WN, lane);
  i32x4 a0[C::SM], b0[C::SN], a1[C::SM], b1[C::SN];
  LinearAcc<C> acc;
  acc.zero();

#pragma unroll 1
  for (int i = 0; i < C::STAGES; ++i) {
#pragma unroll
    for (int j = 0; j < C::LA; ++j) ld.a.issue(p, lds + ld.dst, ld.kb, j, wave, lane);
#pragma unroll
    for (int j = 0; j < C::LB; ++j) ld.b.issue(p, lds + C::A_BYTES + ld.dst, ld.kb, j, wave, lane);
    ld.advance(p, grid);
  }
  linear_sync<(C::STAGES - 1) * (C::LA + C::LB)>();
#pragma unroll
  for (int i = 0; i < C::SM; ++i) ra.read(lds + slice, 0, lane, i, a0);
#pragma unroll
  for (int i = 0; i < C::SN; ++i) rb.read(lds + slice + C::A_BYTES, 0, lane, i, b0);
  int s = slice;  // the group's slice of the current step
  while (cur.w >= 0) {
    for (int kb = cur.kb0; kb < cur.kb1; kb += C::KG) {
      linear_half<C, 1, false>(p, acc, a0, b0, a1, b1, ra, rb, lds + s, lds + C::A_BYTES + s, ld, nullptr, nullptr, wave,
                               lane);
      linear_sync<(C::STAGES - 2) * (C::LA + C::LB)>();
      s = s == slice + (C::STAGES - 1) * C::STAGE ? slice : s + C::STAGE;
      linear_half<C, 0, true>(p, acc, a1, b1, a0, b0, ra, rb, lds + s, lds + C::A_BYTES + s, ld, lds + ld.dst,
                              lds + C::A_BYTES + ld.dst, wave, lane);
      ld.advance(p, grid);
    }
    if constexpr (C::KG > 1) {
      // group 1's sums go through LDS; it writes them again only after the
      // barriers of another tile
      static_assert(C::KG == 2, "two groups");
      typedef typename LinearAcc<C>::V V;
      V* sums = (V*)(lds + C::STAGES * C::STAGE) + gwave * C::SM * C::SN * 64 + lane;
      if (group == 1) {
#pragma unroll
        for (int i = 0; i < C::SM; ++i)
#pragma unroll
          for (int j = 0; j < C::SN; ++j) sums[(i * C::SN + j) * 64] = acc.v[i][j];
      }
      lds_barrier();
      if (group == 0) {
#pragma unroll
        for (int i = 0; i < C::SM; ++i)
#pragma unroll
          for (int j = 0; j < C::SN; ++j) acc.v[i][j] += sums[(i * C::SN + j) * 64];
        store_linear<C>(p, cur, acc, wm, wn, lane);
      }
    } else {
      store_linear<C>(p, cur, acc, wm, wn, lane);
    }
    acc.zero();
    cur = linear_work<C>(p, cur.w + grid);
  }
  // no load may still be writing LDS when the workgroup ends
  __builtin_amdgcn_s_waitcnt(0);
}

template <class C>
__global__ __launch_bounds__(C::THREADS, C::OCC * C::NW / 4) void linear_tile_kernel(LinearParams p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::LDS_BYTES];
  linear_tiles<C>(p, lds, blockIdx.x, gridDim.x);
}

// dX and dW in one launch: the first `blocks_x` workgroups take dX's tiles,
// the others dW's.
template <class X, class W>
__global__ __launch_bounds__(X::THREADS, 2) void linear_grads_kernel(LinearParams px, LinearParams pw, int blocks_x) {
  static_assert(X::THREADS == W::THREADS && X::NW == 8, "one workgroup size, two waves a SIMD");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[X::LDS_BYTES > W::LDS_BYTES ? X::LDS_BYTES : W::LDS_BYTES];
  const int b = blockIdx.x;
  if (b < blocks_x)
    linear_tiles<X>(px, lds, b, blocks_x);
  else
    linear_tiles<W>(pw, lds, b - blocks_x, gridDim.x - blocks_x);
}

}  // namespace fg
