// linear_tile.hpp -- the large-tile kernel of the 8-bit-integer and bf16
// products (operations and epilogues: linear_kernel.hpp).
#pragma once

#include "linear_kernel.hpp"

namespace fg {

// A BM x BN output tile (gated: BN / 2 hidden units, gate and up columns) per
// workgroup of WAVES_M x WAVES_N waves.  A slice is 128 bytes of the
// reduction: 64 bf16 or 128 int8.
template <int E_, int BM_, int BN_, int WAVES_M_, int WAVES_N_, bool TA_ = false, bool TB_ = false>
struct LinearTile {
  static constexpr int E = E_, BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
  static constexpr bool TA = TA_, TB = TB_;
  static constexpr bool INT8 = epi_int8(E), GATED = epi_gated(E);
  static constexpr int ES = INT8 ? 1 : 2;
  static constexpr int NW = WAVES_M * WAVES_N, THREADS = NW * 64;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, SM = WM / 16, SN = WN / 16;
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr int LDS_BYTES = 2 * STAGE;
  static constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;  // 1 KiB loads per wave and slice
  static constexpr int OUT_N = GATED ? BN / 2 : BN;         // output columns of a tile
  // two workgroups share a CU where LDS and registers allow it
  static constexpr int OCC = 2 * LDS_BYTES <= 160 * 1024 ? 2 : 1;
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "loads");
  static_assert(SN % 2 == 0, "column blocks are stored in pairs");
  static_assert(!INT8 || (!TA && !TB), "bytes are staged K-major");
};

// One output tile: its place, and where its operands' first rows lie.
struct LinearWork {
  int w;  // tile id, < 0: none
  int m0, n0;
};

template <class C>
__device__ __forceinline__ LinearWork linear_work(const LinearParams& p, int w) {
  LinearWork t;
  t.w = -1;
  t.m0 = t.n0 = 0;
  if (w < p.num_tiles) {
    int tm, tn;
    raster(w, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    t.w = w;
    t.m0 = tm * C::BM;
    t.n0 = tn * C::OUT_N;
  }
  return t;
}

// 16-byte chunk swizzle of MN-major stage rows (one row per reduction index,
// CH chunks of 8 columns): a transposing fragment read takes, per group of 16
// lanes, 4 rows at one pair of chunks, and its four groups take rows 8 apart;
// moving the pair by (row % 4) + 4 (row / 8 % 4) spreads them over the banks.
template <int CH>
__device__ __forceinline__ int mn_swz(int r) {
  return (((r & 3) | ((r >> 1) & 12)) << 1) & (CH - 1);
}

// N loads of an operand stored K-major: 8 stage rows of 128 bytes each.
template <int N, bool CLIP>
__device__ __forceinline__ void issue_k_major(__amdgpu_buffer_rsrc_t rs, int64_t ld, int row0, int srow0, int k0,
                                              int kbytes, uint8_t* dst, int lane) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int r = 8 * j + (lane >> 3);
    const int c = (lane & 7) ^ swz16(srow0 + r);
    int v = (row0 + r) * (int)ld + c * 16;
    if (CLIP) v = k_clip(v, k0 + c * 16, kbytes);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(dst + j * 1024), 16, v, k0,
                                             0, 0);
  }
}

// N loads of an operand stored MN-major: 1 KiB of whole stage rows each.
template <int N, int COLS>
__device__ __forceinline__ void issue_mn_major(__amdgpu_buffer_rsrc_t rs, int64_t ld, int q0, int cols_left,
                                               uint8_t* dst, int lane) {
  constexpr int CH = COLS / 8, RPL = 64 / CH;  // chunks per row, rows per load
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int r = (q0 + j) * RPL + lane / CH;
    const int c = (lane % CH) ^ mn_swz<CH>(r);
    const int v = c * 8 < cols_left ? r * (int)ld + c * 16 : kOobOffset;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(dst + j * 1024), 16, v, 0,
                                             0, 0);
  }
}

// All loads of slice kb of tile t into `stage`, shared out over the waves.
template <class C>
__device__ __forceinline__ void issue_linear_slice(const LinearParams& p, const LinearWork& t, int kb, uint8_t* stage,
                                                   int wave, int lane) {
  const int kbytes = C::TA ? 0 : p.K * C::ES, k0 = kb * 128;
  const bool clip = k0 + 128 > kbytes;
  uint8_t* a_dst = stage + wave * C::LA * 1024;
  uint8_t* b_dst = stage + C::BM * 128 + wave * C::LB * 1024;
  if constexpr (C::TA) {
    const int left = p.K - kb * 64;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.A + (int64_t)kb * 64 * p.lda + (int64_t)t.m0 * 2,
                                                left > 0 ? (int64_t)(left - 1) * p.lda + (int64_t)(p.M - t.m0) * 2 : 0);
    issue_mn_major<C::LA, C::BM>(ra, p.lda, wave * C::LA, p.M - t.m0, a_dst, lane);
  } else {
    const __amdgpu_buffer_rsrc_t ra =
        make_rsrc(p.A + (int64_t)t.m0 * p.lda, (int64_t)(p.M - t.m0 - 1) * p.lda + kbytes);
    if (clip)
      issue_k_major<C::LA, true>(ra, p.lda, wave * C::LA * 8, wave * C::LA * 8, k0, kbytes, a_dst, lane);
    else
      issue_k_major<C::LA, false>(ra, p.lda, wave * C::LA * 8, wave * C::LA * 8, k0, kbytes, a_dst, lane);
  }
  if constexpr (C::TB) {
    // reduction rows of B: of W, hidden units of one half of the gradient
    // pair; otherwise B's own rows
    int64_t row = (int64_t)kb * 64;
    int left = p.K - kb * 64;
    if (!C::TA && p.F > 0) {
      const int h = row >= p.half ? 1 : 0;
      const int f = (int)row - h * p.half;
      row = (int64_t)h * p.F + f;
      left = p.F - f;
    }
    const __amdgpu_buffer_rsrc_t rb =
        make_rsrc(p.B + row * p.ldb + (int64_t)t.n0 * 2,
                  left > 0 ? (int64_t)(min(left, 64) - 1) * p.ldb + (int64_t)(p.N - t.n0) * 2 : 0);
    issue_mn_major<C::LB, C::BN>(rb, p.ldb, wave * C::LB, p.N - t.n0, b_dst, lane);
  } else if constexpr (C::GATED) {
    // stage rows: 16 gate rows, 16 up rows of the same hidden units, ...
    const int64_t bytes = (int64_t)(p.N - t.n0 - 1) * p.ldb + kbytes;
    const uint8_t* base = p.B + (int64_t)t.n0 * p.ldb;
    const __amdgpu_buffer_rsrc_t rg = make_rsrc(base, bytes), ru = make_rsrc(base + (int64_t)p.N * p.ldb, bytes);
#pragma unroll
    for (int j = 0; j < C::LB; ++j) {
      const int q = wave * C::LB + j;  // 8 stage rows
      const int unit = (q >> 2) * 16 + (q & 1) * 8;
      const __amdgpu_buffer_rsrc_t rb = (q >> 1) & 1 ? ru : rg;
      if (clip)
        issue_k_major<1, true>(rb, p.ldb, unit, q * 8, k0, kbytes, b_dst + j * 1024, lane);
      else
        issue_k_major<1, false>(rb, p.ldb, unit, q * 8, k0, kbytes, b_dst + j * 1024, lane);
    }
  } else {
    const __amdgpu_buffer_rsrc_t rb =
        make_rsrc(p.B + (int64_t)t.n0 * p.ldb, (int64_t)(p.N - t.n0 - 1) * p.ldb + kbytes);
    if (clip)
      issue_k_major<C::LB, true>(rb, p.ldb, wave * C::LB * 8, wave * C::LB * 8, k0, kbytes, b_dst, lane);
    else
      issue_k_major<C::LB, false>(rb, p.ldb, wave * C::LB * 8, wave * C::LB * 8, k0, kbytes, b_dst, lane);
  }
}

// Fragments of half h (64 bytes of the reduction) of a slice: lane l holds
// row l % 16, bytes [16 (l / 16), +16) of the half.
template <int COLS, bool MN, int N>
struct FragReader {
  int off;   // K-major: byte offset of the first fragment's chunk for half 0
  int row0;  // MN-major: first column block of the wave
  __device__ __forceinline__ FragReader(int area, int first_row, int lane) {
    const int l16 = lane & 15, q = lane >> 4;
    if (MN) {
      // lane i of group q reads reduction rows 8 q + i / 4 (and 4 further),
      // columns 4 (i % 4) .. +3 of the block; the transposing read hands it
      // column i of the four rows
      off = area + (8 * q + (l16 >> 2)) * COLS * 2 + (l16 & 1) * 8;
      row0 = (first_row >> 4) * 2 + ((l16 >> 1) & 1);
    } else {
      const int r = first_row + l16;
      off = area + r * 128 + ((q ^ swz16(r)) << 4);
      row0 = 0;
    }
  }
  __device__ __forceinline__ void read(const uint8_t* st, int h, int lane, i32x4 (&f)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (MN) {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const int r = 8 * (lane >> 4) + ((lane & 15) >> 2);  // row within the half
        const int chunk = ((row0 + 2 * i) ^ mn_swz<COLS / 8>(r)) << 4;
        const uint8_t* a = st + off + h * 32 * COLS * 2 + chunk;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)a);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a + 4 * COLS * 2));
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        f[i] = __builtin_bit_cast(i32x4, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      } else {
        f[i] = *(const i32x4*)(st + (off ^ (h * 64)) + i * 2048);
      }
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
  __device__ __forceinline__ void mma(const i32x4 (&a)[C::SM], const i32x4 (&b)[C::SN]) {
#pragma unroll
    for (int j = 0; j < C::SN; ++j)
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

// Four consecutive fp32 (zeros at and past column n_end), one load if aligned.
__device__ __forceinline__ f32x4 load_f32x4(const float* src, int n, int n_end) {
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
  if (n + 4 <= n_end && ((uintptr_t)(src + n) & 15) == 0) {
    x = *(const f32x4*)(src + n);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < n_end) x[r] = src[n + r];
  }
  return x;
}

// Columns [n, n + 8) of an output row from this lane and its neighbour: the
// lanes of quarters kq and kq ^ 1 trade halves of two 16-column blocks, so
// each stores 16 bytes.  n0 is the first block's first column.
__device__ __forceinline__ void store_pair(uint16_t* row, int n0, int n_end, bool ok, bool vec, int lane, uint32_t a0,
                                           uint32_t a1, uint32_t b0, uint32_t b1) {
  const int kq = lane >> 4;
  const bool odd = kq & 1;
  const int r0 = __shfl_xor((int)(odd ? a0 : b0), 16), r1 = __shfl_xor((int)(odd ? a1 : b1), 16);
  const i32x4 w = odd ? i32x4{r0, r1, (int)b0, (int)b1} : i32x4{(int)a0, (int)a1, r0, r1};
  const int n = n0 + (odd ? 16 + 4 * (kq - 1) : 4 * kq);
  if (!ok || n >= n_end) return;
  if (vec && n + 8 <= n_end) {
    *(i32x4*)(row + n) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (n + e < n_end) row[n + e] = (uint16_t)((uint32_t)w[e >> 1] >> ((e & 1) * 16));
  }
}

// The finished tile, straight from the accumulators.  Lane (l16, kq) holds
// row l16 and columns [4 kq, +4) of every 16 x 16 block.
template <class C>
__device__ __forceinline__ void store_linear(const LinearParams& p, const LinearWork& t, const LinearAcc<C>& acc,
                                             int wm, int wn, int lane) {
  const int l16 = lane & 15, kq = lane >> 4;
  constexpr int STEP = C::GATED ? 2 : 1;       // accumulator blocks per output block
  constexpr int NB = C::SN / STEP;             // output blocks of the wave
  const int nw = t.n0 + wn * NB * 16;          // the wave's first output column
  const int n_end = C::E == kEpiGatedGrad ? p.half : p.N;
  const bool vec = (p.ldd & 7) == 0 && ((uintptr_t)p.D & 15) == 0 && (C::E != kEpiGatedGrad || (p.half & 7) == 0);
  f32x4 sb[C::INT8 ? C::SN : 1];
  if constexpr (C::INT8) {
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int n = nw + j * 16 + 4 * kq;
      sb[j * STEP] = load_f32x4(p.sb, n, p.N);
      if (C::GATED) sb[j * STEP + 1] = load_f32x4(p.sb + p.N, n, p.N);
    }
  }
#pragma unroll
  for (int i = 0; i < C::SM; ++i) {
    const int m = t.m0 + wm * C::WM + i * 16 + l16;
    bool ok = m < p.M;
    int64_t drow = m;
    if (C::TA && p.F > 0 && ok) {  // dW: rows of the gradient pair
      drow = pair_row(p, m);
      ok = drow >= 0;
    }
    uint16_t* row = p.D + drow * p.ldd;
    float sa = 0.f;
    if (C::INT8 && ok) sa = p.sa[m];
    uint32_t lo[NB], hi[NB], lo2[C::E == kEpiGatedGrad ? NB : 1], hi2[C::E == kEpiGatedGrad ? NB : 1];
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
      if constexpr (C::E == kEpiGated) {
        if (p.P && ok) {
          float* prow = p.P + (int64_t)m * p.ldp;
          const bool v4 = n + 4 <= p.N && (p.N & 3) == 0 && ((uintptr_t)(prow + n) & 15) == 0;
          if (v4) {
            *(f32x4*)(prow + n) = f32x4{a[0], a[1], a[2], a[3]};
            *(f32x4*)(prow + p.N + n) = f32x4{b[0], b[1], b[2], b[3]};
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (n + r < p.N) {
                prow[n + r] = a[r];
                prow[p.N + n + r] = b[r];
              }
          }
        }
      }
      if constexpr (C::E == kEpiGatedGrad) {
        uint32_t h[2] = {0, 0};
        if (ok) {
          const uint16_t* hrow = p.dH + (int64_t)m * p.lddh;
          if (n + 4 <= p.N && ((uintptr_t)(hrow + n) & 7) == 0) {
            const uint2 u = *(const uint2*)(hrow + n);
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
          gated_grad(dh, a[r], b[r], p.act, dg[r], du[r]);
          if (n + r >= p.N) dg[r] = du[r] = 0.f;
        }
        lo2[j] = pack_bf16x2(du[0], du[1]);
        hi2[j] = pack_bf16x2(du[2], du[3]);
#pragma unroll
        for (int r = 0; r < 4; ++r) a[r] = dg[r];
      } else if constexpr (C::GATED) {
#pragma unroll
        for (int r = 0; r < 4; ++r) a[r] = gated_value(a[r], b[r], p.act);
      }
      lo[j] = pack_bf16x2(a[0], a[1]);
      hi[j] = pack_bf16x2(a[2], a[3]);
    }
#pragma unroll
    for (int j = 0; j + 1 < NB; j += 2) {
      store_pair(row, nw + j * 16, n_end, ok, vec, lane, lo[j], hi[j], lo[j + 1], hi[j + 1]);
      if constexpr (C::E == kEpiGatedGrad)
        store_pair(row + p.half, nw + j * 16, n_end, ok, vec, lane, lo2[j], hi2[j], lo2[j + 1], hi2[j + 1]);
    }
    static_assert(NB % 2 == 0, "output blocks are stored in pairs");
  }
}

// Waits of the main loop: this wave's LDS reads and direct-to-LDS loads are
// done, then the workgroup meets.
__device__ __forceinline__ void linear_sync() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The reduction runs in 128-byte slices through two LDS stages.  A slice's
// fragments are read in halves, each one half ahead of the MFMAs that use it,
// so no MFMA waits for an LDS read that was just issued; one barrier a slice
// lies between the two halves, where every wave has read all of the current
// stage and the next slice (loaded a whole slice earlier) has landed.  The
// loads run two slices ahead and go on into the workgroup's next tile.
template <class C>
__global__ __launch_bounds__(C::THREADS, C::OCC * C::NW / 4) void linear_tile_kernel(LinearParams p) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::LDS_BYTES];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  const int grid = gridDim.x;
  const int nk = p.nk;

  int w = xcd_local_id(blockIdx.x, grid);
  LinearWork cur = linear_work<C>(p, w);
  if (cur.w < 0) return;
  LinearWork ld = cur;  // where the loads are: slice ld_kb of tile ld
  int ld_kb = 0;
  auto load_next = [&](uint8_t* stage) {
    if (ld.w < 0) return;
    issue_linear_slice<C>(p, ld, ld_kb, stage, wave, lane);
    if (++ld_kb == nk) {
      ld_kb = 0;
      ld = linear_work<C>(p, ld.w + grid);
    }
  };

  const FragReader<C::BM, C::TA, C::SM> ra(0, wm * C::WM, lane);
  const FragReader<C::BN, C::TB, C::SN> rb(C::BM * 128, wn * C::WN, lane);
  i32x4 a0[C::SM], b0[C::SN], a1[C::SM], b1[C::SN];
  LinearAcc<C> acc;
  acc.zero();

  load_next(lds);
  linear_sync();
  load_next(lds + C::STAGE);
  ra.read(lds, 0, lane, a0);
  rb.read(lds, 0, lane, b0);
  int s = 0;
  while (cur.w >= 0) {
    for (int kb = 0; kb < nk; ++kb) {
      uint8_t* st = lds + s * C::STAGE;
      rb.read(st, 1, lane, b1);
      ra.read(st, 1, lane, a1);
      __builtin_amdgcn_sched_barrier(0);
      acc.mma(a0, b0);
      linear_sync();
      s ^= 1;
      load_next(st);
      rb.read(lds + s * C::STAGE, 0, lane, b0);
      ra.read(lds + s * C::STAGE, 0, lane, a0);
      __builtin_amdgcn_sched_barrier(0);
      acc.mma(a1, b1);
      __builtin_amdgcn_sched_barrier(0);
    }
    store_linear<C>(p, cur, acc, wm, wn, lane);
    acc.zero();
    cur = linear_work<C>(p, cur.w + grid);
  }
}

}  // namespace fg
