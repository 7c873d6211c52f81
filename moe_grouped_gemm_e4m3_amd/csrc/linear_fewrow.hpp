// linear_fewrow.hpp -- the few-row (decode) kernel of the 8-bit-integer and
// bf16 products: the time is the weight stream's.
//
// A workgroup holds a tile of 16 MF rows and 16 CF weight rows (gated: half
// of them gate rows, half up rows of the same hidden units).  Its waves share
// out the tile's K slices (128 bytes of every row), each streaming its own
// through an LDS ring of DEPTH slots that it alone uses, so the loop has no
// barrier and DEPTH - 1 slices a wave are in flight.  The waves' partials are
// added in wave order.  More rows than a tile holds go to further workgroups
// (parts), which run side by side and share the weights in L2.  Nothing is
// split over workgroups: where tiles are few, smaller row parts occupy the
// device without an exchange (64 x 512 x 8192: four 16-row parts of eight
// waves 4.2 us, one 64-row part 7.2; its slices split over four workgroups
// through memory took 1.4 times the former).
//
// Measured in a HIP graph with the weights in the last-level cache: int8 1 x
// 7168 x 2048 2.9 us (5.1 TB/s), gated int8 16 x 2048 x 7168 5.1 us (5.8 TB/s),
// gated bf16 1 x 2048 x 7168 10.1 us (5.8 TB/s).  int8 128 x 2112 x 7168, 9.9
// us, is bound by what each CU fetches: its activations' rows next to its
// weights'.
#pragma once

#include "linear_tile.hpp"

namespace fg {

template <int E_, int MF_, int CF_, int WAVES_, int DEPTH_>
struct FewRow {
  static constexpr int E = E_, MF = MF_, CF = CF_, WAVES = WAVES_, DEPTH = DEPTH_;
  static constexpr bool INT8 = epi_int8(E), GATED = epi_gated(E);
  static constexpr int ES = INT8 ? 1 : 2;
  static constexpr int THREADS = WAVES * 64;
  static constexpr int ROWS = 16 * MF, COLS = 16 * CF;
  static constexpr int OUT_N = GATED ? COLS / 2 : COLS;
  static constexpr int SLOT = (ROWS + COLS) * 128, RING = DEPTH * SLOT;
  static constexpr int LOADS = (ROWS + COLS) / 8;  // direct-to-LDS loads of a slice
  static constexpr int GROUPS = MF * CF;           // 16 x 16 blocks
  static constexpr int PART = GROUPS * 1024;       // bytes of one partial tile
  static constexpr int LDS_BYTES = WAVES * RING;
  // outputs come in items: four columns of one row (gated: with both products)
  static constexpr int ITEMS = GROUPS * 64 / (GATED ? 2 : 1);
  static constexpr int OCC = 2 * LDS_BYTES <= 160 * 1024 ? 2 : 1;
  static_assert(LDS_BYTES <= 160 * 1024 && PART <= RING, "LDS");
  static_assert((DEPTH - 1) * LOADS < 64, "vmcnt");
};

// Wait until at most N of this wave's vector memory operations are outstanding.
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Four output columns [n, n + 4) of row m from their sums (gated: both products).
template <class C>
__device__ __forceinline__ void fewrow_store(const LinearParams& p, int m, int n, const float (&x)[4],
                                             const float (&y)[4]) {
  if (m >= p.M || n >= p.N) return;
  float a[4], b[4];
  const f32x4 sg = C::INT8 ? load_f32x4(p.sb, n, p.N) : f32x4{0.f, 0.f, 0.f, 0.f};
  const f32x4 su = C::INT8 && C::GATED ? load_f32x4(p.sb + p.N, n, p.N) : f32x4{0.f, 0.f, 0.f, 0.f};
  const float sa = C::INT8 ? p.sa[m] : 0.f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    a[r] = C::INT8 ? x[r] * sa * sg[r] : x[r];
    if (C::GATED) b[r] = C::INT8 ? y[r] * sa * su[r] : y[r];
  }
  if constexpr (C::E == kEpiGatedKeep) {
    float* prow = p.P + (int64_t)m * p.ldp;
    if (n + 4 <= p.N) {
      *(f32x4_at4*)(prow + n) = f32x4{a[0], a[1], a[2], a[3]};
      *(f32x4_at4*)(prow + p.N + n) = f32x4{b[0], b[1], b[2], b[3]};
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < p.N) {
          prow[n + r] = a[r];
          prow[p.N + n + r] = b[r];
        }
    }
  }
  if constexpr (C::GATED) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      a[r] = p.act == kActSilu ? gated_value<kActSilu>(a[r], b[r]) : gated_value<kActGeluTanh>(a[r], b[r]);
  }
  uint16_t* dst = p.D + (int64_t)m * p.ldd + n;
  if (n + 4 <= p.N) {
    *(u32x2_at2*)dst = u32x2{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3])};
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < p.N) dst[r] = bf16_bits(a[r]);
  }
}

// Grid: column tiles x row parts, parts fastest.
template <class C>
__global__ __launch_bounds__(C::THREADS, C::OCC * C::WAVES / 4) void fewrow_kernel(
    LinearParams p, int parts) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::LDS_BYTES];
  typedef typename std::conditional<C::INT8, i32x4, f32x4>::type V;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tile = blockIdx.x / parts;
  const int m0 = (blockIdx.x - tile * parts) * C::ROWS, n0 = tile * C::OUT_N;
  const int kbytes = p.K * C::ES;
  const int n = (p.nk - wave + C::WAVES - 1) / C::WAVES;  // slices wave, wave + WAVES, ... are this wave's

  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.A + (int64_t)m0 * p.lda, (int64_t)(p.M - m0 - 1) * p.lda + kbytes);
  const int64_t b_bytes = (int64_t)(p.N - n0 - 1) * p.ldb + kbytes;
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.B + (int64_t)n0 * p.ldb, b_bytes);
  const __amdgpu_buffer_rsrc_t ru = make_rsrc(p.B + (int64_t)(p.N + n0) * p.ldb, C::GATED ? b_bytes : 0);
  const int r8 = lane >> 3;
  const int col = ((lane & 7) ^ lin_swz(r8)) * 16;
  uint8_t* ring = lds + wave * C::RING;
  // slices past the wave's last load nothing (but count as loads)
  auto load = [&](int i, int slot) {
    const int kb = i < n ? i * C::WAVES + wave : p.nk;
    const int k0 = kb * 128;
    uint8_t* dst = ring + slot * C::SLOT;
    const bool in = kb < p.nk && k0 + col < kbytes;
#pragma unroll
    for (int j = 0; j < C::LOADS; ++j) {
      const bool is_a = j < 2 * C::MF;
      const int q = is_a ? j : j - 2 * C::MF;
      // stage rows of the weights: the first half of the tile gate, the second up
      const bool up = C::GATED && !is_a && q >= C::CF;
      const int row = 8 * (up ? q - C::CF : q) + r8;
      const int v = in ? row * (int)(is_a ? p.lda : p.ldb) + col : kOobOffset;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(is_a ? ra : up ? ru : rb,
                                               (__attribute__((address_space(3))) void*)(dst + j * 1024), 16, v,
                                               kb < p.nk ? k0 : 0, 0, 0);
    }
  };

  V acc[C::MF][C::CF];
#pragma unroll
  for (int i = 0; i < C::MF; ++i)
#pragma unroll
    for (int j = 0; j < C::CF; ++j) acc[i][j] = V{0, 0, 0, 0};
  const int l16 = lane & 15, kq = lane >> 4;
  const int off = l16 * 128 + ((kq ^ lin_swz(l16)) << 4);
  auto compute = [&](int slot) {
    const uint8_t* st = ring + slot * C::SLOT;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      i32x4 a[C::MF], b[C::CF];
#pragma unroll
      for (int i = 0; i < C::MF; ++i) a[i] = *(const i32x4*)(st + (off ^ (h * 64)) + i * 2048);
#pragma unroll
      for (int j = 0; j < C::CF; ++j) b[j] = *(const i32x4*)(st + C::ROWS * 128 + (off ^ (h * 64)) + j * 2048);
#pragma unroll
      for (int j = 0; j < C::CF; ++j)
#pragma unroll
        for (int i = 0; i < C::MF; ++i) {
          if constexpr (C::INT8)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[j], a[i], acc[i][j], 0, 0, 0);
          else
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b[j]),
                                                                __builtin_bit_cast(bf16x8, a[i]), acc[i][j], 0, 0, 0);
        }
    }
  };

#pragma unroll
  for (int d = 0; d < C::DEPTH - 1; ++d) load(d, d);
  int slot = 0;
  for (int i = 0; i < n; ++i) {
    const int into = slot == 0 ? C::DEPTH - 1 : slot - 1;  // the slot read in the last iteration
    load(i + C::DEPTH - 1, into);
    wait_loads<(C::DEPTH - 1) * C::LOADS>();
    compute(slot);
    // the slot is loaded again in the next iteration: its reads are done
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_sched_barrier(0);
    slot = slot == C::DEPTH - 1 ? 0 : slot + 1;
  }
  wait_loads<0>();  // no load may still be writing the ring

  // ---- the waves' partials, added in wave order ----
  V* mine = (V*)(lds + wave * C::RING);
#pragma unroll
  for (int i = 0; i < C::MF; ++i)
#pragma unroll
    for (int j = 0; j < C::CF; ++j) mine[(i * C::CF + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  // item x: the four sums at `first` (and, gated, those of the up product at `second`)
  auto place = [&](int x, int& first, int& second, int& m, int& col0) {
    if (C::GATED && C::CF == 1) {
      // 8 gate and 8 up rows share a block: lanes 0-31 hold the gates
      const int g = x >> 5, l = x & 31;
      first = g * 64 + l;
      second = first + 32;
      m = 16 * g + (l & 15);
      col0 = 4 * (l >> 4);
    } else {
      constexpr int HALF = C::GATED ? (C::CF > 1 ? C::CF / 2 : 1) : C::CF;
      const int g = x >> 6, l = x & 63;
      const int i = g / HALF, j = g % HALF;
      first = (i * C::CF + j) * 64 + l;
      second = first + HALF * 64;
      m = 16 * i + (l & 15);
      col0 = 16 * j + 4 * (l >> 4);
    }
  };
  auto add_waves = [&](int at) {
    V s = ((const V*)lds)[at];
#pragma unroll
    for (int w = 1; w < C::WAVES; ++w) s += ((const V*)(lds + w * C::RING))[at];
    return s;
  };
  constexpr int PER = (C::ITEMS + C::THREADS - 1) / C::THREADS;
#pragma unroll
  for (int y = 0; y < PER; ++y) {
    const int x = y * C::THREADS + tid;
    if (x < C::ITEMS) {
      int first, second, m, c0;
      place(x, first, second, m, c0);
      const V a = add_waves(first), b = C::GATED ? add_waves(second) : a;
      float fa[4], fb[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        fa[r] = (float)a[r];
        fb[r] = (float)b[r];
      }
      fewrow_store<C>(p, m0 + m, n0 + c0, fa, fb);
    }
  }
}

}  // namespace fg
