// linear_kernel.hpp -- 8-bit-integer and bf16 products with the gated
// feed-forward epilogues.
//
//   int8    D[m,n]  = bf16( sa[m] sb[n] sum_k A[m,k] B[n,k] )
//   gated   g = X Wg^T, u = X Wu^T, H = bf16( act(g) u )          W = [Wg; Wu]
//   grad    dg = dH u act'(g), du = dH act(g), dX = [dg du] W, dW = [dg du]^T X
//
// Integer sums are exact in 32 bits (the entry points bound K); bf16 products
// accumulate in fp32.  Scales and activations are applied in fp32 and every
// output is rounded to bf16 once.  The gradient pair [dg du] is the one
// intermediate that is rounded: it is the bf16 operand of two further matrix
// products, as dH is.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gemm_kernel.hpp"

namespace fg {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
// Vectors at addresses that are aligned to their elements only (rows of any
// stride): the compiler makes one access of them, which the hardware takes at
// any address.
typedef i32x4 i32x4_at2 __attribute__((aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_at2 __attribute__((aligned(2)));
typedef f32x4 f32x4_at4 __attribute__((aligned(4)));

enum LinearEpi {
  kEpiInt8,       // D = bf16(sa sb acc)
  kEpiBf16,       // D = bf16(acc)
  kEpiPartial,    // P[split] = acc, [M, N] in fp32: one split of the reduction
  kEpiGated,      // D = bf16(act(g) u)
  kEpiGatedInt8,  // the same with g, u = sa sb acc
  kEpiGatedGrad,  // D = bf16([dg du]) from g, u and dH
  kEpiGatedKeep,  // kEpiGated and P = [g u] in fp32
  // P[split] = [g u], [M, 2 half] in fp32: one split of the reduction
  kEpiGatedPartial,
};
constexpr bool epi_gated(int e) { return e >= kEpiGated; }
constexpr bool epi_partial(int e) { return e == kEpiPartial || e == kEpiGatedPartial; }
constexpr bool epi_int8(int e) { return e == kEpiInt8 || e == kEpiGatedInt8; }

enum { kActSilu = 0, kActGeluTanh = 1 };

struct LinearParams {
  const uint8_t* A;  // [M, K] rows of lda bytes; MN-major: [K, M]
  int64_t lda;
  const uint8_t* B;  // [N, K] rows of ldb bytes (gated: up row f is row N + f); MN-major: [K, N]
  int64_t ldb;
  const float *sa, *sb;  // int8 scales
  uint16_t* D;
  int64_t ldd;  // elements
  float* P;     // pre-activations [M, 2N] (kEpiGatedKeep: written)
  int64_t ldp;
  const uint16_t* dH;  // gradient: [M, N]
  int64_t lddh;
  int M, N, K;  // K in elements
  int act;
  // gradient pair [dg du]: each half padded to `half` columns (zeros past F).
  // As the reduction axis (dX) or the output rows (dW) index r stands for
  // hidden unit r < F of the first half and r - half of the second.
  int F, half;
  // slices of the reduction (partial sums: and of one split, an even number)
  // and output tiles of the persistent grid (linear_tile.hpp)
  int nk, split_nk;
  int tiles_m, tiles_n, num_tiles, group_m;
};

// Row of W (or dW) for column r of the gradient pair; -1 for a padding column.
__device__ __forceinline__ int pair_row(const LinearParams& p, int r) {
  const int h = r >= p.half ? 1 : 0;
  const int f = r - h * p.half;
  return f < p.F ? h * p.F + f : -1;
}

// act(g) = g s with s = 1 / (1 + exp(-y(g))); silu: y = g; gelu (tanh form):
// y = 2 c (g + a g^3), c = sqrt(2 / pi).  The factors of y and log2(e) are one
// constant.  exp overflows to infinity for far negative y, and s is then 0.
constexpr float kLog2e = 1.4426950408889634f, kGelu2C = 1.5957691216057308f, kGeluA = 0.044715f;
template <int ACT>
__device__ __forceinline__ float act_gate(float g) {
  const float z = ACT == kActSilu ? -kLog2e * g : g * __builtin_fmaf(-kLog2e * kGelu2C * kGeluA, g * g, -kLog2e * kGelu2C);
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z));
}
template <int ACT>
__device__ __forceinline__ float gated_value(float g, float u) {
  return g * act_gate<ACT>(g) * u;
}

// dg = dH u act'(g), du = dH act(g), act'(g) = s + g s (1 - s) y'(g).  Where
// s (1 - s) has underflowed the last term is 0 (y' may have overflowed there).
// dH is multiplied last: dH u and dH g may overflow where the gradient, with
// act' or s near 0, does not.
template <int ACT>
__device__ __forceinline__ void gated_grad(float dh, float g, float u, float& dg, float& du) {
  const float s = act_gate<ACT>(g);
  const float t = s * (1.f - s);
  const float slope = ACT == kActSilu ? 1.f : kGelu2C * (1.f + 3.f * kGeluA * g * g);
  dg = dh * (u * (s + (t == 0.f ? 0.f : g * t * slope)));
  du = dh * (g * s);
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t bf16_bits(float v) { return (uint16_t)(pack_bf16x2(v, 0.f) & 0xffff); }

// [dg du] from the pre-activations P = [g u]: the kept ones ([M, 2F]; eight
// columns a thread, bound by HBM: 10 bytes in and 4 out for each hidden unit
// and row), or PARTS of them, partial sums ([M, 2 half] each) that are added
// in order; four columns a thread and eight partials in flight, since the
// tensor is small and its loads' latency counts (112 x 119, 16 partials: 12 us
// with eight columns and four).
template <int ACT, bool PARTS>
__global__ __launch_bounds__(256) void gated_grad_kernel(LinearParams p, int parts) {
  constexpr int C = PARTS ? 4 : 8;
  const int per_row = p.half / C;
  const int64_t total = (int64_t)p.M * per_row;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / per_row;
    const int n = (int)(i - m * per_row) * C;
    const float* gp = p.P + m * p.ldp + n;
    const float* up = gp + (PARTS ? p.half : p.N);
    const uint16_t* hp = p.dH + m * p.lddh + n;
    float g[C], u[C];
    uint32_t h[C / 2];
    if (PARTS || n + C <= p.N) {
      f32x4 gv[C / 4], uv[C / 4];
#pragma unroll
      for (int q = 0; q < C / 4; ++q) {
        gv[q] = *(const f32x4_at4*)(gp + 4 * q);
        uv[q] = *(const f32x4_at4*)(up + 4 * q);
      }
      if constexpr (PARTS) {
        const int64_t one = p.M * p.ldp;
#pragma unroll 8
        for (int k = 1; k < parts; ++k) {
          gv[0] += *(const f32x4*)(gp + k * one);
          uv[0] += *(const f32x4*)(up + k * one);
        }
      }
#pragma unroll
      for (int r = 0; r < C; ++r) {
        g[r] = gv[r / 4][r % 4];
        u[r] = uv[r / 4][r % 4];
      }
    } else {
#pragma unroll
      for (int r = 0; r < C; ++r) {
        g[r] = n + r < p.N ? gp[r] : 0.f;  // padding columns hold zeros
        u[r] = n + r < p.N ? up[r] : 0.f;
      }
    }
    if (n + C <= p.N) {
#pragma unroll
      for (int q = 0; q < C / 4; ++q) {
        const u32x2 v = *(const u32x2_at2*)(hp + 4 * q);
        h[2 * q] = v.x;
        h[2 * q + 1] = v.y;
      }
    } else {
      if constexpr (PARTS) {
        // padding columns hold zeros; their sums need not, where an infinite
        // input met the zeros that stand for their weights
#pragma unroll
        for (int r = 0; r < C; ++r)
          if (n + r >= p.N) g[r] = u[r] = 0.f;
      }
#pragma unroll
      for (int q = 0; q < C / 2; ++q)
        h[q] = (n + 2 * q < p.N ? (uint32_t)hp[2 * q] : 0u) | (n + 2 * q + 1 < p.N ? (uint32_t)hp[2 * q + 1] << 16 : 0u);
    }
    uint32_t dg[C / 2], du[C / 2];
#pragma unroll
    for (int q = 0; q < C / 2; ++q) {
      float a0, b0, a1, b1;
      gated_grad<ACT>(__uint_as_float(h[q] << 16), g[2 * q], u[2 * q], a0, b0);
      gated_grad<ACT>(__uint_as_float(h[q] & 0xffff0000u), g[2 * q + 1], u[2 * q + 1], a1, b1);
      dg[q] = pack_bf16x2(a0, a1);
      du[q] = pack_bf16x2(b0, b1);
    }
    uint16_t* dst = p.D + m * p.ldd + n;
    if constexpr (PARTS) {
      *(uint2*)dst = make_uint2(dg[0], dg[1]);
      *(uint2*)(dst + p.half) = make_uint2(du[0], du[1]);
    } else {
      *(uint4*)dst = make_uint4(dg[0], dg[1], dg[2], dg[3]);
      *(uint4*)(dst + p.half) = make_uint4(du[0], du[1], du[2], du[3]);
    }
  }
}

// D = bf16(sum of `splits` partials P), added in split order, four columns a
// thread (N % 4 == 0).
static __global__ __launch_bounds__(256) void add_partials_kernel(LinearParams p, int splits) {
  const int per_row = p.N / 4;
  const int64_t quads = (int64_t)p.M * per_row;
  const f32x4* src = (const f32x4*)p.P;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < quads; i += (int64_t)gridDim.x * 256) {
    f32x4 s = src[i];
#pragma unroll 8
    for (int k = 1; k < splits; ++k) s += src[k * quads + i];
    const int64_t m = i / per_row;
    *(u32x2_at2*)(p.D + m * p.ldd + (i - m * per_row) * 4) = u32x2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
  }
}

// The 16-byte piece of a row at src as fp32 values.
__device__ __forceinline__ void widen(const uint4& u, float (&x)[4], const float*) {
  x[0] = __uint_as_float(u.x);
  x[1] = __uint_as_float(u.y);
  x[2] = __uint_as_float(u.z);
  x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void widen(const uint4& u, float (&x)[8], const uint16_t*) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// rint(x / s) of V values, packed into bytes.  x * (1 / s) differs from the
// rounded quotient by less than 127 * 3 * 2^-24 < 3e-5, so both round to the
// same integer unless the product lies that close to a half; only then are
// the values divided (about 1 piece in 600; a division is some ten
// instructions, and with one for every value the cast is not bound by HBM).
template <int V>
__device__ __forceinline__ void int8_codes(const float (&x)[V], float s, float inv, uint32_t (&out)[V / 4]) {
  float q[V], far = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float t = x[i] * inv;
    q[i] = __builtin_rintf(t);
    far = fmaxf(far, fabsf(t - q[i]));
  }
  if (far > 0.4999f) {
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] = __builtin_rintf(x[i] / s);
  }
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    out[i] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) out[i] |= ((uint32_t)(int)q[4 * i + j] & 0xffu) << (8 * j);
  }
}

// int8 codes and scale of each row: s = max(amax, 1e-4) (1 / 127), q = rint(x / s).
// One workgroup a row.  The first PIECES 16-byte pieces of each thread stay in
// registers between the two passes, so a row of up to PIECES * THREADS * 16
// bytes is read once; of a longer row the rest is read again.
template <typename T, int THREADS, int PIECES>
__global__ __launch_bounds__(THREADS) void int8_cast_kernel(const T* __restrict__ x, int64_t ldx,
                                                            int8_t* __restrict__ q, float* __restrict__ s, int M,
                                                            int K) {
  constexpr int V = 16 / sizeof(T), WAVES = THREADS / 64;
  __shared__ float red[WAVES];
  const int tid = threadIdx.x, pieces = K / V;
  // unsigned: M may lie less than a grid below 2^31
  for (unsigned m = blockIdx.x; m < (unsigned)M; m += gridDim.x) {
    const uint4* row = (const uint4*)(x + (int64_t)m * ldx);
    uint4 v[PIECES];
#pragma unroll
    for (int j = 0; j < PIECES; ++j) {
      const int i = tid + j * THREADS;
      v[j] = i < pieces ? row[i] : make_uint4(0, 0, 0, 0);
    }
    float amax = 0.f;
    auto take = [&](const uint4& u) {
      float f[V];
      widen(u, f, (const T*)nullptr);
#pragma unroll
      for (int i = 0; i < V; ++i) amax = fmaxf(amax, fabsf(f[i]));
    };
#pragma unroll
    for (int j = 0; j < PIECES; ++j) take(v[j]);
    for (int i = tid + PIECES * THREADS; i < pieces; i += THREADS) take(row[i]);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 64));
    if ((tid & 63) == 0) red[tid >> 6] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) amax = fmaxf(amax, red[w]);
    const float sc = fmaxf(amax, 1e-4f) * (1.0f / 127.0f), inv = 1.0f / sc;
    if (tid == 0) s[m] = sc;
    uint32_t* dst = (uint32_t*)(q + (int64_t)m * K);
    auto put = [&](const uint4& u, int i) {
      float f[V];
      uint32_t c[V / 4];
      widen(u, f, (const T*)nullptr);
      int8_codes<V>(f, sc, inv, c);
      if constexpr (V == 8)
        *(uint2*)(dst + 2 * i) = make_uint2(c[0], c[1]);
      else
        dst[i] = c[0];
    };
#pragma unroll
    for (int j = 0; j < PIECES; ++j) {
      const int i = tid + j * THREADS;
      if (i < pieces) put(v[j], i);
    }
    for (int i = tid + PIECES * THREADS; i < pieces; i += THREADS) put(row[i], i);
    __syncthreads();  // red is free again
  }
}

}  // namespace fg
