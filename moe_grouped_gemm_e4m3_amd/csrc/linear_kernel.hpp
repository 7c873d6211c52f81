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

#include "gemm_kernel.hpp"

namespace fg {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum LinearEpi {
  kEpiInt8,       // D = bf16(sa sb acc)
  kEpiBf16,       // D = bf16(acc)
  kEpiGated,      // D = bf16(act(g) u), optionally P = [g u] in fp32
  kEpiGatedInt8,  // the same with g, u = sa sb acc
  kEpiGatedGrad,  // D = bf16([dg du]) from g, u and dH
};
constexpr bool epi_gated(int e) { return e == kEpiGated || e == kEpiGatedInt8 || e == kEpiGatedGrad; }
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
  float* P;     // gated: pre-activations [M, 2N] or NULL
  int64_t ldp;
  const uint16_t* dH;  // gradient: [M, N]
  int64_t lddh;
  int M, N, K;  // K in elements
  int act;
  // gradient pair [dg du]: each half padded to `half` columns (zeros past F).
  // As the reduction axis (dX) or the output rows (dW) index r stands for
  // hidden unit r < F of the first half and r - half of the second.
  int F, half;
};

// Row of W (or dW) for column r of the gradient pair; -1 for a padding column.
__device__ __forceinline__ int pair_row(const LinearParams& p, int r) {
  const int h = r >= p.half ? 1 : 0;
  const int f = r - h * p.half;
  return f < p.F ? h * p.F + f : -1;
}

__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + __expf(-x)); }

// act(g) = g s with s = sigmoid(y(g)); silu: y = g; gelu (tanh form):
// y = 2 c (g + a g^3), c = sqrt(2 / pi).
constexpr float kGelu2C = 1.5957691216057308f, kGeluA = 0.044715f;
__device__ __forceinline__ float act_gate(float g, int act) {
  return sigmoid(act == kActSilu ? g : kGelu2C * (g + kGeluA * g * g * g));
}
__device__ __forceinline__ float gated_value(float g, float u, int act) { return g * act_gate(g, act) * u; }

// dg = dH u act'(g), du = dH act(g), act'(g) = s + g s (1 - s) y'(g).  Where
// s (1 - s) has underflowed the last term is 0 (y' may have overflowed there).
__device__ __forceinline__ void gated_grad(float dh, float g, float u, int act, float& dg, float& du) {
  const float s = act_gate(g, act);
  const float t = s * (1.f - s);
  const float slope = act == kActSilu ? 1.f : kGelu2C * (1.f + 3.f * kGeluA * g * g);
  dg = dh * u * (s + (t == 0.f ? 0.f : g * t * slope));
  du = dh * g * s;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t bf16_bits(float v) { return (uint16_t)(pack_bf16x2(v, 0.f) & 0xffff); }

// One output element from its accumulators (b: the up product of a gated form).
template <int E>
__device__ __forceinline__ void store_one(const LinearParams& p, int m, int n, float a, float b) {
  if (m >= p.M) return;
  if (E == kEpiGatedGrad) {
    if (n >= p.half) return;
    float dg = 0.f, du = 0.f;
    if (n < p.N) gated_grad(to_f32(p.dH[(int64_t)m * p.lddh + n]), a, b, p.act, dg, du);
    p.D[(int64_t)m * p.ldd + n] = bf16_bits(dg);
    p.D[(int64_t)m * p.ldd + p.half + n] = bf16_bits(du);
    return;
  }
  if (n >= p.N) return;
  if (epi_int8(E)) {
    a = a * p.sa[m] * p.sb[n];
    if (epi_gated(E)) b = b * p.sa[m] * p.sb[p.N + n];
  }
  if (epi_gated(E)) {
    if (E == kEpiGated && p.P) {
      p.P[(int64_t)m * p.ldp + n] = a;
      p.P[(int64_t)m * p.ldp + p.N + n] = b;
    }
    a = gated_value(a, b, p.act);
  }
  p.D[(int64_t)m * p.ldd + n] = bf16_bits(a);
}

// A 64 x 64 output tile per workgroup of four waves; operands go through LDS
// element by element with every index checked.
template <int E, bool TA, bool TB>
__global__ __launch_bounds__(256) void linear_kernel(LinearParams p) {
  constexpr int ES = epi_int8(E) ? 1 : 2;     // bytes of an operand element
  constexpr int KT = 64 / ES;                 // reduction elements of a slice
  constexpr int NB = epi_gated(E) ? 2 : 1;
  __shared__ __attribute__((aligned(16))) uint8_t sA[64 * 80];
  __shared__ __attribute__((aligned(16))) uint8_t sB[NB][64 * 80];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tiles_n = ((E == kEpiGatedGrad ? p.half : p.N) + 63) / 64;
  const int m0 = (int)(blockIdx.x / tiles_n) * 64, n0 = (int)(blockIdx.x % tiles_n) * 64;

  auto get = [&](const uint8_t* base, int64_t ld, bool t, int64_t row, int64_t k) {
    const uint8_t* s = base + (t ? k * ld + row * ES : row * ld + k * ES);
    return ES == 1 ? (int)*s : (int)*(const uint16_t*)s;
  };
  f32x4 facc[NB][4];
  i32x4 iacc[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      facc[b][t] = f32x4{0.f, 0.f, 0.f, 0.f};
      iacc[b][t] = i32x4{0, 0, 0, 0};
    }
  for (int k0 = 0; k0 < p.K; k0 += KT) {
    for (int i = threadIdx.x; i < 64 * KT; i += 256) {
      // neighbouring threads take neighbouring elements of the stored rows
      const int ra = TA ? i & 63 : i / KT, ka = TA ? i >> 6 : i % KT;
      const int rb = TB ? i & 63 : i / KT, kb = TB ? i >> 6 : i % KT;
      int v = 0;
      if (m0 + ra < p.M && k0 + ka < p.K) v = get(p.A, p.lda, TA, m0 + ra, k0 + ka);
      if (ES == 1) sA[ra * 80 + ka] = (uint8_t)v;
      else *(uint16_t*)(sA + ra * 80 + 2 * ka) = (uint16_t)v;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        int64_t row = n0 + rb, k = k0 + kb;
        bool ok = n0 + rb < p.N && k < p.K;
        if (TB && ok && p.F > 0 && !TA) {  // dX: the reduction runs over the gradient pair
          k = pair_row(p, (int)k);
          ok = k >= 0;
        }
        v = ok ? get(p.B, p.ldb, TB, row + (int64_t)b * p.N, k) : 0;
        if (ES == 1) sB[b][rb * 80 + kb] = (uint8_t)v;
        else *(uint16_t*)(sB[b] + rb * 80 + 2 * kb) = (uint16_t)v;
      }
    }
    __syncthreads();
    const int at = (lane & 15) * 80 + (lane >> 4) * 16;
    const i32x4 a = *(const i32x4*)(sA + wave * 16 * 80 + at);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const i32x4 w = *(const i32x4*)(sB[b] + t * 16 * 80 + at);
        if (epi_int8(E))
          iacc[b][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, a, iacc[b][t], 0, 0, 0);
        else
          facc[b][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w),
                                                               __builtin_bit_cast(bf16x8, a), facc[b][t], 0, 0, 0);
      }
    __syncthreads();
  }
  // lane: row lane % 16, four consecutive columns 4 (lane / 16)
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = m0 + wave * 16 + (lane & 15), n = n0 + t * 16 + 4 * (lane >> 4) + r;
      const float a = epi_int8(E) ? (float)iacc[0][t][r] : facc[0][t][r];
      const float b = epi_int8(E) ? (float)iacc[NB - 1][t][r] : facc[NB - 1][t][r];
      if (TA && m < p.M) {  // dW: the output rows are the gradient pair's columns
        const int row = pair_row(p, m);
        if (row >= 0 && n < p.N) p.D[(int64_t)row * p.ldd + n] = bf16_bits(a);
      } else {
        store_one<E>(p, m, n, a, b);
      }
    }
}

// [dg du] from the kept pre-activations P = [g u], one element a thread.
static __global__ __launch_bounds__(256) void gated_grad_kernel(LinearParams p) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= p.half) return;
  for (int m = blockIdx.y; m < p.M; m += gridDim.y) {
    float g = 0.f, u = 0.f;
    if (n < p.N) {
      g = p.P[(int64_t)m * p.ldp + n];
      u = p.P[(int64_t)m * p.ldp + p.N + n];
    }
    store_one<kEpiGatedGrad>(p, m, n, g, u);
  }
}

// int8 codes and scale of each row: s = max(amax, 1e-4) / 127, q = rint(x / s).
template <typename T>
__global__ __launch_bounds__(256) void int8_cast_kernel(const T* x, int64_t ldx, int8_t* q, float* s, int M, int K) {
  __shared__ float red[4];
  for (int m = blockIdx.x; m < M; m += gridDim.x) {
    const T* row = x + (int64_t)m * ldx;
    float amax = 0.f;
    for (int k = threadIdx.x; k < K; k += 256) amax = fmaxf(amax, fabsf(to_f32(row[k])));
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float sc = fmaxf(amax, 1e-4f) / 127.0f;
    if (threadIdx.x == 0) s[m] = sc;
    for (int k = threadIdx.x; k < K; k += 256)
      q[(int64_t)m * K + k] = (int8_t)(int)__builtin_rintf(to_f32(row[k]) / sc);
    __syncthreads();
  }
}

}  // namespace fg
