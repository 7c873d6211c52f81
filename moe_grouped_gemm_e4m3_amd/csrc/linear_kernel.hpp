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
  // slices of the reduction and output tiles of the persistent grid (linear_tile.hpp)
  int nk;
  int tiles_m, tiles_n, num_tiles, group_m;
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

// [dg du] from the kept pre-activations P = [g u], one element a thread.
static __global__ __launch_bounds__(256) void gated_grad_kernel(LinearParams p) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= p.half) return;
  for (int m = blockIdx.y; m < p.M; m += gridDim.y) {
    float dg = 0.f, du = 0.f;
    if (n < p.N) {
      const float* prow = p.P + (int64_t)m * p.ldp;
      gated_grad(to_f32(p.dH[(int64_t)m * p.lddh + n]), prow[n], prow[p.N + n], p.act, dg, du);
    }
    p.D[(int64_t)m * p.ldd + n] = bf16_bits(dg);
    p.D[(int64_t)m * p.ldd + p.half + n] = bf16_bits(du);
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
