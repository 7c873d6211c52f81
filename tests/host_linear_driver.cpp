// host_linear_driver.cpp -- drives the C entry points of the 8-bit-integer
// product and the gated block through their host code, for a build with
// AddressSanitizer and UndefinedBehaviorSanitizer
// (tests/test_host_sanitizers_linear.py).
//
// No GPU is needed: every call fails a host check, is an empty problem, or
// stops at the first device query (FG_EHIP without a device).  Pointers are
// fake device addresses that are never dereferenced.  Exit status 0 and "host
// linear ok" mean every status matched.
#include <cstdint>
#include <cstdio>

#include "fp8gemm.h"

static int g_fail = 0;

#define EXPECT(call, want)                                                                              \
  do {                                                                                                  \
    const int st__ = (int)(call);                                                                       \
    if (st__ != (int)(want)) {                                                                          \
      std::fprintf(stderr, "line %d: %s returned %d, expected %d (%s)\n", __LINE__, #call, st__,          \
                   (int)(want), fg_last_error());                                                       \
      ++g_fail;                                                                                         \
    }                                                                                                   \
  } while (0)

int main() {
  const int8_t* A = reinterpret_cast<const int8_t*>(0x10000);
  int8_t* Q = reinterpret_cast<int8_t*>(0x10000);
  const float* S = reinterpret_cast<const float*>(0x10000);
  float* P = reinterpret_cast<float*>(0x10000);
  const uint16_t* X = reinterpret_cast<const uint16_t*>(0x10000);
  uint16_t* D = reinterpret_cast<uint16_t*>(0x10000);
  void* WS = reinterpret_cast<void*>(0x10000);
  const int64_t big = (int64_t)1 << 60;
  const int top = 0x7fffffff, rows = 1 << 30;
  const int silu = FG_ACT_SILU, gelu = FG_ACT_GELU_TANH;

  EXPECT(int8_cast_per_row(S, 512, Q, P, -1, 512, nullptr), FG_EINVAL);
  EXPECT(int8_cast_per_row(S, 512, Q, P, 4, 500, nullptr), FG_EALIGN);
  EXPECT(int8_cast_per_row(S, 500, Q, P, 4, 512, nullptr), FG_EINVAL);
  EXPECT(int8_cast_per_row(S, 513, Q, P, 4, 512, nullptr), FG_EALIGN);
  EXPECT(int8_cast_per_row(nullptr, 512, Q, P, 4, 512, nullptr), FG_EINVAL);
  EXPECT(int8_cast_per_row(nullptr, 0, nullptr, nullptr, 0, 512, nullptr), FG_OK);
  EXPECT(int8_cast_per_row_bf16(X, 516, Q, P, 4, 512, nullptr), FG_EALIGN);
  EXPECT(int8_cast_per_row_bf16(X, 512, nullptr, P, 4, 512, nullptr), FG_EINVAL);

  // shapes of every plan, as far as the device query
  const int sizes[] = {1, 7, 16, 17, 64, 127, 333, 640, 641, 1000, 4096, 100000, rows / 2};
  const int depths[] = {0, 16, 2048, 65536, 131056};
  for (const int M : sizes)
    for (const int N : sizes)
      for (const int K : depths) {
        EXPECT(gemm_int8_nt(A, 131056, S, A, 131056, S, D, N, M, N, K, nullptr), FG_EHIP);
        EXPECT(gated_ffn_int8(A, 131056, S, A, 131056, S, D, N, M, N, K, silu, nullptr), FG_EHIP);
        EXPECT(gated_ffn_bf16(X, 131056, X, 131056, D, N, nullptr, 0, M, N, K, gelu, nullptr), FG_EHIP);
        EXPECT(gated_ffn_bf16(X, 131056, X, 131056, D, N, P, 2 * (int64_t)N, M, N, K, gelu, nullptr), FG_EHIP);
        const int64_t need = fg_gated_ffn_backward_workspace_bytes(M, N, K);
        if (need < 0 && N <= rows / 4) ++g_fail;
        if (K > 0 && N <= 100000)
          EXPECT(gated_ffn_bf16_backward(X, N, X, 131056, X, 131056, nullptr, 0, D, K, D, K, M, N, K, silu, WS, need,
                                         nullptr),
                 FG_EHIP);
      }
  EXPECT(gemm_int8_nt(A, 512, S, A, 512, S, D, 64, 64, 64, 131072, nullptr), FG_EUNSUPPORTED);
  EXPECT(gemm_int8_nt(A, 512, S, A, 512, S, D, 64, 64, 64, 500, nullptr), FG_EALIGN);
  EXPECT(gemm_int8_nt(A, 520, S, A, 512, S, D, 64, 64, 64, 512, nullptr), FG_EALIGN);
  EXPECT(gemm_int8_nt(A, big, S, A, 512, S, D, 64, 64, 64, 512, nullptr), FG_EUNSUPPORTED);
  EXPECT(gemm_int8_nt(A, 512, S, A, 512, S, D, 64, top, 64, 512, nullptr), FG_EUNSUPPORTED);
  EXPECT(gemm_int8_nt(A, 512, S, A, 512, S, D, 63, 64, 64, 512, nullptr), FG_EINVAL);
  EXPECT(gemm_int8_nt(nullptr, 0, nullptr, nullptr, 0, nullptr, nullptr, 0, 0, 64, 512, nullptr), FG_OK);
  EXPECT(gated_ffn_int8(A, 512, S, A, 512, S, D, 64, 64, 64, 512, 2, nullptr), FG_EINVAL);
  EXPECT(gated_ffn_int8(A, 512, S, A, 512, nullptr, D, 64, 64, 64, 512, silu, nullptr), FG_EINVAL);
  EXPECT(gated_ffn_int8(A, 512, S, A, 512, S, D, 64, 64, rows, 512, silu, nullptr), FG_EUNSUPPORTED);
  EXPECT(gated_ffn_bf16(X, 512, X, 512, D, 64, P, 127, 64, 64, 512, silu, nullptr), FG_EINVAL);
  EXPECT(gated_ffn_bf16(X, 512, X, 512, D, 64, nullptr, 0, 64, 64, 508, silu, nullptr), FG_EALIGN);
  EXPECT(gated_ffn_bf16(X, 512, X, 512, D, 64, nullptr, 0, -1, 64, 512, silu, nullptr), FG_EINVAL);

  const int64_t need = fg_gated_ffn_backward_workspace_bytes(64, 64, 512);
  EXPECT(gated_ffn_bf16_backward(X, 64, X, 512, X, 512, nullptr, 0, D, 512, D, 512, 64, 64, 512, silu, WS, need - 1,
                                 nullptr),
         FG_EINVAL);
  EXPECT(gated_ffn_bf16_backward(X, 64, X, 512, X, 512, nullptr, 0, D, 512, D, 512, 64, 64, 512, silu,
                                 (void*)0x10010, big, nullptr),
         FG_EALIGN);
  EXPECT(gated_ffn_bf16_backward(X, 64, X, 512, X, 512, nullptr, 0, D, 512, D, 512, 64, 64, 512, 7, WS, need, nullptr),
         FG_EINVAL);
  EXPECT(gated_ffn_bf16_backward(X, 64, X, 512, X, 512, nullptr, 0, D, 512, D, 512, 64, rows, 512, silu, WS, big,
                                 nullptr),
         FG_EUNSUPPORTED);
  EXPECT(gated_ffn_bf16_backward(X, rows / 4, X, 512, X, 512, nullptr, 0, D, 512, D, 512, 64, rows / 4, 512, silu, WS,
                                 big, nullptr),
         FG_EUNSUPPORTED);
  EXPECT(gated_ffn_bf16_backward(nullptr, 0, nullptr, 0, nullptr, 0, nullptr, 0, nullptr, 0, nullptr, 0, 64, 64, 512,
                                 silu, nullptr, 0, nullptr),
         FG_OK);
  EXPECT(gated_ffn_bf16_backward(X, 64, X, 512, X, 512, P, 127, D, 512, D, 512, 64, 64, 512, silu, WS, need, nullptr),
         FG_EINVAL);
  if (fg_gated_ffn_backward_workspace_bytes(-1, 1, 1) != -1 || fg_gated_ffn_backward_workspace_bytes(top, 1, 1) != -1)
    ++g_fail;
  if (fg_gated_ffn_backward_workspace_bytes(rows, rows / 4, rows) < ((int64_t)1 << 59)) ++g_fail;

  if (g_fail) {
    std::fprintf(stderr, "%d check(s) failed\n", g_fail);
    return 1;
  }
  std::printf("host linear ok\n");
  return 0;
}
