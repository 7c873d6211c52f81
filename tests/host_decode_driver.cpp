// host_decode_driver.cpp -- drives the C entry points of the router, the 4-bit
// cast and product and the few-token expert layers through their host code, for a
// build with AddressSanitizer and UndefinedBehaviorSanitizer
// (tests/test_host_decode.py).
//
// No GPU is needed: every call fails a host check, is an empty problem, or stops
// at the first HIP call (FG_EHIP without a device).  Pointers are fake device
// addresses that are never dereferenced.  Exit status 0 and "host decode ok" mean
// that every status matched.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

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
  float* S = reinterpret_cast<float*>(0x10000);
  uint16_t* X = reinterpret_cast<uint16_t*>(0x10000);
  uint8_t* Q = reinterpret_cast<uint8_t*>(0x10000);
  int32_t* I = reinterpret_cast<int32_t*>(0x10000);
  void* WS = reinterpret_cast<void*>(0x10000);
  const int64_t big = (int64_t)1 << 60;
  const int top = 0x7fffffff, silu = FG_ACT_SILU, soft = FG_SCORE_SOFTMAX;

  // router: every number of experts' kernel, the largest sizes
  const int counts[] = {1, 64, 65, 128, 200, 256, 257, 512, 1000, 1024};
  for (const int E : counts)
    for (const int T : {1, 5, 1 << 25})
      for (int sigmoid = 0; sigmoid < 2; ++sigmoid) {
        EXPECT(moe_route(S, big, nullptr, I, S, T, E, 1, sigmoid, 1, 1, 1, 1.f, nullptr), FG_EHIP);
        EXPECT(moe_route_bf16(X, E, S, I, S, T, E, E < 64 ? E : 64, sigmoid, 1, 1, 0, 1.f, nullptr), FG_EHIP);
        EXPECT(moe_route_backward(S, S, E, I, S, big, T, E, 1, sigmoid, 1, 1.f, nullptr), FG_EHIP);
        EXPECT(moe_route_backward_bf16(S, X, E, I, X, E, T, E, 1, sigmoid, 0, 1.f, nullptr), FG_EHIP);
      }
  EXPECT(moe_route(S, 8, nullptr, I, S, (1 << 25) + 1, 8, 1, soft, 1, 1, 1, 1.f, nullptr), FG_EUNSUPPORTED);
  EXPECT(moe_route(S, top, nullptr, I, S, top, top, top, soft, top, top, 1, 1.f, nullptr), FG_EUNSUPPORTED);
  EXPECT(moe_route(S, 8, nullptr, I, S, -top - 1, 8, 1, soft, 1, 1, 1, 1.f, nullptr), FG_EINVAL);
  EXPECT(moe_route_backward(S, S, -big, I, S, 8, 1, 8, 1, soft, 1, 1.f, nullptr), FG_EINVAL);

  // 4-bit cast and product: every format and plan, the largest sizes
  const int groups[] = {32, 64, 128, 384, 1 << 20, top / 128 * 128};
  for (const int g : groups)
    for (const int K : {32, 96, 2048, 1 << 20})
      for (const int N : {1, 17, 4096, 1 << 26}) {
        EXPECT(int4_cast_per_group(S, big, Q, X, Q, N, K, g, nullptr), FG_EHIP);
        EXPECT(int4_cast_per_group_bf16(X, 1 << 20, Q, X, nullptr, N, K, g, nullptr), FG_EHIP);
        for (const int M : {1, 2, 3, 8, 16, 17, 64, 1 << 20}) {
          const int64_t need = fg_int4_workspace_bytes(M, N, K);
          if (need < 0) ++g_fail;
          EXPECT(gemm_int4_nt(X, 1 << 21, Q, X, Q, X, big, M, N, K, g, need ? WS : nullptr, need, nullptr), FG_EHIP);
          EXPECT(gemm_int4_nt(X, 1 << 21, Q, X, nullptr, X, N, M, N, K, g, WS, big, nullptr), FG_EHIP);
          if (need) EXPECT(gemm_int4_nt(X, 1 << 21, Q, X, Q, X, N, M, N, K, g, WS, need - 1, nullptr), FG_EINVAL);
        }
      }
  EXPECT(int4_cast_per_group(S, big, Q, X, Q, top, top / 32 * 32, 32, nullptr), FG_EUNSUPPORTED);
  EXPECT(gemm_int4_nt(X, 1 << 21, Q, X, Q, X, big, top, top, top / 32 * 32, 32, WS, big, nullptr), FG_EUNSUPPORTED);
  if (fg_int4_workspace_bytes(top, 1, 32) != -1 || fg_int4_workspace_bytes(-1, 1, 32) != -1) ++g_fail;

  // layers.  With no hidden units the first kernel is left out and `down` is the
  // first to need a device, after the check that its LDS fits: FG_EUNSUPPORTED
  // there would be a plan that does not.
  const char* plans[] = {"", "down-split1", "down-split1-two", "down-split4", "down-split4-two", "down-wide16",
                         "down-wide16-deep", "down-wide32"};
  for (const char* plan : plans) {
    setenv("FG_DECODE_PLAN", plan, 1);
    for (const int T : {1, 2, 4, 7, 8, 16, 17, 63, 64, 65, 1 << 20})
      for (const int k : {1, 2, 8, 32})
        for (const int E : {1, 3, 16, 64, 200, 1024})
          for (const int K : {32, 2048, 4128, 65536}) {
            const int64_t need = fg_moe_ffn_workspace_bytes(T, k, 0);
            const int a = moe_ffn_fp8(X, 1 << 21, nullptr, nullptr, nullptr, nullptr, I, S, X, K, T, k, E, 0, K, silu, WS, need, nullptr);
            const int b = moe_ffn_int4(X, K, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, I, S, X, big, T, k, E, 0, K, 32,
                                       silu, WS, need, nullptr);
            // forced plans may not fit: they are refused before a launch
            const bool ok = *plan ? (a == FG_EHIP || a == FG_EUNSUPPORTED) && (b == FG_EHIP || b == FG_EUNSUPPORTED)
                                  : a == FG_EHIP && b == FG_EHIP;
            if (!ok && ++g_fail < 20) std::fprintf(stderr, "T=%d k=%d E=%d K=%d plan '%s': %d %d\n", T, k, E, K, plan, a, b);
          }
  }
  setenv("FG_DECODE_PLAN", "", 1);
  for (const int T : {1, 5, 64, 1 << 20})
    for (const int F : {32, 704, 65536}) {
      const int64_t need = fg_moe_ffn_workspace_bytes(T, 32, F);
      EXPECT(moe_ffn_fp8(X, 1 << 21, Q, S, Q, S, I, S, X, 65536, T, 32, 1024, F, 65536, silu, WS, need, nullptr), FG_EHIP);
      EXPECT(moe_ffn_fp8(X, 1 << 21, Q, S, Q, S, I, S, X, 65536, T, 32, 1024, F, 65536, silu, WS, need - 1, nullptr), FG_EINVAL);
      EXPECT(moe_ffn_int4(X, 1 << 21, Q, X, Q, Q, X, Q, I, S, X, 65536, T, 32, 1024, F, 65536, 64, silu, WS, big, nullptr), FG_EHIP);
      EXPECT(moe_ffn_int4(X, 1 << 21, Q, X, Q, Q, X, nullptr, I, S, X, 65536, T, 32, 1024, F, 65536, 64, silu, WS, big, nullptr),
             FG_EINVAL);
    }
  EXPECT(moe_ffn_fp8(X, big, Q, S, Q, S, I, S, X, big, top, top, top, top / 16 * 16, top / 16 * 16, silu, WS, big, nullptr),
         FG_EUNSUPPORTED);
  if (fg_moe_ffn_workspace_bytes(top, 32, 32) != -1 || fg_moe_ffn_workspace_bytes(1, 33, 32) != -1) ++g_fail;

  if (g_fail) return std::fprintf(stderr, "%d wrong\n", g_fail), 1;
  std::printf("host decode ok\n");
  return 0;
}
