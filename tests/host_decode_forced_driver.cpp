// host_decode_forced_driver.cpp -- forced plans (FG_DECODE_PLAN) of the 4-bit
// product and the few-token expert layers: one that a call does not have, or that
// does not fit it, leaves the call its own plan (csrc/decode_plan.hpp), for a build
// with AddressSanitizer and UndefinedBehaviorSanitizer (tests/test_host_decode_plans.py).
// No GPU and no HIP.  Exit status 0 and "host forced plans ok" mean that every plan did.
#include <cstdint>
#include <cstdio>
#include <string>

#include "decode_plan.hpp"

using namespace fg;

static long g_fail = 0, g_plans = 0;

#define CHECK(ok, ...)                                        \
  do {                                                        \
    if (!(ok) && ++g_fail <= 20) {                            \
      std::fprintf(stderr, "line %d: %s: ", __LINE__, #ok);   \
      std::fprintf(stderr, __VA_ARGS__);                      \
      std::fprintf(stderr, "\n");                             \
    }                                                         \
  } while (0)

int main() {
  // one or two rows come without a workspace
  for (int M : {1, 2, 3, 64, 1 << 20})
    for (int N : {1, 200, 2112, 1 << 26})
      for (int K : {32, 7168, 1 << 20})
        for (const char* kind : kInt4Names)
          for (int parts = 0; parts <= 8; ++parts) {
            const std::string w = parts ? std::string(kind) + ",kparts" + std::to_string(parts) : kind;
            const Int4Plan p = plan_int4(M, N, K, w.c_str());
            ++g_plans;
            CHECK(M > 2 || p.k_parts == 1, "%s: %d x %d x %d: %d parts", w.c_str(), M, N, K, p.k_parts);
          }
  // LDS of `down`, of what is forced and of what is not
  for (int T : {1, 2, 7, 16, 17, 25, 26, 40, 63, 64, 65, 1 << 20})
    for (int E : {1, 3, 16, 64, 200, 417, 1000, 1024})
      for (int k : {1, 2, 8, 31, 32})
        for (int K : {32, 2048, 4128, 65536})
          for (int F : {0, 32, 2048, 65536})
            for (int fp8 = 0; fp8 < 2; ++fp8) {
              const LayerPlan own = plan_layer(fp8, T, k, E, F, K, "");
              for (int d = -1; d < kDownKinds; ++d) {
                const LayerPlan p = d < 0 ? own : plan_layer(fp8, T, k, E, F, K, kDownNames[d]);
                ++g_plans;
                const int lds = down_lds(fp8, p.down, std::min(T, kLayerTokens), E, k);
                CHECK(lds <= 160 * 1024, "%s forced: T=%d E=%d k=%d K=%d fp8=%d: %s takes %d bytes", d < 0 ? "nothing" : kDownNames[d],
                      T, E, k, K, fp8, kDownNames[p.down], lds);
                CHECK(p.down == own.down || p.down == d, "%s forced, %s taken", d < 0 ? "nothing" : kDownNames[d], kDownNames[p.down]);
              }
            }
  return g_fail ? (std::fprintf(stderr, "%ld of %ld plans wrong\n", g_fail, g_plans), 1)
                : (std::printf("host forced plans ok: %ld\n", g_plans), 0);
}
