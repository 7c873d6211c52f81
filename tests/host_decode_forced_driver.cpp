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
  return g_fail ? (std::fprintf(stderr, "%ld of %ld plans wrong\n", g_fail, g_plans), 1)
                : (std::printf("host forced plans ok: %ld\n", g_plans), 0);
}
