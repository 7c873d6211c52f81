// host_decode_plan_driver.cpp -- runs the plans of the 4-bit product and the
// few-token expert layers (csrc/decode_plan.hpp) over sizes and forced plans, for
// a build with AddressSanitizer and UndefinedBehaviorSanitizer
// (tests/test_host_decode.py).  No GPU and no HIP.  Exit status 0 and "host plans
// ok" mean that every plan kept its limits.
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

static void product(int M, int N, int K, const char* forced) {
  const Int4Plan p = plan_int4(M, N, K, forced);
  ++g_plans;
  CHECK(p.kind >= 0 && p.kind < kInt4Kinds, "%d %d %d: kind %d", M, N, K, p.kind);
  CHECK(p.k_parts >= 1 && p.k_parts <= 16, "%d %d %d: %d parts", M, N, K, p.k_parts);
  CHECK(p.kind >= kWide16 || p.k_parts == 1, "%d %d %d: %d parts of a kernel that has none", M, N, K, p.k_parts);
  CHECK(p.k_parts == 1 || p.k_parts <= ceil_div(K, 256), "%d %d %d: a part without a chunk", M, N, K);
  CHECK(int4_partial_bytes(M, N, p) == (p.k_parts > 1 ? (int64_t)p.k_parts * M * N * 4 : 0), "%d %d %d", M, N, K);
  if (*forced) return;
  CHECK(M > 2 || p.k_parts == 1, "%d %d %d: the Python binding brings no workspace here", M, N, K);
  // grids that a call without a forced plan has: threads in 32 bits, 2^16 row tiles
  if (p.kind >= kWide16) {
    const int rows = p.kind == kWide64 ? 64 : p.kind == kWide32 ? 32 : 16;
    CHECK(ceil_div(M, rows) <= 65535 && (int64_t)ceil_div(N, 128) * 512 <= 0xffffffffll, "%d %d %d", M, N, K);
  } else {
    const int rows = p.kind <= kSplit2Deep ? 2 : p.kind <= kSplit8Deep ? 8 : 16;
    CHECK((int64_t)ceil_div(N, 16) * ceil_div(M, rows) * 512 <= 0xffffffffll, "%d %d %d", M, N, K);
    CHECK(p.kind != kSplit2 && p.kind != kSplit2Deep ? true : M <= 2, "%d %d %d", M, N, K);
  }
}

static void layer(bool fp8, int T, int k, int E, int F, int K, const char* forced) {
  const LayerPlan p = plan_layer(fp8, T, k, E, F, K, forced);
  ++g_plans;
  CHECK(p.up >= 0 && p.up < kUpKinds && p.down >= 0 && p.down < kDownKinds, "up %d down %d", p.up, p.down);
  // kernels that the format has
  CHECK(fp8 ? p.up != kUpWide8 && p.up != kUpSplit2 : p.up != kUpWideDeep, "fp8 %d: up %d", fp8, p.up);
  CHECK(fp8 ? p.down != kDownSplit4Two : p.down != kDownWide16Deep, "fp8 %d: down %d", fp8, p.down);
  CHECK(wide_down(p.down) || p.parts == 1, "down %d: %d parts", p.down, p.parts);
  const int pass = std::min(T, kLayerTokens);
  const int64_t need = p.parts > 1 ? (int64_t)p.parts * pass * K * 4 : 0;
  CHECK(p.parts >= 1 && p.parts <= 65535 && hidden_bytes(T, k, F) + need <= layer_bytes(T, k, F),
        "T=%d k=%d E=%d F=%d K=%d: %d parts", T, k, E, F, K, p.parts);
  CHECK(hidden_bytes(T, k, F) % 256 == 0 && hidden_bytes(T, k, F) >= (int64_t)T * k * F * 4, "T=%d k=%d F=%d", T, k, F);
}

int main() {
  const int rows[] = {1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 63, 64, 65, 1000, 1 << 20};
  const int columns[] = {1, 15, 16, 17, 127, 1000, 2112, 4096, 4097, 24576, 1 << 20, 1 << 26};
  const int depths[] = {0, 32, 224, 256, 288, 1536, 2048, 7168, 16384, 1 << 20};
  std::string words[] = {"", "no such plan", "wide16,kparts9", "kparts0", "kparts", ",", "split", "up-split", "one-part"};
  for (int M : rows)
    for (int N : columns)
      for (int K : depths) {
        for (const std::string& w : words) product(M, N, K, w.c_str());
        for (const char* kind : kInt4Names)
          for (int n = 0; n <= 8; ++n) {
            const std::string w = n ? std::string(kind) + ",kparts" + std::to_string(n) : kind;
            const Int4Plan p = plan_int4(M, N, K, w.c_str());
            CHECK(std::string(kInt4Names[p.kind]) == kind, "%s", w.c_str());
            product(M, N, K, w.c_str());
          }
      }
  const int tokens[] = {1, 2, 3, 4, 5, 8, 9, 16, 17, 64, 65, 130, 1 << 20};
  const int experts[] = {1, 2, 7, 16, 64, 256, 1000, 1024};
  const int choices[] = {1, 2, 8, 31, 32};
  const int widths[] = {0, 16, 32, 704, 2048, 7168, 1 << 16};
  for (int T : tokens)
    for (int E : experts)
      for (int k : choices)
        for (int F : widths)
          for (int K : widths) {
            if (K == 0) continue;
            for (int fp8 = 0; fp8 < 2; ++fp8) {
              for (const std::string& w : words) layer(fp8, T, k, E, F, K, w.c_str());
              for (const char* up : kUpNames) layer(fp8, T, k, E, F, K, up);
              for (const char* down : kDownNames) {
                layer(fp8, T, k, E, F, K, down);
                layer(fp8, T, k, E, F, K, (std::string("one-part,") + down).c_str());
              }
            }
          }
  if (g_fail) return std::fprintf(stderr, "%ld of %ld plans wrong\n", g_fail, g_plans), 1;
  std::printf("host plans ok: %ld\n", g_plans);
  return 0;
}
