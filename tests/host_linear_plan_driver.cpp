// host_linear_plan_driver.cpp -- runs the plans of the 8-bit-integer products
// and the gated block (csrc/linear_plan.hpp) over sizes and CU counts, for a
// build with AddressSanitizer and UndefinedBehaviorSanitizer
// (tests/test_linear_plan_host.py).  No GPU and no HIP.  Exit status 0 and
// "host plans ok" mean that every plan kept its limits.
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "linear_plan.hpp"

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

static const char* const kForced[] = {"", "w256", "w224", "w192", "w160", "mid2", "mid", "half2", "small2", "small",
                                      "few0", "few7", "split-mid", "split-small", "pair", "share-mid-mid",
                                      "share-mid-small", "share-small-mid", "share-small-small", "few8", "none", "split",
                                      "a name longer than any plan's, which fits no buffer made for one"};

// A forced plan that a call does not have leaves it its own.
static const char* const kNotGrads[] = {"small", "w192", "few0", "few7", "few8", "pair", "none", "split"};
static const char* const kNotPair[] = {"w224", "w160", "few0", "few7", "few8", "split-mid", "share-mid-mid", "none", "split"};
static const char* const kNotInt8[] = {"w192", "few8", "pair", "split-mid", "share-mid-mid", "none", "split"};

static bool same(const GradsPlan& a, const GradsPlan& b) {
  return a.shared == b.shared && a.x == b.x && a.w == b.w && a.splits == b.splits && a.split_nk == b.split_nk;
}

// What is true of every split of `nk` slices into partials of `one` bytes, in
// a workspace of `room` bytes.
static void check_split(int splits, int split_nk, int nk, int64_t one, int64_t room, const char* what, long long M,
                        long long F, long long K, int cus) {
  CHECK(splits >= 1 && splits <= kMaxSplits, "%s %lld %lld %lld cus %d: %d splits", what, M, F, K, cus, splits);
  if (splits == 1) return;
  CHECK(split_nk % 2 == 0, "%s %lld %lld %lld cus %d: %d slices a split", what, M, F, K, cus, split_nk);
  CHECK((int64_t)splits * split_nk >= nk && (int64_t)(splits - 1) * split_nk < nk, "%s %lld %lld %lld cus %d: %d x %d of %d",
        what, M, F, K, cus, splits, split_nk, nk);
  CHECK(splits * one <= room && splits * one <= kMaxPartialBytes, "%s %lld %lld %lld cus %d: %d partials of %lld in %lld",
        what, M, F, K, cus, splits, (long long)one, (long long)room);
}

static void forward(int64_t M, int64_t N, int64_t K, bool gated, int item, int cus, const char* forced) {
  const Product p{M, N, slice_count(K, item), gated, false};
  const ForwardPlan plan = plan_forward(p, cus, forced);
  ++g_plans;
  CHECK(plan.few >= -1 && plan.few < kFewRowShapeCount, "few %d", plan.few);
  CHECK(plan.few < 0 || M <= kFewRowMost, "%lld rows", (long long)M);
  // one workgroup a tile: at most 512 threads each, below 2^32 in all
  CHECK(plan.few < 0 || fewrow_groups(p, kFewRowShapes[plan.few]) * 512 < 4294967296.0, "%lld x %lld: shape %d",
        (long long)M, (long long)N, plan.few);
  CHECK(gated ? plan.tile != kW224 && plan.tile != kW160 : plan.tile != kW192, "tile %d", plan.tile);
}

static void own_plans(int64_t M, int64_t N, int64_t K, int cus) {
  const Product a{M, N, slice_count(K, 1), false, false};
  const ForwardPlan f = plan_forward(a, cus, "");
  for (const char* forced : kNotInt8) {
    const ForwardPlan g = plan_forward(a, cus, forced);
    CHECK(f.few == g.few && f.tile == g.tile, "%s: %lld %lld %lld", forced, (long long)M, (long long)N, (long long)K);
  }
  if (K == 0 || N > 1 << 20) return;
  const int64_t cols = pair_cols(N);
  const Product g{M, cols / 2, slice_count(K, 2), true, false};
  const SplitPlan s = plan_recompute(g, cus, "");
  for (const char* forced : kNotPair) {
    const SplitPlan t = plan_recompute(g, cus, forced);
    CHECK(s.splits == t.splits && s.nk == t.nk && plan_tile(g, cus, "").kind == plan_tile(g, cus, forced).kind,
          "%s: %lld %lld %lld", forced, (long long)M, (long long)N, (long long)K);
  }
  const Product x{M, K, slice_count(cols, 2), false, true}, w{cols, K, slice_count(M, 2), false, true};
  for (int which = 1; which <= 3; ++which)
    for (const char* forced : kNotGrads)
      CHECK(same(plan_grads(which & 1 ? &x : nullptr, which & 2 ? &w : nullptr, cus, false, ""),
                 plan_grads(which & 1 ? &x : nullptr, which & 2 ? &w : nullptr, cus, false, forced)),
            "%s: %lld %lld %lld of %d", forced, (long long)M, (long long)N, (long long)K, which);
}

static void backward(int64_t M, int64_t F, int64_t K, int cus, const char* forced) {
  const int64_t cols = pair_cols(F), half = cols / 2, room = backward_bytes(M, F, K) - pair_bytes(M, F);
  const Product g{M, half, slice_count(K, 2), true, false};
  const SplitPlan s = plan_recompute(g, cus, forced);
  check_split(s.splits, s.nk, g.nk, M * cols * 4, room, "pair", M, F, K, cus);
  const Product x{M, K, slice_count(cols, 2), false, true}, w{cols, K, slice_count(M, 2), false, true};
  for (int i = 0; i < 6; ++i) {  // dX, dW, both; the same on some of the CUs only
    const int which = i % 3 + 1;
    const bool capped = i >= 3;
    const GradsPlan plan = plan_grads(which & 1 ? &x : nullptr, which & 2 ? &w : nullptr, cus, capped, forced);
    ++g_plans;
    if (which & 1) {
      check_split(plan.splits, plan.split_nk, x.nk, M * K * 4, room, "dX", M, F, K, cus);
      CHECK(plan.splits > 1 || plan.split_nk == x.nk, "%d slices", plan.split_nk);
      CHECK(plan.splits == 1 || plan.x == kMid || plan.x == kSmall, "tile %d", plan.x);
      CHECK(plan.x != kW192, "tile %d", plan.x);
    }
    CHECK(!plan.shared || (which == 3 && !capped), "one gradient alone, or a cap");
    if (plan.shared) {
      CHECK((plan.x == kMid || plan.x == kSmall) && (plan.w == kMid || plan.w == kSmall), "%d %d", plan.x, plan.w);
      const int bx = plan.x == kMid ? 128 : 64, bw = plan.w == kMid ? 128 : 64;
      CHECK(tile_count(x, bx, bx) * plan.splits + tile_count(w, bw, bw) < (1 << 22), "grid of %lld %lld %lld",
            (long long)M, (long long)F, (long long)K);
    }
  }
}

int main() {
  const int cu_counts[] = {256, 304, 64, 7, 1};
  const int64_t top = (int64_t)1 << 29;
  const int64_t rows[] = {1, 16, 17, 64, 127, 130, 333, 593, 640, 641, 1000, 4096, 100000, top, 2 * top};
  const int64_t wide[] = {1, 8, 33, 64, 65, 300, 1528, 3229, 4096, 65536, 1 << 20, 100000000, top};
  const int64_t depths[] = {0, 16, 112, 352, 1304, 4096, 16384, 131056, 1 << 21};
  for (const char* forced : kForced)
    for (const int cus : cu_counts)
      for (const int64_t M : rows)
        for (const int64_t N : wide)
          for (const int64_t K : depths) {
            if (K <= 131056) {
              forward(M, N, K, false, 1, cus, forced);
              forward(M, N, K, true, 1, cus, forced);
            }
            forward(M, N, K, true, 2, cus, forced);
            if (K > 0 && N <= 1 << 20) backward(M, N, K, cus, forced);
          }
  for (const int cus : cu_counts)
    for (const int64_t M : rows)
      for (const int64_t N : wide)
        for (const int64_t K : depths) own_plans(M, N, K, cus);
  if (g_fail) {
    std::fprintf(stderr, "%ld check(s) failed\n", g_fail);
    return 1;
  }
  std::printf("host plans ok: %ld\n", g_plans);
  return 0;
}
