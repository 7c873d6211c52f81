// linear_plan.hpp -- which kernels a call of the 8-bit-integer products and the
// gated feed-forward block launches.  Host arithmetic alone: it needs no
// device and no HIP, so the sanitizer tests run it over sizes and CU counts.
//
// Each candidate's time is estimated from its tiles and slices with costs
// measured on MI355X (256 CUs; microseconds, a call in a HIP graph; int8 and
// bf16 slices cost the same, both are 128 bytes and 2048 MFMA cycles on the 256
// x 256 tile), and the cheapest runs.  The estimates only rank candidates: fitted to 700 random
// products and 150 gradients, on others the choice is 2 % (gradients 1 %)
// slower than the fastest tile on average.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

namespace fg {

constexpr int kPairAlign = 64;  // columns of each half of the gradient pair

inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Slices of a reduction over K values of `item` bytes.
inline int slice_count(int64_t K, int item) { return (int)std::max<int64_t>(1, (K * item + 127) / 128); }

// A matrix product as the plans see it.
struct Product {
  int64_t M, cols;  // the output; gated: cols hidden units, each of two weight rows
  int nk;           // slices of the reduction
  bool gated;
  bool mn;  // an operand, or both, MN-major
};

enum TileKind { kW256, kW224, kW192, kW160, kMid2, kMid, kHalf2, kSmall2, kSmall };
struct TilePlan {
  TileKind kind;
  double us;
};

// Output tiles of bm rows and bn weight rows.
inline double tile_count(const Product& p, int bm, int bn) {
  const int out_n = p.gated ? bn / 2 : bn;
  return (double)((p.M + bm - 1) / bm) * (double)((p.cols + out_n - 1) / out_n);
}

// One tile per CU and round: `idle` a slice with few CUs at work, `busy` with
// all of them (clock and cache contention, which sets in towards the end),
// `store` for the epilogue.
inline double tile_us(double tiles, int cus, int nk, double idle, double busy, double store) {
  const double load = tiles < cus ? tiles / cus : 1.0;
  return 3.4 + ceil(tiles / cus) * (nk * (idle + (busy - idle) * load * load) + store);
}

// Two workgroups to a CU: `idle` to `one` a slice while every CU has at most
// one, `two` for both.
inline double pairs_us(double tiles, int cus, int nk, double idle, double one, double two, double store) {
  const double full = floor(tiles / (2 * cus)), rest = tiles - full * 2 * cus, load = rest / cus;
  double us = 3.4 + full * (nk * two + store);
  if (rest > 0) us += nk * (rest > cus ? two : idle + (one - idle) * load * load) + store;
  return us;
}

// The tiles below 256 rows, with their times a slice where both operands are
// K-major and where one or both are MN-major (mn).
//
// 64 x 64, eight waves, for few tiles: in two groups (256 x 4096 x 7168 int8 15
// us, 25 on 128 x 128); where operands are MN-major in one, so that every sum
// of a gradient runs in the order of its slices and its bits depend on nothing
// but the split.  There it serves splits and shared launches alone: two
// workgroups of four waves are as fast with few tiles and faster with many.
inline double small_us(double tiles, int cus, int nk, bool mn) {
  return mn ? tile_us(tiles, cus, nk, 0.28, 0.35, 1.2) : tile_us(tiles, cus, nk, 0.177, 0.19, 1.5);
}

// 64 x 64, two workgroups of four waves, where tiles outnumber the CUs (320 x
// 4096 x 1024 int8 6.1 us, 8.3 on eight waves; dX 600 x 1528 x 2048 with the
// pair's pass 18.4 us, 20.7 on 128 x 64).
inline double small2_us(double tiles, int cus, int nk, bool mn) {
  return mn ? pairs_us(tiles, cus, nk, 0.22, 0.32, 0.68, 1.3) : pairs_us(tiles, cus, nk, 0.187, 0.19, 0.54, 1.25);
}

// 128 x 64, two workgroups of eight waves (512 x 4096 x 7168 int8 22 us, 25 on
// 128 x 128 and on 64 x 64; gated bf16 333 x 1056 x 1528 11 us, 17 on 128 x 128).
inline double half2_us(double tiles, int cus, int nk, bool mn) {
  return mn ? pairs_us(tiles, cus, nk, 0.30, 0.39, 0.75, 1.7) : pairs_us(tiles, cus, nk, 0.23, 0.30, 0.66, 1.9);
}

// 128 x 128, eight waves, four stages (1000 x 4096 x 7168 int8 32 us, 70 on
// 256 x 256; rows half a line off, 36).
inline double mid_us(double tiles, int cus, int nk, bool mn) {
  return mn ? tile_us(tiles, cus, nk, 0.46, 0.53, 2.0) : tile_us(tiles, cus, nk, 0.44, 0.51, 2.4);
}

// 128 x 128, two workgroups of four waves (dW 2816 x 2048 x 1500 with the pair's
// pass 33 us, 40 on eight waves).
inline double mid2_us(double tiles, int cus, int nk, bool mn) {
  return mn ? pairs_us(tiles, cus, nk, 0.80, 0.80, 0.90, 1.5) : pairs_us(tiles, cus, nk, 0.70, 0.70, 0.90, 1.5);
}

// `forced` overrides a choice (the environment variable FG_LINEAR_PLAN, for
// tuning and tests): a tile ("w256", "w224", "w192", "w160", "mid2", "mid", "half2",
// "small2", "small"), a few-row shape ("few0" .. "few7"), or for the gradients
// "split-mid", "split-small" (dX's sum), "pair" (the recomputed
// pre-activations' sums) or "share-X-W" (X and W: mid or small).  A plan that
// the call does not have leaves it its own.
inline bool forced_tile(const char* f, const Product& p, TileKind* kind) {
  static const struct {
    const char* name;
    TileKind kind;
  } names[] = {{"w256", kW256}, {"w224", kW224}, {"w192", kW192}, {"w160", kW160},
               {"mid2", kMid2}, {"mid", kMid},   {"half2", kHalf2}, {"small2", kSmall2}, {"small", kSmall}};
  for (const auto& n : names) {
    if (strcmp(f, n.name) != 0) continue;
    *kind = n.kind;
    return (p.gated ? n.kind != kW224 && n.kind != kW160 : n.kind != kW192) && !(p.mn && n.kind == kSmall);
  }
  return false;
}

inline bool shares(const char* forced, TileKind x, TileKind w) {
  char name[32];
  snprintf(name, sizeof name, "share-%s-%s", x == kMid ? "mid" : "small", w == kMid ? "mid" : "small");
  return strcmp(forced, name) == 0;
}

// The cheapest tile for p and its time.
inline TilePlan plan_tile(const Product& p, int cus, const char* forced) {
  TileKind kind;
  if (forced_tile(forced, p, &kind)) return TilePlan{kind, 0.0};
  auto count = [&](int bm, int bn) { return tile_count(p, bm, bn); };
  const bool mn = p.mn;
  TilePlan best{kW256, 1e30};
  auto offer = [&](TileKind kind, double us) {
    if (us < best.us) best = TilePlan{kind, us};
  };
  // 256 rows by 256, 224, 192 or 160: the time of a slice grows with the CUs at
  // work, since the chip's power limits these (int8 4096 x 7168 x 16384: 374 us
  // with 256 columns, 346 with 224; 4096 x 2112 x 7168: 71 with 256, 60 with
  // 160; gated bf16 4096 x 12288 x 1536: 227 with 256, 242 with 192; 1500 x 6000
  // x 3008: 122 and 107.  Between these two the choice is within 1 % of the
  // better on 17 gated shapes, bf16 and int8, of 1000 to 8192 rows, 1536 to
  // 14336 units and reductions of 1024 to 7168).
  offer(kW256, tile_us(count(256, 256), cus, p.nk, 1.2, mn ? 1.3 : 1.45, 4.0));
  if (p.gated) {
    offer(kW192, tile_us(count(256, 192), cus, p.nk, 0.95, 1.15, 4.0));
  } else {
    offer(kW224, tile_us(count(256, 224), cus, p.nk, 1.1, mn ? 1.22 : 1.36, 4.0));
    offer(kW160, tile_us(count(256, 160), cus, p.nk, 0.92, mn ? 0.92 : 1.02, 3.5));
  }
  offer(kMid2, mid2_us(count(128, 128), cus, p.nk, mn));
  offer(kHalf2, half2_us(count(128, 64), cus, p.nk, mn));
  offer(kSmall2, small2_us(count(64, 64), cus, p.nk, mn));
  offer(kMid, mid_us(count(128, 128), cus, p.nk, mn));
  if (!mn) offer(kSmall, small_us(count(64, 64), cus, p.nk, mn));
  return best;
}

// Few-row shapes: 16 mf rows, 16 cf weight rows, waves.  A wave's step of one
// slice takes `idle` to `busy` us by how many CUs are at work; workgroups that
// share a CU take `shared` of their time one after the other.  Fitted to 870
// shapes (1 to 640 rows, 64 to 12000 columns, rows of 256 bytes to 15 KiB,
// int8 and gated bf16): on 300 others the choice, tiles included, is 1 %
// slower than the fastest on average, 45 % at worst.
struct FewRowShape {
  int mf, cf, waves;
  double base, idle, busy, shared;
};
constexpr FewRowShape kFewRowShapes[] = {
    {1, 1, 4, 1.20, 0.17, 0.32, 1.00}, {1, 1, 8, 1.47, 0.26, 0.55, 0.70}, {1, 2, 4, 1.15, 0.21, 0.49, 0.73},
    {2, 1, 4, 1.57, 0.29, 0.36, 0.91}, {2, 2, 4, 1.50, 0.25, 0.54, 0.82}, {4, 1, 4, 2.00, 0.31, 0.47, 1.04},
    {4, 2, 4, 1.80, 0.38, 0.80, 1.09}, {4, 4, 4, 1.75, 1.29, 1.29, 1.32},
};
constexpr int kFewRowShapeCount = sizeof kFewRowShapes / sizeof *kFewRowShapes;
constexpr int kFewRowMost = 640;  // rows up to which these shapes are considered
// Workgroups up to which they are: a grid of 512 threads each stays below 2^32
// threads.  Wider outputs are the tiles', whose grid is persistent.
constexpr int kFewRowMostGroups = (1 << 23) - 1;

// Workgroups of few-row shape f.
inline double fewrow_groups(const Product& p, const FewRowShape& f) {
  return (double)((p.M + 16 * f.mf - 1) / (16 * f.mf)) * ceil((double)p.cols / (p.gated ? 8 * f.cf : 16 * f.cf));
}

inline double fewrow_us(const Product& p, int cus, const FewRowShape& f) {
  const double groups = fewrow_groups(p, f);
  const double load = groups < cus ? groups / cus : 1.0, turns = ceil(groups / cus);
  const double one = 0.9 + (p.nk + f.waves - 1) / f.waves * (f.idle + (f.busy - f.idle) * load);
  return f.base + (turns > 1 ? turns * f.shared : 1.0) * one;
}

inline bool forced_fewrow(const char* f, int shape) {
  return strncmp(f, "few", 3) == 0 && f[3] == '0' + shape && !f[4];
}

// A forward product: few-row shape `few`, or, where that is negative, a tile.
struct ForwardPlan {
  int few;
  TileKind tile;
};
inline ForwardPlan plan_forward(const Product& p, int cus, const char* forced) {
  const TilePlan tile = plan_tile(p, cus, forced);
  ForwardPlan plan{-1, tile.kind};
  if (p.M > kFewRowMost) return plan;
  double least = tile.us;
  for (int i = 0; i < kFewRowShapeCount; ++i) {
    if (fewrow_groups(p, kFewRowShapes[i]) > kFewRowMostGroups) continue;
    const double t = fewrow_us(p, cus, kFewRowShapes[i]);
    if (forced_fewrow(forced, i)) return ForwardPlan{i, tile.kind};
    if (t < least) {
      least = t;
      plan.few = i;
    }
  }
  return plan;
}

// Splits of the reduction over workgroups, in the backward pass: of dX's sum
// over 2F, and of the recomputed pre-activations' over K.  The fp32 partials
// of at most kMaxSplits splits and kMaxPartialBytes go to the workspace and
// the next launch adds them.
constexpr int kMaxSplits = 16;
constexpr int64_t kMaxPartialBytes = (int64_t)32 << 20;

// Workspace bytes for the partials of an M x N output: none where fewer than
// two fit.
inline int64_t partial_bytes(int64_t M, int64_t N) {
  const int64_t one = M * N * 4;
  if (one > kMaxPartialBytes / 2) return 0;
  return round_up(std::min<int64_t>(kMaxSplits, kMaxPartialBytes / one) * one, 256);
}

// Splits of p's reduction on bm x bm tiles, with partials of `one` bytes.
struct SplitPlan {
  double us;
  int splits, nk;  // slices of a split (even)
};

template <class F>
SplitPlan plan_split(const Product& p, int64_t one, int cus, int bm, F cost) {
  const double tiles = tile_count(p, bm, bm);
  SplitPlan s{1e30, 1, p.nk};
  if (one > kMaxPartialBytes / 2 || tiles > cus / 2) return s;
  const int most = (int)std::min<int64_t>(std::min<int64_t>(kMaxSplits, kMaxPartialBytes / one), (int64_t)(cus / tiles));
  s.nk = (int)round_up((p.nk + most - 1) / most, 2);
  s.splits = (p.nk + s.nk - 1) / s.nk;
  // the partials are written and read at about 4 TB/s; the second launch is 2.3 us
  s.us = cost(tiles * s.splits, cus, s.nk, p.mn) + 2.3 + 2.0 * s.splits * one / 4e6;
  return s;
}

// Bytes of the pre-activations' partials: none where 64 x 64 tiles (32 hidden
// units) already take more than a third of 256 CUs.
constexpr int kMaxPairTiles = 85;
inline int64_t pair_partial_bytes(int64_t M, int64_t cols) {
  return (M + 63) / 64 * (cols / 64) > kMaxPairTiles ? 0 : partial_bytes(M, cols);
}

// Columns of the gradient pair [dg du], its bytes, and those of the backward
// pass's workspace: the pair, then partials.
inline int64_t pair_cols(int64_t F) { return 2 * round_up(F, kPairAlign); }
inline int64_t pair_bytes(int64_t M, int64_t F) { return round_up(M * pair_cols(F) * 2, 256); }
inline int64_t backward_bytes(int64_t M, int64_t F, int64_t K) {
  return pair_bytes(M, F) + std::max(partial_bytes(M, K), pair_partial_bytes(M, pair_cols(F)));
}

// Splits of the recomputed pre-activations' sum (one where it stays whole) for
// a gradient pair of M rows, K values a row, g its product.
inline SplitPlan plan_recompute(const Product& g, int cus, const char* forced) {
  SplitPlan s{0.0, 1, g.nk};
  if (pair_partial_bytes(g.M, 2 * g.cols) == 0) return s;
  const SplitPlan split = plan_split(g, g.M * g.cols * 8, cus, 64, small_us);
  const bool take = strcmp(forced, "pair") == 0 || split.us < plan_tile(g, cus, forced).us;  // (a forced tile's is 0)
  return split.splits > 1 && take ? split : s;
}

// dX = pair . W and dW = pair^T . X.  Each has its own plan; where neither
// fills the device, both go into one launch, with 128 x 128 or 64 x 64 tiles
// each.  That launch has a workgroup for every tile, which the device takes as
// CUs become free, so it is not for a call that may use some of the CUs only
// (`capped`): the persistent launches of their own keep to them.
struct GradsPlan {
  bool shared;
  TileKind x, w;
  int splits, split_nk;  // of dX's sum: the splits and their slices
};
inline GradsPlan plan_grads(const Product* x, const Product* w, int cus, bool capped, const char* forced) {
  GradsPlan plan{false, kW256, kW256, 1, 0};
  bool separate = false;  // a forced plan of a launch for each
  double x_us = 0, w_us = 0;
  if (x) {
    plan.split_nk = x->nk;
    const TilePlan t = plan_tile(*x, cus, forced);
    plan.x = t.kind;
    x_us = t.us;
    separate = t.us == 0;
    // 251 x 1016 with 178 slices, with the pair's pass: 55 us on 64 64 x 64
    // tiles, a quarter of the device; split 25 us with the addition.
    const int64_t one = x->M * x->cols * 4;
    const SplitPlan a = plan_split(*x, one, cus, 64, small_us);
    const SplitPlan b = plan_split(*x, one, cus, 128, mid_us);
    const bool force_small = strcmp(forced, "split-small") == 0, force_mid = strcmp(forced, "split-mid") == 0;
    const bool small_tiles = force_small || (!force_mid && a.us <= b.us);
    const SplitPlan& s = small_tiles ? a : b;
    if (s.splits > 1 && (s.us < x_us || force_small || force_mid)) {
      plan.x = small_tiles ? kSmall : kMid;
      plan.splits = s.splits;
      plan.split_nk = s.nk;
      x_us = s.us;
      separate = force_small || force_mid;
    }
  }
  if (w) {
    const TilePlan t = plan_tile(*w, cus, forced);
    plan.w = t.kind;
    w_us = t.us;
  }
  if (!x || !w || separate || capped) return plan;
  // One launch: the workgroups of both, one to a CU, dX's first.  The device
  // is busy for their total, and for the longest one at least.
  const GradsPlan own = plan;
  double least = x_us + w_us;
  for (const TileKind cx : {kMid, kSmall})
    for (const TileKind cw : {kMid, kSmall}) {
      if (own.splits > 1 && cx != own.x) continue;
      const int bx = cx == kMid ? 128 : 64, bw = cw == kMid ? 128 : 64;
      const double nx = tile_count(*x, bx, bx) * own.splits, nw = tile_count(*w, bw, bw);
      const double tx = own.split_nk * (cx == kMid ? 0.57 : 0.45) + (cx == kMid ? 2.5 : 1.5);
      const double tw = w->nk * (cw == kMid ? 0.63 : 0.37) + (cw == kMid ? 2.5 : 1.5);  // both operands MN-major
      const double us = 3.4 + std::max(std::max(tx, tw), (nx * tx + nw * tw) / cus + 0.5 * std::min(tx, tw)) +
                        (own.splits > 1 ? 4.0 : 0.0);
      if (nx + nw >= (1 << 22)) continue;
      const GradsPlan both{true, cx, cw, own.splits, own.split_nk};
      if (shares(forced, cx, cw)) return both;
      if (us < least) {
        least = us;
        plan = both;
      }
    }
  return plan;
}

}  // namespace fg
