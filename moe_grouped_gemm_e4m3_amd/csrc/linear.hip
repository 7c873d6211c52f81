// linear.hip -- C entry points of the 8-bit-integer products and the gated
// feed-forward block (linear_kernel.hpp): argument checks, plans, launches.
// Nothing is launched after a failed check; nothing is allocated.

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "host_common.hpp"
#include "linear_fewrow.hpp"

#define FG_TRY(x)                   \
  do {                              \
    fg_status st__ = (x);           \
    if (st__ != FG_OK) return st__; \
  } while (0)

namespace fg {
namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxRowBytes = (int64_t)1 << 22;  // buffer offsets inside a tile are 32-bit
// |sum| <= 128 * 128 * K must stay below 2^31
constexpr int kMaxInt8K = (1 << 17) - 16;
constexpr int kPairAlign = 64;  // columns of each half of the gradient pair

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

fg_status launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return set_error(FG_EHIP, "%s launch: %s", what, hipGetErrorString(e));
  return FG_OK;
}

// ---------------------------------------------------------------------------
// Plans.  Each candidate's time is estimated from its tiles and slices with
// costs measured on MI355X (256 CUs; microseconds; int8 and bf16 slices cost
// the same, both are 128 bytes and 2048 MFMA cycles on the 256 x 256 tile),
// and the cheapest runs.  The estimates only rank candidates: fitted to 700
// random products and 150 gradients, on others the choice is 2 % (gradients 1 %)
// slower than the fastest tile on average.

// Lays p's output out in C's tiles (`splits` times over).
template <class C>
fg_status set_tiles(LinearParams& p, int64_t cols, const char* what, int splits = 1) {
  const int64_t tm = ((int64_t)p.M + C::BM - 1) / C::BM, tn = (cols + C::OUT_N - 1) / C::OUT_N;
  if (tm * tn * splits >= (1 << 30)) return set_error(FG_EUNSUPPORTED, "%s: too many output tiles", what);
  p.tiles_m = (int)tm;
  p.tiles_n = (int)tn;
  p.num_tiles = (int)(tm * tn) * splits;
  p.group_m = 8;
  return FG_OK;
}

template <class C>
fg_status launch_tile(LinearParams& p, int cus, int64_t cols, void* stream, const char* what, int splits = 1) {
  FG_TRY(set_tiles<C>(p, cols, what, splits));
  const int grid = std::min(cus * C::OCC, p.num_tiles);
  hipLaunchKernelGGL((linear_tile_kernel<C>), dim3((unsigned)grid), dim3(C::THREADS), 0, (hipStream_t)stream, p);
  return launched(what);
}

// Output tiles of BM rows and BN weight rows.
double tile_count(const LinearParams& p, int64_t cols, bool gated, int bm, int bn) {
  const int out_n = gated ? bn / 2 : bn;
  return (double)(((int64_t)p.M + bm - 1) / bm) * (double)((cols + out_n - 1) / out_n);
}

// One tile per CU and round: `idle` a slice with few CUs at work, `busy` with
// all of them (clock and cache contention, which sets in towards the end),
// `store` for the epilogue.
double tile_us(double tiles, int cus, int nk, double idle, double busy, double store) {
  const double load = tiles < cus ? tiles / cus : 1.0;
  return 3.4 + ceil(tiles / cus) * (nk * (idle + (busy - idle) * load * load) + store);
}

// Two workgroups to a CU: `idle` to `one` a slice while every CU has at most
// one, `two` for both.
double pairs_us(double tiles, int cus, int nk, double idle, double one, double two, double store) {
  const double full = floor(tiles / (2 * cus)), rest = tiles - full * 2 * cus, load = rest / cus;
  double us = 3.4 + full * (nk * two + store);
  if (rest > 0) us += nk * (rest > cus ? two : idle + (one - idle) * load * load) + store;
  return us;
}

// The tiles below 256 rows, with their times a slice where both operands are
// K-major and where one or both are MN-major (mn).
//
// 64 x 64, eight waves, for few tiles: in two groups (256 x 4096 x 7168 int8 17
// us, 28 on 128 x 128); where operands are MN-major in one, so that every sum
// of a gradient runs in the order of its slices and its bits depend on nothing
// but the split.  There it serves splits and shared launches alone: two
// workgroups of four waves are as fast with few tiles (dX 333 x 1528 x 2176 13
// us both) and faster with many.
double small_us(double tiles, int cus, int nk, bool mn) {
  return mn ? tile_us(tiles, cus, nk, 0.28, 0.35, 1.2) : tile_us(tiles, cus, nk, 0.177, 0.19, 1.5);
}

// 64 x 64, two workgroups of four waves, where tiles outnumber the CUs (dW
// 2176 x 1528 x 333 12 us, 13 on eight waves).
double small2_us(double tiles, int cus, int nk, bool mn) {
  return mn ? pairs_us(tiles, cus, nk, 0.22, 0.32, 0.68, 1.3) : pairs_us(tiles, cus, nk, 0.187, 0.19, 0.54, 1.25);
}

// 128 x 64, two workgroups of eight waves (512 x 4096 x 7168 int8 28 us, 31 on
// 128 x 128 and on 64 x 64; gated bf16 333 x 1056 x 1528 11 us, 17 on 128 x 128).
double half2_us(double tiles, int cus, int nk, bool mn) {
  return mn ? pairs_us(tiles, cus, nk, 0.30, 0.39, 0.75, 1.7) : pairs_us(tiles, cus, nk, 0.23, 0.30, 0.66, 1.9);
}

// 128 x 128, eight waves, four stages (1000 x 4096 x 7168 int8 33 us, 72 on
// 256 x 256).
double mid_us(double tiles, int cus, int nk, bool mn) {
  return mn ? tile_us(tiles, cus, nk, 0.46, 0.53, 2.0) : tile_us(tiles, cus, nk, 0.44, 0.51, 2.4);
}

// 128 x 128, two workgroups of four waves (dW 3072 x 2048 x 1500 28 us, 33 on
// eight waves).
double mid2_us(double tiles, int cus, int nk, bool mn) {
  return mn ? pairs_us(tiles, cus, nk, 0.80, 0.80, 0.90, 1.5) : pairs_us(tiles, cus, nk, 0.70, 0.70, 0.90, 1.5);
}

template <class C>
fg_status launch_fewrow(const LinearParams& p, void* stream, const char* what) {
  const int64_t parts = ((int64_t)p.M + C::ROWS - 1) / C::ROWS, tiles = ((int64_t)p.N + C::OUT_N - 1) / C::OUT_N;
  if (parts * tiles >= (1 << 23)) return set_error(FG_EUNSUPPORTED, "%s: too many output tiles", what);
  hipLaunchKernelGGL((fewrow_kernel<C>), dim3((unsigned)(parts * tiles)), dim3(C::THREADS), 0, (hipStream_t)stream, p,
                     (int)parts);
  return launched(what);
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
constexpr int kFewRowMost = 640;  // rows up to which these shapes are considered

double fewrow_us(const LinearParams& p, bool gated, int cus, const FewRowShape& f) {
  const double groups = (double)((p.M + 16 * f.mf - 1) / (16 * f.mf)) * ceil((double)p.N / (gated ? 8 * f.cf : 16 * f.cf));
  const double load = groups < cus ? groups / cus : 1.0, turns = ceil(groups / cus);
  const double one = 0.9 + (p.nk + f.waves - 1) / f.waves * (f.idle + (f.busy - f.idle) * load);
  return f.base + (turns > 1 ? turns * f.shared : 1.0) * one;
}

// Splits of the reduction over workgroups, in the backward pass: of dX's sum
// over 2F, and of the recomputed pre-activations' over K.  The fp32 partials
// of at most kMaxSplits splits and kMaxPartialBytes go to the workspace and
// the next launch adds them.
constexpr int kMaxSplits = 16;
constexpr int64_t kMaxPartialBytes = (int64_t)32 << 20;

// Workspace bytes for the partials of an M x N output: none where fewer than
// two fit.
int64_t partial_bytes(int64_t M, int64_t N) {
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
SplitPlan plan_split(const LinearParams& p, int64_t cols, bool gated, bool mn, int64_t one, int cus, int bm, F cost) {
  const double tiles = tile_count(p, cols, gated, bm, bm);
  SplitPlan s{1e30, 1, p.nk};
  if (one > kMaxPartialBytes / 2 || tiles > cus / 2) return s;
  const int most = (int)std::min<int64_t>(std::min<int64_t>(kMaxSplits, kMaxPartialBytes / one), (int64_t)(cus / tiles));
  s.nk = (int)round_up((p.nk + most - 1) / most, 2);
  s.splits = (p.nk + s.nk - 1) / s.nk;
  // the partials are written and read at about 4 TB/s; the second launch is 2.3 us
  s.us = cost(tiles * s.splits, cus, s.nk, mn) + 2.3 + 2.0 * s.splits * one / 4e6;
  return s;
}

// Bytes of the pre-activations' partials: none where 64 x 64 tiles (32 hidden
// units) already take more than a third of 256 CUs.
constexpr int kMaxPairTiles = 85;
int64_t pair_partial_bytes(int64_t M, int64_t cols) {
  return (M + 63) / 64 * (cols / 64) > kMaxPairTiles ? 0 : partial_bytes(M, cols);
}

template <int E>
int slice_count(const LinearParams& p) {
  return (int)std::max<int64_t>(1, ((int64_t)p.K * (epi_int8(E) ? 1 : 2) + 127) / 128);
}

// The cheapest tile for p (its slices set) and its time.
enum TileKind { kW256, kW224, kW192, kW160, kMid2, kMid, kHalf2, kSmall2, kSmall };
struct TilePlan {
  TileKind kind;
  double us;
};

// The environment variable FG_LINEAR_PLAN overrides the choice (tuning and
// tests): a tile ("w256", "w224", "w192", "w160", "mid2", "mid", "half2",
// "small2", "small"), a few-row shape ("few0" .. "few7"), or for the gradients
// "split-mid", "split-small" (dX's sum), "pair" (the recomputed
// pre-activations' sums) or "share-X-W" (X and W: mid or small).  A plan that
// the call does not have leaves it its own.
const char* forced_plan() {
  const char* f = getenv("FG_LINEAR_PLAN");
  return f ? f : "";
}

bool forced_tile(bool gated, TileKind* kind) {
  static const struct {
    const char* name;
    TileKind kind;
  } names[] = {{"w256", kW256}, {"w224", kW224}, {"w192", kW192}, {"w160", kW160},
               {"mid2", kMid2}, {"mid", kMid},   {"half2", kHalf2}, {"small2", kSmall2}, {"small", kSmall}};
  const char* f = forced_plan();
  if (!*f) return false;
  for (const auto& n : names)
    if (strcmp(f, n.name) == 0 && (gated ? n.kind != kW224 && n.kind != kW160 : n.kind != kW192)) {
      *kind = n.kind;
      return true;
    }
  return false;
}

bool shares(const char* forced, TileKind x, TileKind w) {
  char name[32];
  snprintf(name, sizeof name, "share-%s-%s", x == kMid ? "mid" : "small", w == kMid ? "mid" : "small");
  return strcmp(forced, name) == 0;
}

TilePlan plan_tile(const LinearParams& p, int64_t cols, bool gated, bool mn, int cus) {
  TileKind forced;
  if (forced_tile(gated, &forced)) return TilePlan{forced, 0.0};
  auto count = [&](int bm, int bn) { return tile_count(p, cols, gated, bm, bn); };
  TilePlan best{kW256, 1e30};
  auto offer = [&](TileKind kind, double us) {
    if (us < best.us) best = TilePlan{kind, us};
  };
  // 256 rows by 256, 224, 192 or 160: the time of a slice grows with the CUs at
  // work, since the chip's power limits these (int8 4096 x 7168 x 16384: 372 us
  // with 256 columns, 343 with 224; 4096 x 2112 x 7168: 78 with 256, 60 with
  // 160; gated bf16 4096 x 12288 x 1536: 238 with 256, 266 with 192).
  offer(kW256, tile_us(count(256, 256), cus, p.nk, 1.2, mn ? 1.3 : 1.45, 4.0));
  if (gated) {
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

template <int E, bool TA, bool TB>
using MidTile = LinearTile<E, 128, 128, 4, 2, 1, 4, TA, TB>;
template <int E, bool TA, bool TB>
using SmallTile = LinearTile<E, 64, 64, TA || TB ? 4 : 2, 2, TA || TB ? 1 : 2, 4, TA, TB>;

template <int E, bool TA = false, bool TB = false>
fg_status launch_planned(LinearParams& p, TileKind kind, int64_t cols, int cus, void* stream, const char* what) {
  switch (kind) {
    case kW224:
      if constexpr (!epi_gated(E)) return launch_tile<LinearTile<E, 256, 224, 4, 2, 1, 2, TA, TB>>(p, cus, cols, stream, what);
      break;
    case kW192:
      if constexpr (epi_gated(E)) return launch_tile<LinearTile<E, 256, 192, 4, 2, 1, 2, TA, TB>>(p, cus, cols, stream, what);
      break;
    case kW160:
      if constexpr (!epi_gated(E)) return launch_tile<LinearTile<E, 256, 160, 4, 2, 1, 2, TA, TB>>(p, cus, cols, stream, what);
      break;
    case kMid2: return launch_tile<LinearTile<E, 128, 128, 2, 2, 1, 2, TA, TB>>(p, cus, cols, stream, what);
    case kHalf2: return launch_tile<LinearTile<E, 128, 64, 4, 2, 1, 3, TA, TB>>(p, cus, cols, stream, what);
    case kSmall2: return launch_tile<LinearTile<E, 64, 64, 2, 2, 1, 4, TA, TB>>(p, cus, cols, stream, what);
    case kMid: return launch_tile<MidTile<E, TA, TB>>(p, cus, cols, stream, what);
    case kSmall:
      if constexpr (!TA && !TB) return launch_tile<SmallTile<E, TA, TB>>(p, cus, cols, stream, what);
      break;
    default: break;
  }
  return launch_tile<LinearTile<E, 256, 256, 4, 2, 1, 2, TA, TB>>(p, cus, cols, stream, what);
}

// One product: the operands of the forward passes and of the recomputed
// gradient pair, both K-major.
template <int E>
fg_status launch_linear(LinearParams& p, void* stream, const char* what) {
  int cus = 0;
  FG_TRY(usable_cus(&cus));
  constexpr bool gated = epi_gated(E);
  const int64_t cols = E == kEpiGatedGrad ? p.half : p.N;
  p.nk = slice_count<E>(p);
  const TilePlan tile = plan_tile(p, cols, gated, false, cus);
  if constexpr (E != kEpiGatedGrad) {
    if (p.M <= kFewRowMost) {
      int best = -1;
      double least = tile.us;
      for (int i = 0; i < (int)(sizeof kFewRowShapes / sizeof *kFewRowShapes); ++i) {
        const double t = fewrow_us(p, gated, cus, kFewRowShapes[i]);
        if (t < least) {
          least = t;
          best = i;
        }
      }
      const char* f = forced_plan();
      if (strncmp(f, "few", 3) == 0 && f[3] >= '0' && f[3] <= '7' && !f[4]) best = f[3] - '0';
      switch (best) {
        case 0: return launch_fewrow<FewRow<E, 1, 1, 4, 2>>(p, stream, what);
        case 1: return launch_fewrow<FewRow<E, 1, 1, 8, 2>>(p, stream, what);
        case 2: return launch_fewrow<FewRow<E, 1, 2, 4, 2>>(p, stream, what);
        case 3: return launch_fewrow<FewRow<E, 2, 1, 4, 3>>(p, stream, what);
        case 4: return launch_fewrow<FewRow<E, 2, 2, 4, 2>>(p, stream, what);
        case 5: return launch_fewrow<FewRow<E, 4, 1, 4, 2>>(p, stream, what);
        case 6: return launch_fewrow<FewRow<E, 4, 2, 4, 2>>(p, stream, what);
        case 7: return launch_fewrow<FewRow<E, 4, 4, 4, 2>>(p, stream, what);
        default: break;
      }
    }
  }
  return launch_planned<E>(p, tile.kind, cols, cus, stream, what);
}

// ---------------------------------------------------------------------------
// dX = pair . W and dW = pair^T . X, either or both.  Each has its own plan;
// where neither fills the device, both go into one launch, with 128 x 128 or
// 64 x 64 tiles each.

struct GradPlan {
  TileKind kind;
  int splits;  // of dX's sum
  double us;   // in a launch of its own
};

// Adds dX's partials.
fg_status launch_add(const LinearParams& p, int splits, void* stream, const char* what) {
  const int64_t blocks = ((int64_t)p.M * (p.N / 4) + 255) / 256;
  hipLaunchKernelGGL(add_partials_kernel, dim3((unsigned)std::min<int64_t>(blocks, 1 << 16)), dim3(256), 0,
                     (hipStream_t)stream, p, splits);
  return launched(what);
}

template <class X, class W>
fg_status launch_both(LinearParams& x, int splits, LinearParams& w, void* stream, const char* what) {
  FG_TRY((set_tiles<X>(x, x.N, what, splits)));
  FG_TRY((set_tiles<W>(w, w.N, what)));
  hipLaunchKernelGGL((linear_grads_kernel<X, W>), dim3((unsigned)(x.num_tiles + w.num_tiles)), dim3(X::THREADS), 0,
                     (hipStream_t)stream, x, w, x.num_tiles);
  return launched(what);
}

template <int EX>
fg_status launch_both(LinearParams& x, TileKind kx, int splits, LinearParams& w, TileKind kw, void* stream,
                      const char* what) {
  using MX = MidTile<EX, false, true>;
  using SX = SmallTile<EX, false, true>;
  using MW = MidTile<kEpiBf16, true, true>;
  using SW = SmallTile<kEpiBf16, true, true>;
  if (kx == kMid)
    return kw == kMid ? launch_both<MX, MW>(x, splits, w, stream, what) : launch_both<MX, SW>(x, splits, w, stream, what);
  return kw == kMid ? launch_both<SX, MW>(x, splits, w, stream, what) : launch_both<SX, SW>(x, splits, w, stream, what);
}

fg_status launch_grads(LinearParams* x, LinearParams* w, void* stream, const char* what) {
  int cus = 0;
  FG_TRY(usable_cus(&cus));
  GradPlan px{kW256, 1, 0}, pw{kW256, 1, 0};
  double x_us = 0, w_us = 0;
  if (x) {
    x->nk = slice_count<kEpiBf16>(*x);
    x->split_nk = x->nk;
    const TilePlan t = plan_tile(*x, x->N, false, true, cus);
    px.kind = t.kind;
    px.us = t.us;
    // 251 x 1016 with 178 slices: 52 us on 64 64 x 64 tiles, a quarter of the
    // device; split 27 us with the addition.
    const int64_t one = (int64_t)x->M * x->N * 4;
    const SplitPlan a = plan_split(*x, x->N, false, true, one, cus, 64, small_us);
    const SplitPlan b = plan_split(*x, x->N, false, true, one, cus, 128, mid_us);
    const char* f = forced_plan();
    const bool force_small = strcmp(f, "split-small") == 0, force_mid = strcmp(f, "split-mid") == 0;
    const bool small_tiles = force_small || (!force_mid && a.us <= b.us);
    const SplitPlan& s = small_tiles ? a : b;
    if (x->P && s.splits > 1 && (s.us < px.us || force_small || force_mid)) {
      px = GradPlan{small_tiles ? kSmall : kMid, s.splits, s.us};
      x->split_nk = s.nk;
    }
    x_us = px.us;
  }
  if (w) {
    w->nk = slice_count<kEpiBf16>(*w);
    const TilePlan t = plan_tile(*w, w->N, false, true, cus);
    pw.kind = t.kind;
    pw.us = t.us;
    w_us = pw.us;
  }
  if (x && w) {
    // One launch: the workgroups of both, one to a CU, dX's first.  The device
    // is busy for their total, and for the longest one at least.
    double least = x_us + w_us;
    TileKind kx = kW256, kw = kW256;
    const char* forced = forced_plan();
    for (const TileKind cx : {kMid, kSmall})
      for (const TileKind cw : {kMid, kSmall}) {
        if (px.splits > 1 && cx != px.kind) continue;
        const int bx = cx == kMid ? 128 : 64, bw = cw == kMid ? 128 : 64;
        const double nx = tile_count(*x, x->N, false, bx, bx) * px.splits, nw = tile_count(*w, w->N, false, bw, bw);
        const double tx = x->split_nk * (cx == kMid ? 0.57 : 0.45) + (cx == kMid ? 2.5 : 1.5);
        const double tw = w->nk * (cw == kMid ? 0.63 : 0.37) + (cw == kMid ? 2.5 : 1.5);  // both operands MN-major
        const double us = 3.4 + std::max(std::max(tx, tw), (nx * tx + nw * tw) / cus + 0.5 * std::min(tx, tw)) +
                          (px.splits > 1 ? 4.0 : 0.0);
        if (nx + nw >= (1 << 22)) continue;
        if (*forced ? shares(forced, cx, cw) : us < least) {
          least = us;
          kx = cx;
          kw = cw;
        }
      }
    if (kx != kW256) {
      if (px.splits == 1) return launch_both<kEpiBf16>(*x, kx, 1, *w, kw, stream, what);
      FG_TRY(launch_both<kEpiPartial>(*x, kx, px.splits, *w, kw, stream, what));
      return launch_add(*x, px.splits, stream, what);
    }
  }
  if (x) {
    if (px.splits > 1) {
      if (px.kind == kSmall)
        FG_TRY((launch_tile<SmallTile<kEpiPartial, false, true>>(*x, cus, x->N, stream, what, px.splits)));
      else
        FG_TRY((launch_tile<MidTile<kEpiPartial, false, true>>(*x, cus, x->N, stream, what, px.splits)));
      FG_TRY(launch_add(*x, px.splits, stream, what));
    } else {
      FG_TRY((launch_planned<kEpiBf16, false, true>(*x, px.kind, x->N, cus, stream, what)));
    }
  }
  if (w) FG_TRY((launch_planned<kEpiBf16, true, true>(*w, pw.kind, w->N, cus, stream, what)));
  return FG_OK;
}

// Sizes every entry point shares; *empty when there is no output element.
fg_status check_sizes(int M, int N, int K, int mult, bool* empty) {
  *empty = false;
  if (M < 0 || N < 0 || K < 0) return set_error(FG_EINVAL, "negative size: %d rows, %d columns, K=%d", M, N, K);
  if (K % mult) return set_error(FG_EALIGN, "K=%d is not a multiple of %d", K, mult);
  if (M == 0 || N == 0) {
    *empty = true;
    return FG_OK;
  }
  if (M > kMaxRows || N > kMaxRows / 2) return set_error(FG_EUNSUPPORTED, "more than 2^30 rows");
  return FG_OK;
}

fg_status check_operand(const void* ptr, int64_t ld, int64_t cols, int item, const char* name, const char* ld_name) {
  FG_TRY(require_ptr(ptr, 16, name));
  FG_TRY(require_ld(ld, cols, 16 / item, ld_name));
  if (ld * item > kMaxRowBytes) return set_error(FG_EUNSUPPORTED, "%s=%lld: rows above 4 MiB", ld_name, (long long)ld);
  return FG_OK;
}

// Operands and the bytes between their rows.  Not called where K is 0: the
// kernels then read nothing, and pointers and strides, which nobody checked,
// must not go into their ranges.
void set_operands(LinearParams& p, const void* A, int64_t lda, const void* B, int64_t ldb) {
  p.A = (const uint8_t*)A;
  p.lda = lda;
  p.B = (const uint8_t*)B;
  p.ldb = ldb;
}

fg_status check_workspace(const void* ws, int64_t bytes, int64_t need) {
  if (bytes < 0) return set_error(FG_EINVAL, "workspace_bytes=%lld is negative", (long long)bytes);
  if (!ws && bytes > 0) return set_error(FG_EINVAL, "workspace is NULL");
  if (ws && ((uintptr_t)ws & 255)) return set_error(FG_EALIGN, "workspace is not 256-byte aligned");
  if (bytes < need)
    return set_error(FG_EINVAL, "workspace_bytes=%lld is smaller than the %lld needed", (long long)bytes,
                     (long long)need);
  return FG_OK;
}

fg_status check_activation(int act) {
  if (act != FG_ACT_SILU && act != FG_ACT_GELU_TANH) return set_error(FG_EINVAL, "activation=%d is not known", act);
  return FG_OK;
}

int64_t pair_cols(int F) { return 2 * round_up(F, kPairAlign); }

// The gradient pair, then partials.
int64_t pair_bytes(int M, int F) { return round_up((int64_t)M * pair_cols(F) * 2, 256); }
int64_t backward_bytes(int M, int F, int K) {
  return pair_bytes(M, F) + std::max(partial_bytes(M, K), pair_partial_bytes(M, pair_cols(F)));
}

// [dg du] from pre-activations in g.P: kept ones, or `parts` partial sums.
template <bool PARTS>
fg_status launch_gated_grad(const LinearParams& g, int parts, void* stream, const char* what) {
  const int64_t blocks = ((int64_t)g.M * (g.half / (PARTS ? 4 : 8)) + 255) / 256;
  const dim3 grid((unsigned)std::min<int64_t>(blocks, 1 << 16));
  if (g.act == kActSilu)
    hipLaunchKernelGGL((gated_grad_kernel<kActSilu, PARTS>), grid, dim3(256), 0, (hipStream_t)stream, g, parts);
  else
    hipLaunchKernelGGL((gated_grad_kernel<kActGeluTanh, PARTS>), grid, dim3(256), 0, (hipStream_t)stream, g, parts);
  return launched(what);
}

// [dg du] with the pre-activations recomputed: in the product's own epilogue,
// or, where its tiles leave most of the device idle, from partial sums in
// `partials` (with dW, 395 x 36 x 6232: 40 us without, 22 with; 595 x 175 x
// 3320: 31 and 24).
fg_status launch_recompute(LinearParams& g, float* partials, void* stream, const char* what) {
  int cus = 0;
  FG_TRY(usable_cus(&cus));
  if (pair_partial_bytes(g.M, 2 * g.half) > 0) {
    g.nk = slice_count<kEpiGatedPartial>(g);
    const int64_t one = (int64_t)g.M * g.half * 8;
    const SplitPlan s = plan_split(g, g.half, true, false, one, cus, 64, small_us);
    const char* f = forced_plan();
    if (s.splits > 1 && (*f ? strcmp(f, "pair") == 0 : s.us < plan_tile(g, g.half, true, false, cus).us)) {
      g.P = partials;
      g.ldp = 2 * g.half;
      g.split_nk = s.nk;
      FG_TRY((launch_tile<SmallTile<kEpiGatedPartial, false, false>>(g, cus, g.half, stream, what, s.splits)));
      return launch_gated_grad<true>(g, s.splits, stream, what);
    }
  }
  return launch_linear<kEpiGatedGrad>(g, stream, what);
}

template <typename T>
fg_status cast_rows(const T* x, int64_t ldx, int8_t* q, float* s, int M, int K, void* stream, const char* what) {
  clear_error();
  if (M < 0 || K < 0) return set_error(FG_EINVAL, "negative size M=%d K=%d", M, K);
  if (K % 16) return set_error(FG_EALIGN, "K=%d is not a multiple of 16", K);
  if (M == 0) return FG_OK;
  FG_TRY(require_ptr(s, 4, "s"));
  if (K > 0) {
    FG_TRY(require_ptr(x, 16, "x"));
    FG_TRY(require_ptr(q, 16, "q"));
    FG_TRY(require_ld(ldx, K, 16 / (int)sizeof(T), "ldx"));
  }
  const int pieces = K / (16 / (int)sizeof(T));
  const dim3 grid((unsigned)std::min(M, 1 << 20));
  // Two pieces a thread while they hold the row (4096 x 7168 bf16: 512 threads
  // 15.0 us, 5.9 TB/s; 4096 x 1024: 256 threads 5.7 us), four of a longer one.
  if (pieces <= 512)
    hipLaunchKernelGGL((int8_cast_kernel<T, 256, 2>), grid, dim3(256), 0, (hipStream_t)stream, x, ldx, q, s, M, K);
  else if (pieces <= 1024)
    hipLaunchKernelGGL((int8_cast_kernel<T, 512, 2>), grid, dim3(512), 0, (hipStream_t)stream, x, ldx, q, s, M, K);
  else
    hipLaunchKernelGGL((int8_cast_kernel<T, 512, 4>), grid, dim3(512), 0, (hipStream_t)stream, x, ldx, q, s, M, K);
  return launched(what);
}

}  // namespace
}  // namespace fg

using namespace fg;

extern "C" {

fg_status int8_cast_per_row(const float* x, int64_t ldx, int8_t* q, float* s, int M, int K, void* stream) {
  return cast_rows(x, ldx, q, s, M, K, stream, "int8_cast_per_row");
}

fg_status int8_cast_per_row_bf16(const uint16_t* x, int64_t ldx, int8_t* q, float* s, int M, int K, void* stream) {
  return cast_rows(x, ldx, q, s, M, K, stream, "int8_cast_per_row_bf16");
}

fg_status gemm_int8_nt(const int8_t* A, int64_t lda, const float* sa, const int8_t* B, int64_t ldb, const float* sb,
                       uint16_t* D, int64_t ldd, int M, int N, int K, void* stream) {
  clear_error();
  bool empty;
  FG_TRY(check_sizes(M, N, K, 16, &empty));
  if (empty) return FG_OK;
  if (K > kMaxInt8K) return set_error(FG_EUNSUPPORTED, "K=%d: sums of more than %d products", K, kMaxInt8K);
  FG_TRY(require_ptr(D, 2, "D"));
  FG_TRY(require_ld(ldd, N, 1, "ldd"));
  FG_TRY(require_ptr(sa, 4, "sa"));
  FG_TRY(require_ptr(sb, 4, "sb"));
  if (K > 0) {
    FG_TRY(check_operand(A, lda, K, 1, "A", "lda"));
    FG_TRY(check_operand(B, ldb, K, 1, "B", "ldb"));
  }
  LinearParams p{};
  if (K > 0) set_operands(p, A, lda, B, ldb);
  p.sa = sa; p.sb = sb;
  p.D = D; p.ldd = ldd; p.M = M; p.N = N; p.K = K;
  return launch_linear<kEpiInt8>(p, stream, "gemm_int8_nt");
}

fg_status gated_ffn_int8(const int8_t* X, int64_t ldx, const float* sx, const int8_t* W, int64_t ldw,
                         const float* sw, uint16_t* H, int64_t ldh, int M, int F, int K, int activation,
                         void* stream) {
  clear_error();
  bool empty;
  FG_TRY(check_sizes(M, F, K, 16, &empty));
  FG_TRY(check_activation(activation));
  if (empty) return FG_OK;
  if (K > kMaxInt8K) return set_error(FG_EUNSUPPORTED, "K=%d: sums of more than %d products", K, kMaxInt8K);
  FG_TRY(require_ptr(H, 2, "H"));
  FG_TRY(require_ld(ldh, F, 1, "ldh"));
  FG_TRY(require_ptr(sx, 4, "sx"));
  FG_TRY(require_ptr(sw, 4, "sw"));
  if (K > 0) {
    FG_TRY(check_operand(X, ldx, K, 1, "X", "ldx"));
    FG_TRY(check_operand(W, ldw, K, 1, "W", "ldw"));
  }
  LinearParams p{};
  if (K > 0) set_operands(p, X, ldx, W, ldw);
  p.sa = sx; p.sb = sw;
  p.D = H; p.ldd = ldh; p.M = M; p.N = F; p.K = K; p.act = activation;
  return launch_linear<kEpiGatedInt8>(p, stream, "gated_ffn_int8");
}

fg_status gated_ffn_bf16(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, uint16_t* H, int64_t ldh,
                         float* P, int64_t ldp, int M, int F, int K, int activation, void* stream) {
  clear_error();
  bool empty;
  FG_TRY(check_sizes(M, F, K, 8, &empty));
  FG_TRY(check_activation(activation));
  if (empty) return FG_OK;
  FG_TRY(require_ptr(H, 2, "H"));
  FG_TRY(require_ld(ldh, F, 1, "ldh"));
  if (P) {
    FG_TRY(require_ptr(P, 4, "P"));
    FG_TRY(require_ld(ldp, 2 * (int64_t)F, 1, "ldp"));
  }
  if (K > 0) {
    FG_TRY(check_operand(X, ldx, K, 2, "X", "ldx"));
    FG_TRY(check_operand(W, ldw, K, 2, "W", "ldw"));
  }
  LinearParams p{};
  if (K > 0) set_operands(p, X, 2 * ldx, W, 2 * ldw);
  p.D = H; p.ldd = ldh; p.P = P; p.ldp = ldp; p.M = M; p.N = F; p.K = K; p.act = activation;
  return P ? launch_linear<kEpiGatedKeep>(p, stream, "gated_ffn_bf16")
           : launch_linear<kEpiGated>(p, stream, "gated_ffn_bf16");
}

fg_status gated_ffn_bf16_backward(const uint16_t* dH, int64_t lddh, const uint16_t* X, int64_t ldx,
                                  const uint16_t* W, int64_t ldw, const float* P, int64_t ldp, uint16_t* dX,
                                  int64_t lddx, uint16_t* dW, int64_t lddw, int M, int F, int K, int activation,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
  const char* what = "gated_ffn_bf16_backward";
  clear_error();
  if (M < 0 || F < 0 || K < 0) return set_error(FG_EINVAL, "negative size M=%d F=%d K=%d", M, F, K);
  if (K % 8) return set_error(FG_EALIGN, "K=%d is not a multiple of 8", K);
  FG_TRY(check_activation(activation));
  // no gradient element is asked for: dX is M x K, dW 2F x K
  if (K == 0 || ((!dX || M == 0) && (!dW || F == 0))) return FG_OK;
  if (M > kMaxRows || F > kMaxRows / 4) return set_error(FG_EUNSUPPORTED, "more than 2^30 rows");
  FG_TRY(check_workspace(workspace, workspace_bytes, M > 0 && F > 0 ? backward_bytes(M, F, K) : 0));
  if (dX && M > 0) {
    FG_TRY(require_ptr(dX, 2, "dX"));
    FG_TRY(require_ld(lddx, K, 1, "lddx"));
  }
  if (dW && F > 0) {
    FG_TRY(require_ptr(dW, 2, "dW"));
    FG_TRY(require_ld(lddw, K, 1, "lddw"));
  }
  LinearParams p{};
  p.act = activation;
  p.F = F;
  p.half = (int)(pair_cols(F) / 2);
  const int64_t pair_ld = pair_cols(F);
  if (M > 0 && F > 0) {
    FG_TRY(require_ptr(dH, 2, "dH"));
    FG_TRY(require_ld(lddh, F, 1, "lddh"));
    FG_TRY(check_operand(X, ldx, K, 2, "X", "ldx"));
    FG_TRY(check_operand(W, ldw, K, 2, "W", "ldw"));
    if (pair_ld * 2 > kMaxRowBytes) return set_error(FG_EUNSUPPORTED, "F=%d: rows above 4 MiB", F);
    if (P) {
      FG_TRY(require_ptr(P, 4, "P"));
      FG_TRY(require_ld(ldp, 2 * (int64_t)F, 1, "ldp"));
    }
    LinearParams g = p;
    g.A = (const uint8_t*)X; g.lda = 2 * ldx; g.B = (const uint8_t*)W; g.ldb = 2 * ldw;
    g.dH = dH; g.lddh = lddh; g.P = const_cast<float*>(P); g.ldp = ldp;
    g.D = (uint16_t*)workspace; g.ldd = pair_ld;
    g.M = M; g.N = F; g.K = K;
    FG_TRY(P ? launch_gated_grad<false>(g, 0, stream, what)
             : launch_recompute(g, (float*)((uint8_t*)workspace + pair_bytes(M, F)), stream, what));
  }
  // With M or F of zero the reductions below are empty and write zeros.
  LinearParams x = p, w = p;
  const bool want_x = dX && M > 0, want_w = dW && F > 0;
  if (want_x) {
    x.A = (const uint8_t*)workspace; x.lda = 2 * pair_ld; x.B = (const uint8_t*)W; x.ldb = 2 * ldw;
    x.D = dX; x.ldd = lddx; x.M = M; x.N = K; x.K = F > 0 ? (int)pair_ld : 0;
    if (F > 0 && partial_bytes(M, K) > 0) x.P = (float*)((uint8_t*)workspace + pair_bytes(M, F));
  }
  if (want_w) {
    w.A = (const uint8_t*)workspace; w.lda = 2 * pair_ld; w.B = (const uint8_t*)X; w.ldb = 2 * ldx;
    w.D = dW; w.ldd = lddw; w.M = (int)pair_ld; w.N = K; w.K = M;
  }
  return launch_grads(want_x ? &x : nullptr, want_w ? &w : nullptr, stream, what);
}

int64_t fg_gated_ffn_backward_workspace_bytes(int M, int F, int K) {
  if (M < 0 || F < 0 || K < 0 || M > kMaxRows || F > kMaxRows / 4 || K > kMaxRows) return -1;
  return M > 0 && F > 0 && K > 0 ? backward_bytes(M, F, K) : 0;
}

}  // extern "C"
