// decode_plan.hpp -- which kernels the 4-bit product and the few-token expert
// layers run: host arithmetic on sizes only.
//
// Two organisations (weight_stream.hpp): waves of a workgroup that share out a
// tile's reduction, each with its own columns of the activations ("split": many
// small tiles, for few rows), and waves with weight rows of their own that share
// the activations' columns ("wide": fewer bytes through LDS for each weight, for
// more rows).  The figures beside the rules are in microseconds, in a HIP graph.
//
// FG_DECODE_PLAN names parts of a plan, separated by commas, for tuning and
// tests; one that a call does not have or that does not fit LDS leaves it its own.
#pragma once

#include <stdint.h>
#include <string.h>

#include <algorithm>

namespace fg {

constexpr int kLayerTokens = 64;        // tokens a pass over the experts' weights serves
constexpr int64_t kPartialBytes = 512 << 10;  // of a token's partial sums

// Whether `name` is one of the comma-separated words of `forced`.
inline bool names(const char* forced, const char* name) {
  const size_t n = strlen(name);
  for (const char* p = forced; (p = strstr(p, name)) != nullptr; p += n)
    if ((p == forced || p[-1] == ',') && (p[n] == 0 || p[n] == ',')) return true;
  return false;
}

inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// ---------------------------------------------------------------------------
// gemm_int4_nt

enum Int4Kind { kSplit2, kSplit2Deep, kSplit8, kSplit8Deep, kSplit16, kSplit16Deep, kWide16, kWide32, kWide64, kInt4Kinds };
constexpr const char* kInt4Names[kInt4Kinds] = {"split2", "split2deep", "split8", "split8deep", "split16", "split16deep",
                                                "wide16", "wide32", "wide64"};
struct Int4Plan {
  Int4Kind kind;
  int k_parts;  // wide: parts of the reduction, joined by a second kernel
};

// What a plan takes, in microseconds, for more than eight rows: fitted to 16
// weights of 512 x 512 to 7168 x 16384 with 12 to 256 rows, where it is within
// 20% of most times.  A workgroup's start and end, a chunk of 256 columns, and
// rounds of 256 workgroups; parts are added by a second kernel, which reads what
// the first has written.
inline double split16_cost(int M, int N, int chunks) {
  const double rounds = ceil_div((int64_t)ceil_div(N, 16) * ceil_div(M, 16), 256);
  return 1.5 + rounds * (2.0 + 0.65 * ceil_div(chunks, 4));
}
inline double wide_cost(Int4Kind kind, int M, int N, int chunks, int parts) {
  const int rows = kind == kWide64 ? 64 : kind == kWide32 ? 32 : 16;
  const double start = kind == kWide64 ? 3.6 : kind == kWide32 ? 3.4 : 3.0, chunk = kind == kWide64 ? 1.9 : kind == kWide32 ? 1.23 : 1.03;
  const double rounds = ceil_div((int64_t)ceil_div(N, 128) * ceil_div(M, rows) * parts, 256);
  const double join = parts > 1 ? 2.5 + 0.1 * parts + 2e-6 * parts * M * N : 0.0;
  return rounds * (start + chunk * ceil_div(chunks, parts)) + join;
}
// Parts of the reduction: at most one round of workgroups, two chunks each at least.
inline int wide_parts(Int4Kind kind, int M, int N, int chunks) {
  const int rows = kind == kWide64 ? 64 : kind == kWide32 ? 32 : 16;
  const int64_t tiles = (int64_t)ceil_div(N, 128) * ceil_div(M, rows);
  const int most = (int)std::max<int64_t>(1, std::min<int64_t>({256 / tiles, chunks / 2, 16}));
  int best = 1;
  for (int n = 2; n <= most; ++n)
    if (wide_cost(kind, M, N, chunks, n) < wide_cost(kind, M, N, chunks, best)) best = n;
  return best;
}

inline Int4Plan plan_int4(int M, int N, int K, const char* forced) {
  const int chunks = ceil_div(K, 256);
  // The reduction of a 16-column tile over eight waves instead of four where the
  // tiles are few or the reduction is long (1 x 2112 x 7168: eight 5.5, four 6.3; 1 x
  // 7168 x 16384: 13.0 and 14.2), not elsewhere (1 x 24576 x 1536: 10.0 and 7.7).
  const bool deep = chunks >= 16 && N <= 4096;
  Int4Kind kind;
  if (M <= 2)
    kind = deep || chunks >= 32 ? kSplit2Deep : kSplit2;
  else if (M <= 8)
    // 4 x 24576 x 1536: split 10.8, wide 8.2; 4 x 16384 x 4096: 11.3 and 12.1
    kind = ceil_div(N, 16) > 1024 ? kWide16 : deep ? kSplit8Deep : kSplit8;
  else {
    kind = deep && N < 4096 ? kSplit16Deep : kSplit16;
    double least = split16_cost(M, N, chunks);
    for (Int4Kind wide : {kWide16, kWide32, kWide64}) {
      const double cost = wide_cost(wide, M, N, chunks, wide_parts(wide, M, N, chunks));
      if (cost < least) {
        least = cost;
        kind = wide;
      }
    }
  }
  for (int k = 0; k < kInt4Kinds; ++k)
    if (names(forced, kInt4Names[k])) kind = (Int4Kind)k;
  Int4Plan p{kind, 1};
  if (kind >= kWide16 && M > 2) {  // one or two rows have no workspace, whatever kernel is asked for
    p.k_parts = wide_parts(kind, M, N, chunks);
    for (int n = 1; n <= 8 && n <= std::max(1, chunks); ++n) {
      const char word[] = {'k', 'p', 'a', 'r', 't', 's', (char)('0' + n), 0};
      if (names(forced, word)) p.k_parts = n;
    }
  }
  return p;
}

inline int64_t int4_partial_bytes(int M, int N, const Int4Plan& p) {
  return p.k_parts > 1 ? (int64_t)p.k_parts * M * N * 4 : 0;
}

// ---------------------------------------------------------------------------
// expert layers

enum UpKind { kUpSplit2, kUpSplit4, kUpSplit16, kUpWide, kUpWideDeep, kUpWide8, kUpKinds };
constexpr const char* kUpNames[kUpKinds] = {"up-split2", "up-split4", "up-split16", "up-wide", "up-wide-deep", "up-wide8"};
enum DownKind { kDownSplit1, kDownSplit1Two, kDownSplit4, kDownSplit4Two, kDownWide16, kDownWide16Deep, kDownWide32, kDownKinds };
constexpr const char* kDownNames[kDownKinds] = {"down-split1", "down-split1-two", "down-split4", "down-split4-two", "down-wide16",
                                                "down-wide16-deep", "down-wide32"};
struct LayerPlan {
  UpKind up;
  DownKind down;
  int parts;  // wide down: parts of the experts' chunks, joined by a third kernel
};
inline constexpr bool wide_down(DownKind k) { return k >= kDownWide16; }

// The `down` kernels: tiles of 16 outputs of a wave, waves, ring slots, tokens of an
// expert in one go.  4 bits: the activations of 32 tokens instead of 24 would not
// leave LDS for the sums of 64.  kDownSplit1Two in e4m3 is for
// calls that name it.
struct DownShape {
  int tiles, waves, depth, rows;
};
constexpr DownShape down_shape(bool fp8, DownKind k) {
  return k == kDownSplit1       ? DownShape{1, 8, 2, 1}
         : k == kDownSplit1Two  ? DownShape{2, 8, fp8 ? 3 : 2, 1}
         : k == kDownSplit4     ? DownShape{1, 8, 2, 4}
         : k == kDownSplit4Two  ? DownShape{2, 4, 3, 4}
         : k == kDownWide16     ? DownShape{2, 4, 2, 16}
         : k == kDownWide16Deep ? DownShape{2, 4, 3, 16}
                                : DownShape{2, 4, fp8 ? 3 : 2, fp8 ? 32 : 24};
}
// KiB of `rows` bf16 rows of a chunk's activations.
constexpr int x_kib(bool fp8, int rows) { return rows * (fp8 ? 256 : 512) > 1024 ? rows * (fp8 ? 256 : 512) / 1024 : 1; }
// LDS bytes of a wave's scales: 4-bit groups of each row of its tiles, and one word between rows.
constexpr int scale_bytes(bool fp8, int tiles, int groups = 32) { return fp8 ? 0 : 16 * tiles * (groups + 1) * 4; }
// LDS bytes of `down`: weights of a split wave or of all wide ones, and three bf16 of each hidden unit of a chunk
// (where waves share them two times).
constexpr int down_ring(bool fp8, DownKind k) {
  const DownShape s = down_shape(fp8, k);
  return s.depth * (wide_down(k) ? s.waves : 1) * s.tiles * 2048;
}
constexpr int down_x(bool fp8, DownKind k) { return down_shape(fp8, k).rows * 3 * (fp8 ? 256 : 512) * (wide_down(k) ? 2 : 1); }
// What `down` knows of a pass's pairs (experts_kernel.hpp).
inline int pairs_bytes(int E, int T, int k) { return E * 12 + T * k * 6 + 4; }
inline int down_lds(bool fp8, DownKind kind, int T, int E, int k) {
  const DownShape s = down_shape(fp8, kind);
  const int own = down_ring(fp8, kind) + down_x(fp8, kind), scales = scale_bytes(fp8, s.tiles), sums = T * s.tiles * 64;
  return (wide_down(kind) ? own + s.waves * (scales + sums) : s.waves * (own + scales + sums)) + pairs_bytes(E, T, k);
}
constexpr int kLds = 160 * 1024;

// The rules are simple ones that lose least over 2700 layers of 1 to 68 tokens, 4
// to 128 experts, drawn alike, and weights of 256 to 2048 x 1024 to 7168: 1 to 2%
// of a layer's time on average against the best kernel of each, for either half and
// format; one layer in 20 loses more than 10%, none more than 40%.
inline LayerPlan plan_layer(bool fp8, int T, int k, int E, int F, int K, const char* forced) {
  T = std::min(T, kLayerTokens);
  const int pairs = T * k, active = std::min(E, pairs);  // experts with tokens, at most
  const int64_t wide8 = (int64_t)ceil_div(F, 128) * active;  // workgroups of 128 hidden units
  LayerPlan p{};
  // up, by an expert's tokens.  Few of them want many small workgroups (e4m3, T=7,
  // 64 experts of 1024 x 4096: split 37, wide 45; 4 bits, T=9, 16 of 2048 x 7168:
  // split 95, wide 109); more of them, with work for every CU, waves that share
  // their columns (4 bits, T=67, 8 of 1408 x 1024: wide 47, split 61; e4m3, T=38,
  // 64 of 256 x 2048: wide 34, split 35), which long rows give a deeper ring (32
  // of 2048 x 4096: 82 for 90).
  if (fp8) {
    if (2 * pairs < 5 * active || T <= 4)
      p.up = T > 4 && K < 2048 && wide8 >= 256 ? kUpWide : kUpSplit4;
    else
      p.up = wide8 < 88 ? kUpSplit16 : wide8 < 176 || K >= 4096 ? kUpWideDeep : kUpWide;
  } else if (2 * pairs < 9 * active) {
    // room for two tokens only leaves more workgroups on a CU (T=2, 16 experts of 2048 x 7168: 75 for 79)
    p.up = T <= 2 ? kUpSplit2 : wide8 < 448 ? kUpSplit4 : kUpWide8;
  } else {
    p.up = wide8 < 88 ? kUpSplit16 : wide8 < 384 ? kUpWide : kUpWide8;
  }
  for (int i = 0; i < kUpKinds; ++i)
    if (names(forced, kUpNames[i]) && (fp8 ? i != kUpWide8 && i != kUpSplit2 : i != kUpWideDeep)) p.up = (UpKind)i;
  // down.  A third kernel costs about 3 us, so that few pairs go without (e4m3,
  // T=8, 2 of 8 experts of 512 x 1024: split 13.3, wide 16.1; 4 bits, T=9, 2 of 64 of
  // 512 x 2048: 20.9 and 21.1), unless there are few outputs for much work (e4m3,
  // T=5, 4 of 64 of 2048 x 1024: split 48.6, wide 36.6).
  const bool few = pairs < (fp8 ? 26 : 22) && (K >= 2048 || (int64_t)active * F * K <= 1 << 24);
  const int tiles = ceil_div(K, 128);
  const bool one = 8 * pairs < 9 * active && (!fp8 || (int64_t)active * F * K < 43000000);  // a token for each expert
  if (T == 1 || (few && one))
    // two tiles: over 4096 outputs 4 bits are 1.5% faster so (190 layers), e4m3 1% slower (200); up to 4096, 6% and more slower
    p.down = !fp8 && K > 4096 && T <= 16 ? kDownSplit1Two : kDownSplit1;
  else if (few)
    // 4 bits, T=2, 4 experts of 2048 x 7168: 32.5 for 36.5; of 2048 x 4096: 27.3 for 21.7
    p.down = !fp8 && K > 4096 ? kDownSplit4Two : kDownSplit4;
  else if (pairs >= 14 * active)
    p.down = kDownWide32;  // e4m3, T=64, 8 of 16 experts of 2048 x 4096: 135 for 151; 4 bits no faster and no slower
  else
    // a third slot: 1.5% faster for more than 32 tokens of long reads (48 layers of 100 MB and more); 2 to 9% slower
    // where it costs a second workgroup on the CU
    p.down = fp8 && T > 32 && (int64_t)active * F * K >= 100000000 ? kDownWide16Deep : kDownWide16;
  // what many experts or pairs leave no LDS for
  if (down_lds(fp8, p.down, T, E, k) > kLds) p.down = kDownWide16;
  for (int i = 0; i < kDownKinds; ++i)
    if (names(forced, kDownNames[i]) && (fp8 ? i != kDownSplit4Two : i != kDownWide16Deep) &&
        down_lds(fp8, (DownKind)i, T, E, k) <= kLds)
      p.down = (DownKind)i;
  p.parts = 1;
  if (wide_down(p.down)) {
    // workgroups for one round: two on a CU where their LDS allows it
    const int round = fp8 && p.down == kDownWide16 && T <= 32 ? 512 : 256;
    const int64_t chunks = (int64_t)active * ceil_div(F, fp8 ? 128 : 256);
    p.parts = (int)std::max<int64_t>(1, std::min<int64_t>({round / tiles, chunks, kPartialBytes / 4 / K}));
    if (T == 1 || names(forced, "one-part")) p.parts = 1;
  }
  return p;
}

// Workspace: the hidden units of every pair, then partial sums.
inline int64_t hidden_bytes(int T, int k, int F) { return ((int64_t)T * k * F * 4 + 255) / 256 * 256; }
inline int64_t layer_bytes(int T, int k, int F) {
  return hidden_bytes(T, k, F) + (T > 1 ? std::min(T, kLayerTokens) * kPartialBytes : 0);
}

}  // namespace fg
