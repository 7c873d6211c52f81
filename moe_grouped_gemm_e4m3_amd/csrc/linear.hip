// linear.hip -- C entry points of the 8-bit-integer products and the gated
// feed-forward block (linear_kernel.hpp): argument checks and the launches that
// linear_plan.hpp chooses.  Nothing is launched after a failed check; nothing
// is allocated.

#include <algorithm>
#include <cstdio>
#include <cstdlib>

#include "host_common.hpp"
#include "linear_fewrow.hpp"
#include "linear_plan.hpp"

#define FG_TRY(x)                   \
  do {                              \
    fg_status st__ = (x);           \
    if (st__ != FG_OK) return st__; \
  } while (0)

namespace fg {
namespace {

// rows of an output, and of the weights of a gated output
constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxRowBytes = (int64_t)1 << 22;  // buffer offsets inside a tile are 32-bit
// |sum| <= 128 * 128 * K must stay below 2^31
constexpr int kMaxInt8K = (1 << 17) - 16;

fg_status launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return set_error(FG_EHIP, "%s launch: %s", what, hipGetErrorString(e));
  return FG_OK;
}

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

// FG_PRINT_CONFIGS: a launch's product on C's tiles.
template <class C>
void print_tiles(const LinearParams& p, const char* what, const char* launch, int splits, int grid) {
  if (print_launches())
    fprintf(stderr, "[fp8gemm] %s %s M=%d N=%d K=%d tile=%dx%d threads=%d tiles=%d splits=%d grid=%d\n", what, launch, p.M,
            p.N, p.K, C::BM, C::BN, C::THREADS, p.num_tiles, splits, grid);
}

// The launch of a product on C's tiles, as print_tiles() names it.
template <class C>
const char* launch_name() {
  if (C::E == kEpiGatedGrad || C::E == kEpiGatedPartial) return "pair";
  return C::TA ? "dW" : C::TB ? "dX" : "product";
}

template <class C>
fg_status launch_tile(LinearParams& p, int cus, int64_t cols, void* stream, const char* what, int splits = 1) {
  FG_TRY(set_tiles<C>(p, cols, what, splits));
  const int grid = std::min(cus * C::OCC, p.num_tiles);
  print_tiles<C>(p, what, launch_name<C>(), splits, grid);
  hipLaunchKernelGGL((linear_tile_kernel<C>), dim3((unsigned)grid), dim3(C::THREADS), 0, (hipStream_t)stream, p);
  return launched(what);
}

template <class C>
fg_status launch_fewrow(const LinearParams& p, void* stream, const char* what) {
  const int64_t parts = ((int64_t)p.M + C::ROWS - 1) / C::ROWS, tiles = ((int64_t)p.N + C::OUT_N - 1) / C::OUT_N;
  if (print_launches())
    fprintf(stderr, "[fp8gemm] %s product M=%d N=%d K=%d few-row rows=%d cols=%d waves=%d grid=%lld\n", what, p.M, p.N, p.K,
            C::ROWS, C::COLS, C::WAVES, (long long)(parts * tiles));
  hipLaunchKernelGGL((fewrow_kernel<C>), dim3((unsigned)(parts * tiles)), dim3(C::THREADS), 0, (hipStream_t)stream, p,
                     (int)parts);
  return launched(what);
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

// The environment variable that overrides a plan (linear_plan.hpp).
const char* forced_plan() {
  const char* f = getenv("FG_LINEAR_PLAN");
  return f ? f : "";
}

// p's product as the plans see it, its slices laid out in p.
template <int E>
Product product(LinearParams& p, int64_t cols, bool mn) {
  p.nk = p.split_nk = slice_count(p.K, epi_int8(E) ? 1 : 2);
  return Product{p.M, cols, p.nk, epi_gated(E), mn};
}

// One forward product.
template <int E>
fg_status launch_linear(LinearParams& p, void* stream, const char* what) {
  int cus = 0;
  FG_TRY(usable_cus(&cus));
  const ForwardPlan plan = plan_forward(product<E>(p, p.N, false), cus, forced_plan());
  switch (plan.few) {
    case 0: return launch_fewrow<FewRow<E, 1, 1, 4, 2>>(p, stream, what);
    case 1: return launch_fewrow<FewRow<E, 1, 1, 8, 2>>(p, stream, what);
    case 2: return launch_fewrow<FewRow<E, 1, 2, 4, 2>>(p, stream, what);
    case 3: return launch_fewrow<FewRow<E, 2, 1, 4, 3>>(p, stream, what);
    case 4: return launch_fewrow<FewRow<E, 2, 2, 4, 2>>(p, stream, what);
    case 5: return launch_fewrow<FewRow<E, 4, 1, 4, 2>>(p, stream, what);
    case 6: return launch_fewrow<FewRow<E, 4, 2, 4, 2>>(p, stream, what);
    case 7: return launch_fewrow<FewRow<E, 4, 4, 4, 2>>(p, stream, what);
    default: return launch_planned<E>(p, plan.tile, p.N, cus, stream, what);
  }
}

// ---------------------------------------------------------------------------
// dX = pair . W and dW = pair^T . X, either or both.

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
  print_tiles<X>(x, what, "shared dX", splits, x.num_tiles + w.num_tiles);
  print_tiles<W>(w, what, "shared dW", 1, x.num_tiles + w.num_tiles);
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
  bool capped = false;
  FG_TRY(usable_cus(&cus, &capped));
  Product px{}, pw{};
  if (x) px = product<kEpiBf16>(*x, x->N, true);
  if (w) pw = product<kEpiBf16>(*w, w->N, true);
  const GradsPlan plan = plan_grads(x ? &px : nullptr, w ? &pw : nullptr, cus, capped, forced_plan());
  if (x) x->split_nk = plan.split_nk;
  if (plan.shared) {
    if (plan.splits == 1) return launch_both<kEpiBf16>(*x, plan.x, 1, *w, plan.w, stream, what);
    FG_TRY(launch_both<kEpiPartial>(*x, plan.x, plan.splits, *w, plan.w, stream, what));
    return launch_add(*x, plan.splits, stream, what);
  }
  if (x) {
    if (plan.splits > 1) {
      if (plan.x == kSmall)
        FG_TRY((launch_tile<SmallTile<kEpiPartial, false, true>>(*x, cus, x->N, stream, what, plan.splits)));
      else
        FG_TRY((launch_tile<MidTile<kEpiPartial, false, true>>(*x, cus, x->N, stream, what, plan.splits)));
      FG_TRY(launch_add(*x, plan.splits, stream, what));
    } else {
      FG_TRY((launch_planned<kEpiBf16, false, true>(*x, plan.x, x->N, cus, stream, what)));
    }
  }
  if (w) FG_TRY((launch_planned<kEpiBf16, true, true>(*w, plan.w, w->N, cus, stream, what)));
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
  if (M > kMaxRows) return set_error(FG_EUNSUPPORTED, "M=%d: more than 2^30 rows", M);
  if (N > kMaxRows / 2) return set_error(FG_EUNSUPPORTED, "%d output columns, more than 2^29", N);
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
// `partials` (with dW, 395 x 36 x 6232: 36 us without, 19 with; 595 x 175 x
// 3320: 26 and 21).
fg_status launch_recompute(LinearParams& g, float* partials, void* stream, const char* what) {
  int cus = 0;
  FG_TRY(usable_cus(&cus));
  const Product whole = product<kEpiGatedGrad>(g, g.half, false);
  const SplitPlan split = plan_recompute(whole, cus, forced_plan());
  if (split.splits == 1)
    return launch_planned<kEpiGatedGrad>(g, plan_tile(whole, cus, forced_plan()).kind, g.half, cus, stream, what);
  g.P = partials;
  g.ldp = 2 * g.half;
  g.split_nk = split.nk;
  FG_TRY((launch_tile<SmallTile<kEpiGatedPartial, false, false>>(g, cus, g.half, stream, what, split.splits)));
  return launch_gated_grad<true>(g, split.splits, stream, what);
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
  // 16 us, 5.5 TB/s; 4096 x 1024: 256 threads 6.1 us), four of a longer one
  // (4096 x 7168 fp32: 22 us, 6.7 TB/s from the last-level cache).
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
  if (M > kMaxRows) return set_error(FG_EUNSUPPORTED, "M=%d: more than 2^30 rows", M);
  if (F > kMaxRows / 4) return set_error(FG_EUNSUPPORTED, "F=%d: more than 2^28 hidden units", F);
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
    if (F > 0) x.P = (float*)((uint8_t*)workspace + pair_bytes(M, F));  // partials, where the plan splits the sum
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
