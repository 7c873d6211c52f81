// linear.hip -- C entry points of the 8-bit-integer products and the gated
// feed-forward block (linear_kernel.hpp): argument checks, plans, launches.
// Nothing is launched after a failed check; nothing is allocated.

#include <algorithm>
#include <cmath>

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
// and the cheapest runs.  The estimates only rank candidates.

template <class C>
fg_status launch_tile(LinearParams& p, int cus, int64_t cols, void* stream, const char* what) {
  const int64_t tm = ((int64_t)p.M + C::BM - 1) / C::BM, tn = (cols + C::OUT_N - 1) / C::OUT_N;
  if (tm * tn >= (1 << 30)) return set_error(FG_EUNSUPPORTED, "%s: too many output tiles", what);
  p.tiles_m = (int)tm;
  p.tiles_n = (int)tn;
  p.num_tiles = (int)(tm * tn);
  p.group_m = 8;
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
// all of them (clock and cache contention).
double tile_us(double tiles, int cus, int nk, double idle, double busy) {
  const double load = tiles < cus ? tiles / cus : 1.0;
  return 3.0 + ceil(tiles / cus) * (nk * (idle + (busy - idle) * load) + 1.5);
}

// Two workgroups per CU: a round that leaves one workgroup per CU is cheaper.
double tile2_us(double tiles, int cus, int nk, double one, double two) {
  const double full = floor(tiles / (2 * cus)), rest = tiles - full * 2 * cus;
  return 3.0 + full * (nk * two + 1.5) + (rest > 0 ? nk * (rest > cus ? two : one) + 1.5 : 0);
}

template <class C>
fg_status launch_fewrow(const LinearParams& p, void* stream, const char* what) {
  const int64_t parts = ((int64_t)p.M + C::ROWS - 1) / C::ROWS, tiles = ((int64_t)p.N + C::OUT_N - 1) / C::OUT_N;
  if (parts * tiles >= (1 << 23)) return set_error(FG_EUNSUPPORTED, "%s: too many output tiles", what);
  hipLaunchKernelGGL((fewrow_kernel<C>), dim3((unsigned)(parts * tiles)), dim3(C::THREADS), 0, (hipStream_t)stream, p,
                     (int)parts);
  return launched(what);
}

// A few-row workgroup fetches its rows' slices at about 80 GB/s; a launch's
// rounds each add about 2 us of latency.
double fewrow_us(const LinearParams& p, bool gated, int cus, int mf, int cf) {
  const double parts = (double)((p.M + 16 * mf - 1) / (16 * mf)), out_n = gated ? 8 * cf : 16 * cf;
  const double groups = parts * ceil(p.N / out_n), bytes = (double)p.nk * 128 * (std::min(p.M, 16 * mf) + 16 * cf);
  return 1.0 + ceil(groups / cus) * (2.0 + bytes / 80e3);
}

template <int E, bool TA = false, bool TB = false>
fg_status launch_linear(LinearParams& p, void* stream, const char* what) {
  int cus = 0;
  FG_TRY(usable_cus(&cus));
  constexpr bool gated = epi_gated(E);
  const int64_t cols = E == kEpiGatedGrad ? p.half : p.N;
  p.nk = (int)std::max<int64_t>(1, ((int64_t)p.K * (epi_int8(E) ? 1 : 2) + 127) / 128);
  // 256 x 256: 1.2 us a slice alone, 1.7 with every CU at work (4096 x 4096 x
  // 7168 int8 95 us).  128 x 128, two workgroups of four waves: 0.66 alone,
  // 1.0 for both (112 us on that shape); one of eight waves with four stages:
  // 0.48 and 0.58 (34 us on 1000 x 4096 x 7168, 71 on 256 x 256 tiles).
  // 64 x 64 with eight stages: 0.33 (20 us on 256 x 4096 x 7168, 27 on
  // 128 x 128 tiles).
  const double big = tile_us(tile_count(p, cols, gated, 256, 256), cus, p.nk, 1.2, 1.7);
  const double mid2 = tile2_us(tile_count(p, cols, gated, 128, 128), cus, p.nk, 0.66, 1.0);
  const double mid = tile_us(tile_count(p, cols, gated, 128, 128), cus, p.nk, 0.48, 0.58);
  const double small = tile_us(tile_count(p, cols, gated, 64, 64), cus, p.nk, 0.33, 0.33);
  const double tile = std::min(std::min(big, mid2), std::min(mid, small));
  if constexpr (!TA && !TB && E != kEpiGatedGrad) {
    if (p.M <= 256) {
      static const int shapes[][2] = {{1, 1}, {1, 2}, {2, 1}, {2, 2}, {4, 1}, {4, 2}, {4, 4}};
      int best = -1;
      double least = tile;
      for (int i = 0; i < 7; ++i) {
        const double t = fewrow_us(p, gated, cus, shapes[i][0], shapes[i][1]);
        if (t < least) {
          least = t;
          best = i;
        }
      }
      switch (best) {
        case 0:
          // long chains of slices are shared out over eight waves (1 x 2112 x
          // 7168 5.1 us against 6.1, 1 x 2048 x 1024 3.1 against 2.8)
          if (p.nk >= 32) return launch_fewrow<FewRow<E, 1, 1, 8, 2>>(p, stream, what);
          return launch_fewrow<FewRow<E, 1, 1, 4, 2>>(p, stream, what);
        case 1: return launch_fewrow<FewRow<E, 1, 2, 4, 2>>(p, stream, what);
        case 2: return launch_fewrow<FewRow<E, 2, 1, 4, 3>>(p, stream, what);
        case 3: return launch_fewrow<FewRow<E, 2, 2, 4, 2>>(p, stream, what);
        case 4: return launch_fewrow<FewRow<E, 4, 1, 4, 2>>(p, stream, what);
        case 5: return launch_fewrow<FewRow<E, 4, 2, 4, 2>>(p, stream, what);
        case 6: return launch_fewrow<FewRow<E, 4, 4, 4, 2>>(p, stream, what);
        default: break;
      }
    }
  }
  if (tile == big) return launch_tile<LinearTile<E, 256, 256, 4, 2, 2, TA, TB>>(p, cus, cols, stream, what);
  if (tile == mid2) return launch_tile<LinearTile<E, 128, 128, 2, 2, 2, TA, TB>>(p, cus, cols, stream, what);
  if (tile == mid) return launch_tile<LinearTile<E, 128, 128, 4, 2, 4, TA, TB>>(p, cus, cols, stream, what);
  return launch_tile<LinearTile<E, 64, 64, 2, 2, 8, TA, TB>>(p, cus, cols, stream, what);
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

int64_t backward_bytes(int M, int F) { return round_up((int64_t)M * pair_cols(F) * 2, 256); }

template <typename T>
fg_status cast_rows(const T* x, int64_t ldx, int8_t* q, float* s, int M, int K, void* stream, const char* what) {
  clear_error();
  if (M < 0 || K < 0) return set_error(FG_EINVAL, "negative size M=%d K=%d", M, K);
  if (K % 16) return set_error(FG_EALIGN, "K=%d is not a multiple of 16", K);
  if (M == 0 || K == 0) return FG_OK;
  FG_TRY(require_ptr(x, 16, "x"));
  FG_TRY(require_ptr(q, 16, "q"));
  FG_TRY(require_ptr(s, 4, "s"));
  FG_TRY(require_ld(ldx, K, 16 / (int)sizeof(T), "ldx"));
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
  p.A = (const uint8_t*)A; p.lda = lda; p.B = (const uint8_t*)B; p.ldb = ldb; p.sa = sa; p.sb = sb;
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
  p.A = (const uint8_t*)X; p.lda = ldx; p.B = (const uint8_t*)W; p.ldb = ldw; p.sa = sx; p.sb = sw;
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
  p.A = (const uint8_t*)X; p.lda = 2 * ldx; p.B = (const uint8_t*)W; p.ldb = 2 * ldw;
  p.D = H; p.ldd = ldh; p.P = P; p.ldp = ldp; p.M = M; p.N = F; p.K = K; p.act = activation;
  return launch_linear<kEpiGated>(p, stream, "gated_ffn_bf16");
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
  FG_TRY(check_workspace(workspace, workspace_bytes, M > 0 && F > 0 ? backward_bytes(M, F) : 0));
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
    if (P) {
      const int64_t blocks = ((int64_t)M * (g.half / 8) + 255) / 256;
      hipLaunchKernelGGL(gated_grad_kernel, dim3((unsigned)std::min<int64_t>(blocks, 1 << 16)), dim3(256), 0,
                         (hipStream_t)stream, g);
      FG_TRY(launched(what));
    } else {
      FG_TRY((launch_linear<kEpiGatedGrad>(g, stream, what)));
    }
  }
  // With M or F of zero the reductions below are empty and write zeros.
  if (dX && M > 0) {
    LinearParams g = p;
    g.A = (const uint8_t*)workspace; g.lda = 2 * pair_ld; g.B = (const uint8_t*)W; g.ldb = 2 * ldw;
    g.D = dX; g.ldd = lddx; g.M = M; g.N = K; g.K = F > 0 ? (int)pair_ld : 0;
    FG_TRY((launch_linear<kEpiBf16, false, true>(g, stream, what)));
  }
  if (dW && F > 0) {
    LinearParams g = p;
    g.A = (const uint8_t*)workspace; g.lda = 2 * pair_ld; g.B = (const uint8_t*)X; g.ldb = 2 * ldx;
    g.D = dW; g.ldd = lddw; g.M = (int)pair_ld; g.N = K; g.K = M;
    FG_TRY((launch_linear<kEpiBf16, true, true>(g, stream, what)));
  }
  return FG_OK;
}

int64_t fg_gated_ffn_backward_workspace_bytes(int M, int F) {
  if (M < 0 || F < 0 || M > kMaxRows || F > kMaxRows / 4) return -1;
  return M > 0 && F > 0 ? backward_bytes(M, F) : 0;
}

}  // extern "C"
