// int4.hip -- C entry points of the 4-bit cast and product (int4_kernel.hpp):
// argument checks and launches.  Nothing is launched after a failed check;
// nothing is allocated.

#include <algorithm>
#include <cstdio>

#include "host_common.hpp"
#include "int4_host.hpp"
#include "int4_kernel.hpp"

#define FG_TRY(x)                   \
  do {                              \
    fg_status st__ = (x);           \
    if (st__ != FG_OK) return st__; \
  } while (0)

namespace fg {

fg_status check_group(int group) {
  if (group != 32 && group != 64 && (group <= 0 || group % 128))
    return set_error(FG_EINVAL, "group=%d is not 32, 64 or a multiple of 128", group);
  return FG_OK;
}

namespace {

constexpr int kMaxK = 1 << 20;   // rows of activations of 2 MiB, offsets of a tile's rows in 32 bits
constexpr int kMaxRows = 1 << 30;

fg_status launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return set_error(FG_EHIP, "%s launch: %s", what, hipGetErrorString(e));
  return FG_OK;
}

template <typename T>
fg_status cast(const T* x, int64_t ldx, uint8_t* q, uint16_t* s, uint8_t* z, int N, int K, int group, void* stream,
               const char* what) {
  clear_error();
  if (N < 0 || K < 0) return set_error(FG_EINVAL, "negative size N=%d K=%d", N, K);
  if (K % 32) return set_error(FG_EALIGN, "K=%d is not a multiple of 32", K);
  FG_TRY(check_group(group));
  if (N == 0 || K == 0) return FG_OK;
  if (K > kMaxK) return set_error(FG_EUNSUPPORTED, "K=%d above 2^20", K);
  FG_TRY(require_ptr(x, 16, "x"));
  FG_TRY(require_ptr(q, 16, "q"));
  FG_TRY(require_ptr(s, 2, "s"));
  FG_TRY(require_ld(ldx, K, 16 / (int)sizeof(T), "ldx"));
  Int4CastParams p{};
  p.x = x; p.ldx = ldx; p.q = q; p.s = s; p.z = z;
  p.N = N; p.K = K; p.group = group;
  p.groups = int4_groups(K, group);
  p.words = int4_row_bytes(K) / 4;
  p.per_row = p.groups;
  p.units = (int64_t)N * p.per_row;
  const int lanes = group <= 128 ? group / 8 : 64;
  const int64_t blocks = std::min<int64_t>((p.units * lanes + 255) / 256, 1 << 20);
  const dim3 grid((unsigned)blocks), threads(256);
  switch (lanes) {
    case 4: hipLaunchKernelGGL((int4_cast_kernel<T, 4>), grid, threads, 0, (hipStream_t)stream, p); break;
    case 8: hipLaunchKernelGGL((int4_cast_kernel<T, 8>), grid, threads, 0, (hipStream_t)stream, p); break;
    case 16: hipLaunchKernelGGL((int4_cast_kernel<T, 16>), grid, threads, 0, (hipStream_t)stream, p); break;
    default: hipLaunchKernelGGL((int4_cast_kernel<T, 64>), grid, threads, 0, (hipStream_t)stream, p); break;
  }
  return launched(what);
}

template <class C>
fg_status launch_product(Int4Params& p, void* stream) {
  const int64_t tiles = ((int64_t)p.N + C::COLS - 1) / C::COLS;
  p.parts = (p.M + C::ROWS - 1) / C::ROWS;
  if (tiles * p.parts >= (1 << 30)) return set_error(FG_EUNSUPPORTED, "gemm_int4_nt: too many output tiles");
  if (print_launches())
    fprintf(stderr, "[fp8gemm] gemm_int4_nt M=%d N=%d K=%d group=%d rows=%d cols=%d waves=%d grid=%lld\n", p.M, p.N, p.K,
            p.group, C::ROWS, C::COLS, C::WAVES, (long long)(tiles * p.parts));
  hipLaunchKernelGGL((int4_product_kernel<C>), dim3((unsigned)(tiles * p.parts)), dim3(C::THREADS), 0,
                     (hipStream_t)stream, p);
  return launched("gemm_int4_nt");
}

template <int GPC>
fg_status launch_gpc(Int4Params& p, void* stream) {
  if (p.M <= 16) return launch_product<Int4Tile<GPC, 1, 1, 4, 2>>(p, stream);
  if (p.M <= 32) return launch_product<Int4Tile<GPC, 2, 2, 4, 2>>(p, stream);
  return launch_product<Int4Tile<GPC, 4, 2, 4, 1>>(p, stream);
}

}  // namespace
}  // namespace fg

using namespace fg;

extern "C" {

fg_status int4_cast_per_group(const float* w, int64_t ldw, uint8_t* q, uint16_t* s, uint8_t* z, int N, int K, int group,
                              void* stream) {
  return cast(w, ldw, q, s, z, N, K, group, stream, "int4_cast_per_group");
}

fg_status int4_cast_per_group_bf16(const uint16_t* w, int64_t ldw, uint8_t* q, uint16_t* s, uint8_t* z, int N, int K,
                                   int group, void* stream) {
  return cast(w, ldw, q, s, z, N, K, group, stream, "int4_cast_per_group_bf16");
}

fg_status gemm_int4_nt(const uint16_t* A, int64_t lda, const uint8_t* B, const uint16_t* sb, const uint8_t* zb,
                       uint16_t* D, int64_t ldd, int M, int N, int K, int group, void* stream) {
  clear_error();
  if (M < 0 || N < 0 || K < 0) return set_error(FG_EINVAL, "negative size M=%d N=%d K=%d", M, N, K);
  if (K % 32) return set_error(FG_EALIGN, "K=%d is not a multiple of 32", K);
  FG_TRY(check_group(group));
  if (M == 0 || N == 0) return FG_OK;
  if (M > kMaxRows || N > kMaxRows) return set_error(FG_EUNSUPPORTED, "M=%d N=%d: more than 2^30", M, N);
  if (K > kMaxK) return set_error(FG_EUNSUPPORTED, "K=%d above 2^20", K);
  FG_TRY(require_ptr(D, 2, "D"));
  FG_TRY(require_ld(ldd, N, 1, "ldd"));
  Int4Params p{};
  p.D = D; p.ldd = ldd; p.M = M; p.N = N; p.K = K; p.group = group;
  if (K > 0) {
    FG_TRY(require_ptr(A, 16, "A"));
    FG_TRY(require_ld(lda, K, 8, "lda"));
    if (lda > ((int64_t)1 << 21)) return set_error(FG_EUNSUPPORTED, "lda=%lld: rows above 4 MiB", (long long)lda);
    FG_TRY(require_ptr(B, 16, "B"));
    FG_TRY(require_ptr(sb, 2, "sb"));
    p.A = A; p.lda = lda; p.B = B; p.s = sb; p.z = zb;
    p.groups = int4_groups(K, group);
    p.row_bytes = int4_row_bytes(K);
    p.wide = int4_wide(K, sb, zb);
  }
  if (group == 32) return launch_gpc<4>(p, stream);
  if (group == 64) return launch_gpc<2>(p, stream);
  return launch_gpc<1>(p, stream);
}

}  // extern "C"
