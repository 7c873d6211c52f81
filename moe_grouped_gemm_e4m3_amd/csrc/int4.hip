// int4.hip -- C entry points of the 4-bit cast and product (int4_kernel.hpp):
// argument checks and launches.  Nothing is launched after a failed check;
// nothing is allocated.

#include <algorithm>
#include <cstdio>
#include <cstdlib>

#include "decode_plan.hpp"
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
constexpr int kMaxM = 1 << 20, kMaxN = 1 << 26;  // a grid's threads in 32 bits

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

struct ProductLaunch {
  Int4Params& p;
  Int4Plan plan;
  float* partial;
  void* stream;

  template <class C>
  fg_status split() const {
    const int64_t tiles = ceil_div(p.N, C::COLS);
    p.parts = ceil_div(p.M, C::ROWS);
    if (tiles * p.parts * C::THREADS > 0xffffffff) return set_error(FG_EUNSUPPORTED, "gemm_int4_nt: too many output tiles");
    print();
    hipLaunchKernelGGL((int4_product_kernel<C>), dim3((unsigned)(tiles * p.parts)), dim3(C::THREADS), 0, (hipStream_t)stream, p);
    return launched("gemm_int4_nt");
  }

  template <class C>
  fg_status wide() const {
    const dim3 grid(ceil_div(p.N, C::COLS), ceil_div(p.M, C::ROWS), plan.k_parts);
    if (grid.y > 65535) return set_error(FG_EUNSUPPORTED, "gemm_int4_nt: M=%d: too many row tiles", p.M);
    print();
    hipLaunchKernelGGL((int4_wide_kernel<C>), grid, dim3(C::THREADS), 0, (hipStream_t)stream, p, partial);
    FG_TRY(launched("gemm_int4_nt"));
    if (plan.k_parts == 1) return FG_OK;
    const int64_t blocks = ((int64_t)p.M * p.N + 1023) / 1024;
    hipLaunchKernelGGL(join_parts_kernel, dim3((unsigned)std::min<int64_t>(blocks, 1 << 16)), dim3(256), 0, (hipStream_t)stream,
                       partial, plan.k_parts, p.D, p.ldd, p.M, p.N);
    return launched("gemm_int4_nt");
  }

  void print() const {
    if (print_launches())
      fprintf(stderr, "[fp8gemm] gemm_int4_nt M=%d N=%d K=%d group=%d %s parts=%d\n", p.M, p.N, p.K, p.group,
              kInt4Names[plan.kind], plan.k_parts);
  }

  template <class Fmt>
  fg_status run() const {
    switch (plan.kind) {
      case kSplit2: return split<Int4Tile<Fmt, 2, 1, 4, 2>>();
      case kSplit2Deep: return split<Int4Tile<Fmt, 2, 1, 8, 2>>();
      case kSplit8: return split<Int4Tile<Fmt, 8, 1, 4, 2>>();
      case kSplit8Deep: return split<Int4Tile<Fmt, 8, 1, 8, 2>>();
      case kSplit16: return split<Int4Tile<Fmt, 16, 1, 4, 2>>();
      case kSplit16Deep: return split<Int4Tile<Fmt, 16, 1, 6, 2>>();
      case kWide16: return wide<Int4Wide<Fmt, 16, 1, 8, 2>>();
      case kWide32: return wide<Int4Wide<Fmt, 32, 1, 8, 2>>();
      default: return wide<Int4Wide<Fmt, 64, 1, 8, 2>>();
    }
  }
};

Int4Plan planned(int M, int N, int K) {
  const char* forced = getenv("FG_DECODE_PLAN");
  return plan_int4(M, N, K, forced ? forced : "");
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
                       uint16_t* D, int64_t ldd, int M, int N, int K, int group, void* workspace, int64_t workspace_bytes,
                       void* stream) {
  clear_error();
  if (M < 0 || N < 0 || K < 0) return set_error(FG_EINVAL, "negative size M=%d N=%d K=%d", M, N, K);
  if (K % 32) return set_error(FG_EALIGN, "K=%d is not a multiple of 32", K);
  FG_TRY(check_group(group));
  if (M == 0 || N == 0) return FG_OK;
  if (M > kMaxM) return set_error(FG_EUNSUPPORTED, "M=%d: more than 2^20 rows", M);
  if (N > kMaxN) return set_error(FG_EUNSUPPORTED, "N=%d: more than 2^26 columns", N);
  if (K > kMaxK) return set_error(FG_EUNSUPPORTED, "K=%d above 2^20", K);
  const Int4Plan plan = planned(M, N, K);
  const int64_t need = int4_partial_bytes(M, N, plan);
  if (workspace_bytes < 0) return set_error(FG_EINVAL, "workspace_bytes=%lld is negative", (long long)workspace_bytes);
  if (!workspace && workspace_bytes > 0) return set_error(FG_EINVAL, "workspace is NULL");
  if (workspace && ((uintptr_t)workspace & 255)) return set_error(FG_EALIGN, "workspace is not 256-byte aligned");
  if (workspace_bytes < need)
    return set_error(FG_EINVAL, "workspace_bytes=%lld is smaller than the %lld needed", (long long)workspace_bytes,
                     (long long)need);
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
  }
  return with_int4_format(group, zb != nullptr, ProductLaunch{p, plan, (float*)workspace, stream});
}

int64_t fg_int4_workspace_bytes(int M, int N, int K) {
  if (M < 0 || N < 0 || K < 0 || K % 32 || M > kMaxM || N > kMaxN || K > kMaxK) return -1;
  return M > 0 && N > 0 ? int4_partial_bytes(M, N, planned(M, N, K)) : 0;
}

}  // extern "C"
