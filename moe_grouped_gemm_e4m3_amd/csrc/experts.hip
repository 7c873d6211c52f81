// experts.hip -- C entry points of the expert router (route_kernel.hpp) and of
// the expert layers for a few tokens (experts_kernel.hpp): argument checks and
// launches.  Nothing is launched after a failed check; nothing is allocated.

#include <algorithm>
#include <cstdio>

#include "experts_kernel.hpp"
#include "host_common.hpp"
#include "int4_host.hpp"
#include "route_kernel.hpp"

#define FG_TRY(x)                   \
  do {                              \
    fg_status st__ = (x);           \
    if (st__ != FG_OK) return st__; \
  } while (0)

namespace fg {
namespace {

constexpr int kMaxTokens = 1 << 20;
constexpr int kMaxWidth = 1 << 16;  // K and F of a layer: offsets of 64 tokens' rows and of a weight tile in 32 bits
constexpr int64_t kMaxLd = (int64_t)1 << 21;

fg_status launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return set_error(FG_EHIP, "%s launch: %s", what, hipGetErrorString(e));
  return FG_OK;
}

// ---------------------------------------------------------------------------
// router

template <typename L, int SLOTS>
fg_status launch_route(const RouteParams& p, void* stream) {
  const dim3 grid((unsigned)(((int64_t)p.T + kRouteWaves - 1) / kRouteWaves)), threads(64 * kRouteWaves);
  if (p.bias || p.groups > 1)
    hipLaunchKernelGGL((route_kernel<L, SLOTS, true>), grid, threads, 0, (hipStream_t)stream, p);
  else
    hipLaunchKernelGGL((route_kernel<L, SLOTS, false>), grid, threads, 0, (hipStream_t)stream, p);
  return launched("moe_route");
}

template <typename L>
fg_status launch_route(const RouteParams& p, void* stream) {
  if (p.E <= 64) return launch_route<L, 1>(p, stream);
  if (p.E <= 128) return launch_route<L, 2>(p, stream);
  if (p.E <= 256) return launch_route<L, 4>(p, stream);
  if (p.E <= 512) return launch_route<L, 8>(p, stream);
  return launch_route<L, 16>(p, stream);
}

template <typename L, int SLOTS>
fg_status launch_route_backward(const RouteGradParams& p, void* stream) {
  const dim3 grid((unsigned)(((int64_t)p.T + kRouteWaves - 1) / kRouteWaves));
  hipLaunchKernelGGL((route_backward_kernel<L, SLOTS>), grid, dim3(64 * kRouteWaves), 0, (hipStream_t)stream, p);
  return launched("moe_route_backward");
}

template <typename L>
fg_status launch_route_backward(const RouteGradParams& p, void* stream) {
  if (p.E <= 64) return launch_route_backward<L, 1>(p, stream);
  if (p.E <= 128) return launch_route_backward<L, 2>(p, stream);
  if (p.E <= 256) return launch_route_backward<L, 4>(p, stream);
  if (p.E <= 512) return launch_route_backward<L, 8>(p, stream);
  return launch_route_backward<L, 16>(p, stream);
}

fg_status check_route(int T, int E, int k, int scoring) {
  if (T < 0) return set_error(FG_EINVAL, "negative size T=%d", T);
  if (E <= 0) return set_error(FG_EINVAL, "E=%d experts", E);
  if (k <= 0 || k > E) return set_error(FG_EINVAL, "k=%d of %d experts", k, E);
  if (scoring != FG_SCORE_SOFTMAX && scoring != FG_SCORE_SIGMOID)
    return set_error(FG_EINVAL, "scoring=%d is not known", scoring);
  if (E > kMaxRouteExperts) return set_error(FG_EUNSUPPORTED, "E=%d: more than %d experts", E, kMaxRouteExperts);
  if (k > kMaxRouteChoices) return set_error(FG_EUNSUPPORTED, "k=%d: more than %d choices", k, kMaxRouteChoices);
  return FG_OK;
}

template <typename L>
fg_status route(const L* logits, int64_t ld, const float* bias, int32_t* ids, float* w, int T, int E, int k, int scoring,
                int groups, int top, int normalize, float scale, void* stream) {
  clear_error();
  FG_TRY(check_route(T, E, k, scoring));
  if (groups <= 0 || E % groups) return set_error(FG_EINVAL, "groups=%d does not divide E=%d", groups, E);
  if (top <= 0 || top > groups) return set_error(FG_EINVAL, "top_groups=%d of %d groups", top, groups);
  if (groups > kMaxRouteGroups) return set_error(FG_EUNSUPPORTED, "groups=%d: more than %d", groups, kMaxRouteGroups);
  if (T == 0) return FG_OK;
  FG_TRY(require_ptr(logits, sizeof(L), "logits"));
  FG_TRY(require_ld(ld, E, 1, "ld"));
  if (bias) FG_TRY(require_ptr(bias, 4, "bias"));
  FG_TRY(require_ptr(ids, 4, "ids"));
  FG_TRY(require_ptr(w, 4, "weights"));
  RouteParams p{};
  p.logits = logits; p.ld = ld; p.bias = bias; p.ids = ids; p.w = w;
  p.T = T; p.E = E; p.k = k; p.groups = groups; p.top = top;
  p.sigmoid = scoring == FG_SCORE_SIGMOID; p.normalize = normalize != 0; p.scale = scale;
  return launch_route<L>(p, stream);
}

template <typename L>
fg_status route_backward(const float* dw, const L* logits, int64_t ld, const int32_t* ids, L* dl, int64_t ld_dl, int T,
                         int E, int k, int scoring, int normalize, float scale, void* stream) {
  clear_error();
  FG_TRY(check_route(T, E, k, scoring));
  if (T == 0) return FG_OK;
  FG_TRY(require_ptr(dw, 4, "dweights"));
  FG_TRY(require_ptr(logits, sizeof(L), "logits"));
  FG_TRY(require_ld(ld, E, 1, "ld"));
  FG_TRY(require_ptr(ids, 4, "ids"));
  FG_TRY(require_ptr(dl, sizeof(L), "dlogits"));
  FG_TRY(require_ld(ld_dl, E, 1, "ld_dl"));
  RouteGradParams p{};
  p.dw = dw; p.logits = logits; p.ld = ld; p.ids = ids; p.dl = dl; p.ld_dl = ld_dl;
  p.T = T; p.E = E; p.k = k;
  p.sigmoid = scoring == FG_SCORE_SIGMOID; p.normalize = normalize != 0; p.scale = scale;
  return launch_route_backward<L>(p, stream);
}

// ---------------------------------------------------------------------------
// expert layers

template <class C>
fg_status launch_down(const ExpertParams& p, int passes, void* stream, const char* what) {
  const int tiles = (p.K + C::COLS - 1) / C::COLS;
  if (print_launches())
    fprintf(stderr, "[fp8gemm] %s down T=%d K=%d F=%d rows=%d cols=%d waves=%d grid=%dx%d\n", what, p.T, p.K, p.F, C::ROWS,
            C::COLS, C::WAVES, tiles, passes);
  hipLaunchKernelGGL((experts_down_kernel<C>), dim3(tiles, passes), dim3(C::THREADS), C::lds_bytes(p.T),
                     (hipStream_t)stream, p);
  return launched(what);
}

template <int FMT, int GPC>
fg_status launch_layer(const ExpertParams& p, void* stream, const char* what) {
  const int passes = (p.T + kLayerTokens - 1) / kLayerTokens;
  const int pairs = std::min(p.T, kLayerTokens) * p.k;
  ExpertParams u = p;
  u.by_pair = pairs < p.E;
  if (p.F > 0) {
    const dim3 grid(p.F / 16, u.by_pair ? pairs : p.E, passes);
    if (print_launches())
      fprintf(stderr, "[fp8gemm] %s up T=%d F=%d K=%d grid=%dx%dx%d\n", what, p.T, p.F, p.K, grid.x, grid.y, grid.z);
    hipLaunchKernelGGL((experts_up_kernel<FMT, GPC>), grid, dim3(64 * kUpWaves), 0, (hipStream_t)stream, u);
    FG_TRY(launched(what));
  }
  if (p.T <= 16) return launch_down<DownTile<FMT, GPC, 1, 1, 8, 2>>(p, passes, stream, what);
  return launch_down<DownTile<FMT, GPC, 2, 1, 8, 1>>(p, passes, stream, what);
}

int64_t layer_bytes(int T, int k, int F) { return (int64_t)T * k * F * 4; }

fg_status check_layer(const ExpertParams& p, int mult, const void* workspace, int64_t workspace_bytes, int scale_align,
                      bool* empty) {
  *empty = false;
  if (p.T < 0 || p.K < 0 || p.F < 0) return set_error(FG_EINVAL, "negative size T=%d K=%d F=%d", p.T, p.K, p.F);
  if (p.k <= 0) return set_error(FG_EINVAL, "k=%d choices", p.k);
  if (p.E <= 0) return set_error(FG_EINVAL, "E=%d experts", p.E);
  if (p.K % mult) return set_error(FG_EALIGN, "K=%d is not a multiple of %d", p.K, mult);
  if (p.F % mult) return set_error(FG_EALIGN, "F=%d is not a multiple of %d", p.F, mult);
  if (p.act != FG_ACT_SILU && p.act != FG_ACT_GELU_TANH) return set_error(FG_EINVAL, "activation=%d is not known", p.act);
  if (p.T == 0 || p.K == 0) {
    *empty = true;
    return FG_OK;
  }
  if (p.T > kMaxTokens) return set_error(FG_EUNSUPPORTED, "T=%d: more than 2^20 tokens", p.T);
  if (p.K > kMaxWidth || p.F > kMaxWidth) return set_error(FG_EUNSUPPORTED, "K=%d F=%d: more than 2^16", p.K, p.F);
  if (p.E > kMaxExperts) return set_error(FG_EUNSUPPORTED, "E=%d: more than %d experts", p.E, kMaxExperts);
  if (p.k > kMaxChoices) return set_error(FG_EUNSUPPORTED, "k=%d: more than %d choices", p.k, kMaxChoices);
  FG_TRY(require_ptr(p.X, 16, "X"));
  FG_TRY(require_ld(p.ldx, p.K, 8, "ldx"));
  if (p.ldx > kMaxLd) return set_error(FG_EUNSUPPORTED, "ldx=%lld: rows above 4 MiB", (long long)p.ldx);
  FG_TRY(require_ptr(p.ids, 4, "ids"));
  FG_TRY(require_ptr(p.w, 4, "weights"));
  FG_TRY(require_ptr(p.D, 2, "D"));
  FG_TRY(require_ld(p.ldd, p.K, 1, "ldd"));
  if (p.F > 0) {
    FG_TRY(require_ptr(p.W1, 16, "W1"));
    FG_TRY(require_ptr(p.W2, 16, "W2"));
    FG_TRY(require_ptr(p.s1, scale_align, "s1"));
    FG_TRY(require_ptr(p.s2, scale_align, "s2"));
  }
  const int64_t need = layer_bytes(p.T, p.k, p.F);
  if (workspace_bytes < 0) return set_error(FG_EINVAL, "workspace_bytes=%lld is negative", (long long)workspace_bytes);
  if (!workspace && workspace_bytes > 0) return set_error(FG_EINVAL, "workspace is NULL");
  if (workspace && ((uintptr_t)workspace & 255)) return set_error(FG_EALIGN, "workspace is not 256-byte aligned");
  if (workspace_bytes < need)
    return set_error(FG_EINVAL, "workspace_bytes=%lld is smaller than the %lld needed", (long long)workspace_bytes,
                     (long long)need);
  return FG_OK;
}

}  // namespace
}  // namespace fg

using namespace fg;

extern "C" {

fg_status moe_route(const float* logits, int64_t ld, const float* bias, int32_t* ids, float* weights, int T, int E, int k,
                    int scoring, int groups, int top_groups, int normalize, float scale, void* stream) {
  return route(logits, ld, bias, ids, weights, T, E, k, scoring, groups, top_groups, normalize, scale, stream);
}

fg_status moe_route_bf16(const uint16_t* logits, int64_t ld, const float* bias, int32_t* ids, float* weights, int T, int E,
                         int k, int scoring, int groups, int top_groups, int normalize, float scale, void* stream) {
  return route(logits, ld, bias, ids, weights, T, E, k, scoring, groups, top_groups, normalize, scale, stream);
}

fg_status moe_route_backward(const float* dweights, const float* logits, int64_t ld, const int32_t* ids, float* dlogits,
                             int64_t ld_dl, int T, int E, int k, int scoring, int normalize, float scale, void* stream) {
  return route_backward(dweights, logits, ld, ids, dlogits, ld_dl, T, E, k, scoring, normalize, scale, stream);
}

fg_status moe_route_backward_bf16(const float* dweights, const uint16_t* logits, int64_t ld, const int32_t* ids,
                                  uint16_t* dlogits, int64_t ld_dl, int T, int E, int k, int scoring, int normalize,
                                  float scale, void* stream) {
  return route_backward(dweights, logits, ld, ids, dlogits, ld_dl, T, E, k, scoring, normalize, scale, stream);
}

int64_t fg_moe_ffn_workspace_bytes(int T, int k, int F) {
  if (T < 0 || k < 0 || F < 0 || T > kMaxTokens || k > kMaxChoices || F > kMaxWidth) return -1;
  return layer_bytes(T, k, F);
}

fg_status moe_ffn_fp8(const uint16_t* X, int64_t ldx, const uint8_t* W1, const float* s1, const uint8_t* W2,
                      const float* s2, const int32_t* ids, const float* weights, uint16_t* D, int64_t ldd, int T, int k,
                      int E, int F, int K, int activation, void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  ExpertParams p{};
  p.X = X; p.ldx = ldx; p.W1 = W1; p.s1 = s1; p.W2 = W2; p.s2 = s2; p.ids = ids; p.w = weights; p.D = D; p.ldd = ldd;
  p.H = (uint16_t*)workspace;
  p.T = T; p.k = k; p.E = E; p.F = F; p.K = K; p.act = activation;
  bool empty;
  FG_TRY(check_layer(p, 16, workspace, workspace_bytes, 4, &empty));
  if (empty) return FG_OK;
  p.row1 = K; p.row2 = F;
  p.groups1 = (K + 127) / 128; p.groups2 = (F + 127) / 128;
  return launch_layer<kFp8Block, 1>(p, stream, "moe_ffn_fp8");
}

fg_status moe_ffn_int4(const uint16_t* X, int64_t ldx, const uint8_t* W1, const uint16_t* s1, const uint8_t* z1,
                       const uint8_t* W2, const uint16_t* s2, const uint8_t* z2, const int32_t* ids, const float* weights,
                       uint16_t* D, int64_t ldd, int T, int k, int E, int F, int K, int group, int activation,
                       void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  ExpertParams p{};
  p.X = X; p.ldx = ldx; p.W1 = W1; p.s1 = s1; p.z1 = z1; p.W2 = W2; p.s2 = s2; p.z2 = z2; p.ids = ids; p.w = weights;
  p.D = D; p.ldd = ldd;
  p.H = (uint16_t*)workspace;
  p.T = T; p.k = k; p.E = E; p.F = F; p.K = K; p.act = activation; p.group = group;
  FG_TRY(check_group(group));
  bool empty;
  FG_TRY(check_layer(p, 32, workspace, workspace_bytes, 2, &empty));
  if (empty) return FG_OK;
  p.row1 = int4_row_bytes(K); p.row2 = int4_row_bytes(F);
  p.groups1 = int4_groups(K, group); p.groups2 = int4_groups(F, group);
  p.wide1 = int4_wide(K, s1, z1); p.wide2 = int4_wide(F, s2, z2);
  const char* what = "moe_ffn_int4";
  if (group == 32) return launch_layer<kInt4Group, 4>(p, stream, what);
  if (group == 64) return launch_layer<kInt4Group, 2>(p, stream, what);
  return launch_layer<kInt4Group, 1>(p, stream, what);
}

}  // extern "C"
