// experts.hip -- C entry points of the expert router (route_kernel.hpp) and of
// the expert layers for a few tokens (experts_kernel.hpp): argument checks and
// launches.  Nothing is launched after a failed check; nothing is allocated.

#include <algorithm>
#include <atomic>
#include <cstdio>
#include <cstdlib>

#include "decode_plan.hpp"
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

constexpr int kMaxTokens = 1 << 20, kMaxRouted = 1 << 25;  // the router's threads in 32 bits
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
  const dim3 grid(ceil_div(p.T, kRouteWaves)), threads(64 * kRouteWaves);
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
  const dim3 grid(ceil_div(p.T, kRouteWaves));
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
  if (T > kMaxRouted) return set_error(FG_EUNSUPPORTED, "T=%d: more than 2^25 tokens", T);
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

// More than 64 KiB of dynamic LDS has to be asked for: once for a kernel and device
// (a bit of `allowed`), and the most there is, since the limit is the process's and
// another thread's call may need more than this one.
fg_status allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>& allowed, const char* what) {
  if (bytes > kLds) return set_error(FG_EUNSUPPORTED, "%s: %d bytes of LDS", what, bytes);
  int device = 0;
  hipError_t e = hipGetDevice(&device);
  if (e != hipSuccess) return set_error(FG_EHIP, "%s: hipGetDevice: %s", what, hipGetErrorString(e));
  const uint64_t bit = device < 64 ? (uint64_t)1 << device : 0;
  if (allowed.load() & bit) return FG_OK;
  e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e != hipSuccess) return set_error(FG_EHIP, "%s: %d bytes of LDS: %s", what, kLds, hipGetErrorString(e));
  allowed.fetch_or(bit);
  return FG_OK;
}

struct LayerLaunch {
  const ExpertParams& p;
  LayerPlan plan;
  int passes;  // of 64 tokens
  float* partial;
  void* stream;
  const char* what;

  void print(const char* kernel, const char* kind, int parts) const {
    if (print_launches())
      fprintf(stderr, "[fp8gemm] %s %s T=%d k=%d E=%d F=%d K=%d %s parts=%d\n", what, kernel, p.T, p.k, p.E, p.F, p.K, kind,
              parts);
  }

  template <class C>
  fg_status up() const {
    const int pairs = std::min(p.T, kLayerTokens) * p.k;
    ExpertParams u = p;
    u.by_pair = pairs < p.E;
    const dim3 grid(ceil_div(p.F, C::UNITS), u.by_pair ? pairs : p.E, passes);
    print("up", kUpNames[plan.up], 1);
    if constexpr (C::WIDE)
      hipLaunchKernelGGL((experts_wide_up_kernel<C>), grid, dim3(C::THREADS), 0, (hipStream_t)stream, u);
    else
      hipLaunchKernelGGL((experts_up_kernel<C>), grid, dim3(C::THREADS), 0, (hipStream_t)stream, u);
    return launched(what);
  }

  template <class C>
  fg_status down() const {
    const int lds = down_lds(C::Fmt::FP8, plan.down, std::min(p.T, kLayerTokens), p.E, p.k);
    static std::atomic<uint64_t> allowed{0};
    FG_TRY(allow_lds((const void*)experts_down_kernel<C>, lds, allowed, what));
    print("down", kDownNames[plan.down], 1);
    hipLaunchKernelGGL((experts_down_kernel<C>), dim3(ceil_div(p.K, C::COLS), passes), dim3(C::THREADS), lds,
                       (hipStream_t)stream, p);
    return launched(what);
  }

  // A pass of tokens at a time: they share the partial sums' place.
  template <class C>
  fg_status down_wide() const {
    const int lds = down_lds(C::Fmt::FP8, plan.down, std::min(p.T, kLayerTokens), p.E, p.k);
    static std::atomic<uint64_t> allowed{0};
    FG_TRY(allow_lds((const void*)experts_wide_down_kernel<C>, lds, allowed, what));
    for (int t0 = 0; t0 < p.T; t0 += kLayerTokens) {
      const int T = std::min(kLayerTokens, p.T - t0);
      print("down", kDownNames[plan.down], plan.parts);
      hipLaunchKernelGGL((experts_wide_down_kernel<C>), dim3(ceil_div(p.K, C::COLS), plan.parts), dim3(C::THREADS), lds,
                         (hipStream_t)stream, p, t0, partial);
      FG_TRY(launched(what));
      if (plan.parts == 1) continue;
      hipLaunchKernelGGL(join_parts_kernel, dim3(ceil_div((int64_t)T * p.K, 1024)), dim3(256), 0, (hipStream_t)stream, partial,
                         plan.parts, p.D + (int64_t)t0 * p.ldd, p.ldd, T, p.K);
      FG_TRY(launched(what));
    }
    return FG_OK;
  }
};

template <class Fmt>
fg_status launch_layer(const ExpertParams& p, void* stream, const char* what) {
  const char* forced = getenv("FG_DECODE_PLAN");
  const LayerPlan plan = plan_layer(Fmt::FP8, p.T, p.k, p.E, p.F, p.K, forced ? forced : "");
  const LayerLaunch l{p, plan, ceil_div(p.T, kLayerTokens), (float*)((uint8_t*)p.H + hidden_bytes(p.T, p.k, p.F)), stream, what};
  if (p.F > 0) {
    fg_status st = FG_OK;
    switch (plan.up) {
      case kUpSplit2:
        if constexpr (!Fmt::FP8) st = l.up<UpTile<Fmt, 1, 4, 2, 2>>();
        break;
      case kUpSplit4: st = l.up<UpTile<Fmt, 1, 4, 2, 4>>(); break;
      case kUpSplit16: st = l.up<UpTile<Fmt, 1, 4, 2, 16>>(); break;
      case kUpWide: st = l.up<WideUp<Fmt, 1, 4, 2, Fmt::FP8 ? 32 : 16>>(); break;
      case kUpWideDeep:
        if constexpr (Fmt::FP8) st = l.up<WideUp<Fmt, 1, 4, 3, 32>>();
        break;
      case kUpWide8:
        // scales of groups of 32 leave no room for 32 tokens
        if constexpr (!Fmt::FP8) st = l.up<WideUp<Fmt, 1, 8, 2, Fmt::GPC == 4 ? 16 : 32>>();
        break;
      default: break;
    }
    FG_TRY(st);
  }
  switch (plan.down) {
    case kDownSplit1: return l.down<DownTile<Fmt, kDownSplit1>>();
    case kDownSplit1Two: return l.down<DownTile<Fmt, kDownSplit1Two>>();
    case kDownSplit4: return l.down<DownTile<Fmt, kDownSplit4>>();
    case kDownSplit4Two:
      if constexpr (!Fmt::FP8) return l.down<DownTile<Fmt, kDownSplit4Two>>();
      break;
    case kDownWide16: return l.down_wide<WideDown<Fmt, kDownWide16>>();
    case kDownWide16Deep:
      if constexpr (Fmt::FP8) return l.down_wide<WideDown<Fmt, kDownWide16Deep>>();
      break;
    case kDownWide32: return l.down_wide<WideDown<Fmt, kDownWide32>>();
    default: break;
  }
  return FG_OK;
}

struct LaunchLayer {
  const ExpertParams& p;
  void* stream;
  template <class Fmt>
  fg_status run() const {
    return launch_layer<Fmt>(p, stream, "moe_ffn_int4");
  }
};

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
  if (T < 0 || k <= 0 || F < 0 || F % 16 || T > kMaxTokens || k > kMaxChoices || F > kMaxWidth) return -1;
  return layer_bytes(T, k, F);
}

fg_status moe_ffn_fp8(const uint16_t* X, int64_t ldx, const uint8_t* W1, const float* s1, const uint8_t* W2,
                      const float* s2, const int32_t* ids, const float* weights, uint16_t* D, int64_t ldd, int T, int k,
                      int E, int F, int K, int activation, void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  ExpertParams p{};
  p.X = X; p.ldx = ldx; p.W1 = W1; p.s1 = s1; p.W2 = W2; p.s2 = s2; p.ids = ids; p.w = weights; p.D = D; p.ldd = ldd;
  p.H = (float*)workspace;
  p.T = T; p.k = k; p.E = E; p.F = F; p.K = K; p.act = activation;
  bool empty;
  FG_TRY(check_layer(p, 16, workspace, workspace_bytes, 4, &empty));
  if (empty) return FG_OK;
  p.row1 = K; p.row2 = F;
  p.groups1 = (K + 127) / 128; p.groups2 = (F + 127) / 128;
  return launch_layer<Fp8Block>(p, stream, "moe_ffn_fp8");
}

fg_status moe_ffn_int4(const uint16_t* X, int64_t ldx, const uint8_t* W1, const uint16_t* s1, const uint8_t* z1,
                       const uint8_t* W2, const uint16_t* s2, const uint8_t* z2, const int32_t* ids, const float* weights,
                       uint16_t* D, int64_t ldd, int T, int k, int E, int F, int K, int group, int activation,
                       void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  ExpertParams p{};
  p.X = X; p.ldx = ldx; p.W1 = W1; p.s1 = s1; p.z1 = z1; p.W2 = W2; p.s2 = s2; p.z2 = z2; p.ids = ids; p.w = weights;
  p.D = D; p.ldd = ldd;
  p.H = (float*)workspace;
  p.T = T; p.k = k; p.E = E; p.F = F; p.K = K; p.act = activation; p.group = group;
  FG_TRY(check_group(group));
  if ((z1 != nullptr) != (z2 != nullptr)) return set_error(FG_EINVAL, "z1 and z2: one of them is NULL");
  bool empty;
  FG_TRY(check_layer(p, 32, workspace, workspace_bytes, 2, &empty));
  if (empty) return FG_OK;
  p.row1 = int4_row_bytes(K); p.row2 = int4_row_bytes(F);
  p.groups1 = int4_groups(K, group); p.groups2 = int4_groups(F, group);
  // the zero points of both matrices, or of neither: a missing one is refused above
  return with_int4_format(group, z1 != nullptr, LaunchLayer{p, stream});
}

}  // extern "C"
