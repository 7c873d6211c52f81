// host_decode_lds_driver.cpp -- what the few-token expert layers set on their
// kernels (tests/test_host_decode_plans.py).  The runtime's calls for the device and
// for a kernel's attributes are replaced by ones that keep a record; no GPU is
// needed, since a launch fails behind them.
//
// A kernel's limit of dynamic LDS is the process's, not the call's: where each call
// set its own need, a call of few tokens would lower it under a call of many on
// another thread.  Every kernel has to get one value, the most, once on a device.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <mutex>
#include <thread>
#include <vector>

#include <hip/hip_runtime.h>

#include "fp8gemm.h"

static std::mutex g_lock;
static thread_local int g_device = 0;
static std::map<std::pair<const void*, int>, std::vector<int>> g_set;  // by kernel and device

extern "C" hipError_t hipGetDevice(int* device) {
  *device = g_device;
  return hipSuccess;
}
extern "C" hipError_t hipFuncSetAttribute(const void* kernel, hipFuncAttribute, int value) {
  std::lock_guard<std::mutex> hold(g_lock);
  g_set[{kernel, g_device}].push_back(value);
  return hipSuccess;
}

static void calls(int device, unsigned seed) {
  g_device = device;
  uint16_t* X = reinterpret_cast<uint16_t*>(0x10000);
  float* S = reinterpret_cast<float*>(0x10000);
  int32_t* I = reinterpret_cast<int32_t*>(0x10000);
  void* WS = reinterpret_cast<void*>(0x10000);
  const int tokens[] = {64, 1, 40, 2, 17, 8, 64, 5, 30, 1};
  for (int i = 0; i < 10; ++i)
    for (int E : {1, 16, 200}) {
      const int T = tokens[(i + seed) % 10], k = 2, K = 4096;
      // no hidden units: the second half's kernel is the first, and needs no more than these addresses
      const int64_t need = fg_moe_ffn_workspace_bytes(T, k, 0);
      moe_ffn_fp8(X, K, nullptr, nullptr, nullptr, nullptr, I, S, X, K, T, k, E, 0, K, FG_ACT_SILU, WS, need, nullptr);
      moe_ffn_int4(X, K, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, I, S, X, K, T, k, E, 0, K, 128, FG_ACT_SILU, WS, need,
                   nullptr);
    }
}

int main() {
  const char* plans[] = {"", "down-split1", "down-split4", "down-wide16", "down-wide32"};
  for (const char* plan : plans) {
    setenv("FG_DECODE_PLAN", plan, 1);
    calls(0, 0);
    calls(1, 3);
  }
  std::vector<std::thread> threads;
  for (int t = 0; t < 4; ++t) threads.emplace_back(calls, 2, 3 * t);
  for (std::thread& t : threads) t.join();
  int wrong = 0;
  for (const auto& s : g_set) {
    for (int v : s.second) wrong += v != s.second[0] || v < 64 * 1024 || v > 160 * 1024;
    if (s.first.second < 2) wrong += s.second.size() != 1;  // threads may set the same value side by side
  }
  if (g_set.empty() || wrong) return std::fprintf(stderr, "%d wrong of %zu kernels\n", wrong, g_set.size()), 1;
  std::printf("host lds ok: %zu\n", g_set.size());
  return 0;
}
