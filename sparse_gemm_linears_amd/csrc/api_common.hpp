// Checks and status mapping shared by the C entry points (api.hip,
// api_layer.hip): size limits, pointer alignment and aliasing, the device
// check, and the status of a launch.
#pragma once

#include <atomic>
#include <cstring>

#include "../../include/fp8lin.h"
#include "launch.hpp"

namespace fp8lin {

constexpr int64_t kMaxDim = int64_t(1) << 24;
constexpr int kMaxDeviceIds = 64;
inline std::atomic<int> g_arch_ok[kMaxDeviceIds];  // 0 = unknown, 1 = gfx950, 2 = other

struct Range {
  const void *p;
  int64_t bytes;
};

inline bool overlaps(const Range &a, const Range &b) {
  if (a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a0 < b0 + (uintptr_t)b.bytes && b0 < a0 + (uintptr_t)a.bytes;
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// Every output range against every input range and every other output range.
inline bool any_alias(const Range *outs, int n_out, const Range *ins, int n_in) {
  for (int i = 0; i < n_out; i++) {
    for (int j = 0; j < n_in; j++)
      if (overlaps(outs[i], ins[j])) return true;
    for (int j = i + 1; j < n_out; j++)
      if (overlaps(outs[i], outs[j])) return true;
  }
  return false;
}

inline fp8l_status check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
    (void)hipGetLastError();
    return FP8L_ERR_DEVICE;
  }
  if (dev < kMaxDeviceIds) {
    const int known = g_arch_ok[dev].load(std::memory_order_relaxed);
    if (known) return known == 1 ? FP8L_OK : FP8L_ERR_DEVICE;
  }
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
    (void)hipGetLastError();
    return FP8L_ERR_DEVICE;
  }
  const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  if (dev < kMaxDeviceIds) g_arch_ok[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
  return ok ? FP8L_OK : FP8L_ERR_DEVICE;
}

constexpr int64_t kMaxElems = int64_t(1) << 36;  // keeps every grid and index in range

inline bool bad_mk(int64_t M, int64_t K) {
  return M < 0 || K <= 0 || K % 128 != 0 || M > kMaxDim || K > kMaxDim || M * K > kMaxElems;
}
inline bool bad_nk(int64_t N, int64_t K) {
  return N <= 0 || K <= 0 || N % 128 != 0 || K % 128 != 0 || N > kMaxDim || K > kMaxDim || N * K > kMaxElems;
}
inline bool bad_mn(int64_t M, int64_t N) { return M * N > kMaxElems; }

inline fp8l_status launched(hipError_t e) {
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return e == hipErrorOutOfMemory ? FP8L_ERR_MEMORY : FP8L_ERR_LAUNCH;
  }
  return FP8L_OK;
}

// Status of a call that held scratch memory: the launches' status first, then
// that of handing the scratch back (a one-off allocation's stream-ordered free).
inline fp8l_status finished(hipError_t e, CallScratch &sc) {
  const hipError_t f = sc.release();
  return launched(e != hipSuccess ? e : f);
}

}  // namespace fp8lin
