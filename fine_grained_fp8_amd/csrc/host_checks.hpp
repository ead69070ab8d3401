// Argument checks shared by the files that implement the C ABI: the device
// query, alignment, byte ranges and their overlap, launch status.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "fp8bs.h"

namespace {

constexpr int kMaxDevices = 64;
// 0 = unknown, 1 = gfx950, 2 = other
std::atomic<int> g_device_kind[kMaxDevices];

[[maybe_unused]] fp8_status check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
    (void)hipGetLastError();
    return FP8_ERR_DEVICE;
  }
  if (dev >= kMaxDevices) return FP8_ERR_DEVICE;
  int kind = g_device_kind[dev].load(std::memory_order_relaxed);
  if (kind == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
      (void)hipGetLastError();
      return FP8_ERR_DEVICE;
    }
    kind = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    g_device_kind[dev].store(kind, std::memory_order_relaxed);
  }
  return kind == 1 ? FP8_OK : FP8_ERR_DEVICE;
}

[[maybe_unused]] bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
[[maybe_unused]] bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// [lo, hi) byte range of a row-major matrix with `rows` rows of `row_bytes`
// at stride `ld_bytes`.
struct Range {
  uintptr_t lo, hi;
};
[[maybe_unused]] Range span(const void* p, int64_t rows, int64_t row_bytes, int64_t ld_bytes) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  if (rows <= 0 || row_bytes <= 0) return {b, b};
  return {b, b + static_cast<uintptr_t>((rows - 1) * ld_bytes + row_bytes)};
}
[[maybe_unused]] bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

[[maybe_unused]] fp8_status launched(hipError_t e) {
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return FP8_ERR_LAUNCH;
  }
  return FP8_OK;
}

}  // namespace
