// Host-side checks shared by the C-ABI sources. Library-internal.
#pragma once
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/ssd.h"

namespace ssd {

constexpr int64_t kMaxIndex = (int64_t(1) << 31) - 1;

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void* p, int64_t bytes) {
  uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, a + static_cast<uintptr_t>(bytes)};
}

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline ssd_status device_ready() {
  static std::atomic<bool> seen{false};  // devices do not go away once a call has found one
  if (seen.load(std::memory_order_relaxed)) return SSD_OK;
  int n = 0;
  if (hipGetDeviceCount(&n) != hipSuccess || n <= 0) return SSD_ERR_NO_DEVICE;
  seen.store(true, std::memory_order_relaxed);
  return SSD_OK;
}

inline ssd_status from_hip(hipError_t e) {
  if (e == hipSuccess) return SSD_OK;
  if (e == hipErrorOutOfMemory) return SSD_ERR_OUT_OF_MEMORY;
  return SSD_ERR_HIP;
}

}  // namespace ssd
