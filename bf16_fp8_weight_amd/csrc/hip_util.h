// hip_util.h -- host-side helpers over the HIP runtime shared by the entry
// points that touch a GPU: error texts, the scoped current device, and the
// check that a range lies in one allocation of the expected kind.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>
#include <string>

#include "wt.h"

namespace wt {

inline std::string hip_msg(const char *what, hipError_t e) {
  return std::string(what) + ": " + hipGetErrorName(e) + " (" + hipGetErrorString(e) + ")";
}

// Makes `dev` current for the scope and restores the caller's device on
// exit; a no-op (one hipGetDevice) when `dev` is current already.
struct DeviceGuard {
  int prev = -1;
  bool switched = false;
  explicit DeviceGuard(int dev) {
    if (hipGetDevice(&prev) != hipSuccess) {
      (void)hipGetLastError();
      prev = -1;
    }
    if (dev >= 0 && dev != prev && hipSetDevice(dev) == hipSuccess) switched = prev >= 0;
  }
  ~DeviceGuard() {
    if (switched) (void)hipSetDevice(prev);
  }
};

// Checks that [p, p + bytes) lies in one allocation of the expected kind.
inline wt_status check_memory(const void *p, uint64_t bytes, int32_t kind, int device, const std::string &what,
                              std::string *err) {
  if (bytes == 0) return WT_OK;
  hipPointerAttribute_t a;
  std::memset(&a, 0, sizeof a);
  hipError_t e = hipPointerGetAttributes(&a, p);
  if (e != hipSuccess) {
    (void)hipGetLastError();
    *err = what + ": pointer is not HIP device or pinned host memory";
    return WT_E_INVAL;
  }
  if (kind == WT_MEM_DEVICE) {
    if (a.type != hipMemoryTypeDevice) {
      *err = what + ": expected device memory";
      return WT_E_INVAL;
    }
    if (a.device != device) {
      *err = what + ": device memory of another GPU";
      return WT_E_INVAL;
    }
  } else {
    if (a.type != hipMemoryTypeHost) {
      *err = what + ": expected pinned host memory";
      return WT_E_INVAL;
    }
  }
  // extent: the allocation that holds p must also hold p + bytes - 1 (device
  // allocations and pinned host allocations alike are tracked by the runtime)
  hipDeviceptr_t base = nullptr;
  size_t size = 0;
  if (hipMemGetAddressRange(&base, &size, (hipDeviceptr_t)p) == hipSuccess && base) {
    const uint64_t lo = (uint64_t)(uintptr_t)base, hi = lo + size;
    if ((uint64_t)(uintptr_t)p < lo || (uint64_t)(uintptr_t)p + bytes > hi) {
      *err = what + ": range runs past the end of its allocation";
      return WT_E_RANGE;
    }
  } else {
    (void)hipGetLastError();
  }
  return WT_OK;
}

}  // namespace wt
