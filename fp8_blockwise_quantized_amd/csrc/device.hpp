// The current device as the C-ABI entry points see it: architecture check and compute-unit count.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>

#include "validate.hpp"

namespace fp8bq {

constexpr int kMaxDevices = 64;
// Per-device cache: 0 = unknown, 1 = gfx950, 2 = other architecture.  Benign races (all writers
// store the same value).
inline std::atomic<int> g_dev_state[kMaxDevices];
inline std::atomic<int> g_dev_cus[kMaxDevices];

// Returns kOk if the current device is a gfx950; fills *cus with its compute-unit count and *index
// with its index (each if not null).
inline int current_device(int* cus, int* index = nullptr) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
    (void)hipGetLastError();
    return kErrDevice;
  }
  int state = g_dev_state[dev].load(std::memory_order_relaxed);
  if (state == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
      (void)hipGetLastError();
      return kErrDevice;
    }
    state = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
    g_dev_cus[dev].store(prop.multiProcessorCount, std::memory_order_relaxed);
    g_dev_state[dev].store(state, std::memory_order_relaxed);
  }
  if (cus) *cus = g_dev_cus[dev].load(std::memory_order_relaxed);
  if (index) *index = dev;
  return state == 1 ? kOk : kErrDevice;
}

inline int launched(hipError_t e) { return e == hipSuccess ? kOk : kErrLaunch; }

}  // namespace fp8bq
