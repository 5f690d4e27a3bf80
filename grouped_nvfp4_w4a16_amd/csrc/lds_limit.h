// The dynamic LDS limit of kernels that take more than 64 KB.
#pragma once

#include <hip/hip_runtime.h>

#include <mutex>

namespace moe {

// Raises kKern's limit to `bytes`, once per device. False if the device refuses it.
template <auto kKern>
bool allow_lds(int bytes) {
  constexpr int kMaxDevices = 64;
  static std::mutex mu;
  static bool done[kMaxDevices] = {};
  int device = 0;
  if (hipGetDevice(&device) != hipSuccess || device < 0) return false;
  std::lock_guard<std::mutex> lock(mu);
  if (device < kMaxDevices && done[device]) return true;
  if (hipFuncSetAttribute(reinterpret_cast<const void *>(kKern),
                          hipFuncAttributeMaxDynamicSharedMemorySize, bytes) != hipSuccess) {
    (void)hipGetLastError();  // reported here, not by a later call
    return false;
  }
  if (device < kMaxDevices) done[device] = true;
  return true;
}

}  // namespace moe
