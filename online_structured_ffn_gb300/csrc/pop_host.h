// Host helpers of the C-ABI files of the 8-bit and trainable operators: messages, device checks, allocations.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

#include "pop_ffn.h"

namespace pop {

inline pop_status report(std::string& msg, pop_status s, const char* call, const char* why) noexcept {
  try {
    msg = std::string(call) + ": " + why;
  } catch (...) {
  }
  return s;
}

inline pop_status report_cuda(std::string& msg, cudaError_t e, const char* call) noexcept {
  if (e == cudaSuccess) return POP_OK;
  cudaGetLastError();  // it is reported here: a later call that asks the runtime for the last error is not to find it
  return report(msg, e == cudaErrorMemoryAllocation ? POP_ERR_OOM : POP_ERR_CUDA, call, cudaGetErrorString(e));
}

inline bool off(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

template <class T>
cudaError_t dalloc(T** p, size_t n) {
  return cudaMalloc(reinterpret_cast<void**>(p), (n ? n : 1) * sizeof(T));
}

inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 1;
  return n > 0 ? n : 1;
}

inline int current_device() {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}

// Makes a device the current one for as long as it lives.
struct OnDevice {
  int was;
  explicit OnDevice(int device) : was(current_device()) {
    if (was != device) cudaSetDevice(device);
    else was = -1;
  }
  ~OnDevice() {
    if (was >= 0) cudaSetDevice(was);
  }
};

}  // namespace pop
