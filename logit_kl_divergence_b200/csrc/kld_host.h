// kld_host.h -- what the translation units of the C ABI share: the mapping of
// CUDA errors to status codes and the device guard.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "kld_stats.h"

namespace kld {

// Notes the error's text for kld_last_cuda_error and returns its status.
kld_status_t cuda_fail(cudaError_t e, const char* what);

#define KLD_CUDA(call)                                       \
  do {                                                       \
    cudaError_t _e = (call);                                 \
    if (_e != cudaSuccess) return kld::cuda_fail(_e, #call); \
  } while (0)

// Whether two ranges of bytes have none in common (a null or empty one has no bytes).
inline bool apart(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return !a || !b || a_bytes <= 0 || b_bytes <= 0 || x + static_cast<uintptr_t>(a_bytes) <= y ||
         y + static_cast<uintptr_t>(b_bytes) <= x;
}

// KLD_OK when `device` exists and is of compute capability 10.0; *sms: its
// SM count.
kld_status_t check_device(int device, int* sms);

// Makes the handle's device current for the duration of a call.
class DeviceGuard {
 public:
  explicit DeviceGuard(int dev) {
    ok_ = cudaGetDevice(&prev_) == cudaSuccess;
    if (ok_ && prev_ != dev) ok_ = cudaSetDevice(dev) == cudaSuccess;
    switched_ = ok_ && prev_ != dev;
  }
  ~DeviceGuard() {
    if (switched_) cudaSetDevice(prev_);
  }
  bool ok() const { return ok_; }

 private:
  int prev_ = 0;
  bool ok_ = false;
  bool switched_ = false;
};

}  // namespace kld
