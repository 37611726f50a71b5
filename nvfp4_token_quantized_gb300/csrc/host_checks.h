// host_checks.h - argument checks that the entry points of the operators
// around the layer share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/moe_nvfp4.h"

namespace moe {

constexpr int64_t MAX_ROWS = 0x7fffffff;  // one grid dimension

// MOE_OK if the current device is one the kernels were built for; asked of
// the runtime once per device.
inline moe_status check_device() {
  constexpr int MAX_DEVICES = 64;
  static std::atomic<signed char> known[MAX_DEVICES];  // 0: not asked, 1: sm_103, -1: another
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) {
    cudaGetLastError();
    return MOE_ERR_UNSUPPORTED;
  }
  signed char k = known[dev].load(std::memory_order_relaxed);
  if (k == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
      cudaGetLastError();
      return MOE_ERR_CUDA;
    }
    k = major == 10 && minor == 3 ? 1 : -1;
    known[dev].store(k, std::memory_order_relaxed);
  }
  return k == 1 ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

inline int dtype_bytes(int dtype) {
  switch (dtype) {
    case MOE_DTYPE_BF16:
    case MOE_DTYPE_F16: return 2;
    case MOE_DTYPE_F32: return 4;
  }
  return 0;
}

inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline moe_status launched(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ERR_CUDA;
}

// Rows of `width` bytes, `pitch` bytes apart.
struct Rows {
  const void* p;
  int64_t rows, width, pitch;
};

inline bool overlap(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0) return false;
  const intptr_t a0 = (intptr_t)a.p, b0 = (intptr_t)b.p;
  const int64_t na = (a.rows - 1) * a.pitch + a.width, nb = (b.rows - 1) * b.pitch + b.width;
  if (a0 + na <= b0 || b0 + nb <= a0) return false;
  if (a.rows == 1 || b.rows == 1 || a.pitch != b.pitch) return true;
  // columns of one wider array may lie between each other's
  const int64_t P = a.pitch, d = ((b0 - a0) % P + P) % P;
  return !(d >= a.width && d + b.width <= P);
}

inline bool same_rows(const Rows& a, const Rows& b) {
  return a.p == b.p && a.width == b.width && (a.pitch == b.pitch || a.rows == 1);
}

}  // namespace moe
