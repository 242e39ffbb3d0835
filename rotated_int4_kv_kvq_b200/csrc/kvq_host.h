// kvq_host.h -- argument checks and device facts shared by the C-ABI front
// ends (kvq_api.cu, kvq_paged_api.cu).  Not part of the public API.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "kvq.h"

namespace kvq {
namespace host {

constexpr int kMaxDevices = 64;

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline kvq_status check_shape(int32_t d, int32_t group, kvq_rot rot) {
  if (rot != KVQ_ROT_SRFT && rot != KVQ_ROT_SRHT) return KVQ_ERR_BAD_ROT;
  if (d != 64 && d != 128 && d != 256) return KVQ_ERR_BAD_DIM;
  if ((group != 32 && group != 64 && group != 128 && group != 256) || group > d)
    return KVQ_ERR_BAD_GROUP;
  return KVQ_OK;
}

// Per-device facts, looked up once: SM count and whether the device is
// compute capability 10.0 (the only one this sm_100a build runs on).
struct DeviceInfo {
  int sm_count = 0;
  bool ok = false;
};

inline kvq_status device_info(DeviceInfo* out) {
  static DeviceInfo info[kMaxDevices];
  static bool done[kMaxDevices];
  static std::mutex mu;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return KVQ_ERR_CUDA;
  }
  std::lock_guard<std::mutex> g(mu);
  if (!done[dev]) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return KVQ_ERR_CUDA;
    }
    info[dev].sm_count = sms;
    info[dev].ok = (major == 10 && minor == 0);
    done[dev] = true;
  }
  *out = info[dev];
  return info[dev].ok ? KVQ_OK : KVQ_ERR_UNSUPPORTED_DEVICE;
}

inline kvq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA; }

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

}  // namespace host
}  // namespace kvq
