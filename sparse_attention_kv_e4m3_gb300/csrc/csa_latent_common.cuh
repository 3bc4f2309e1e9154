// csa_latent_common.cuh — what the latent-cache operators share: record layout,
// page lookup, and small host checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "csa_latent.h"

namespace csa_latent {

constexpr int kDim = CSA_LATENT_DIM;   // latent values of a record
constexpr int kPageRecs = CSA_PAGE_RECORDS;
constexpr int kCodeBytes = kDim / 2;   // MXFP4: code bytes, then kDim / 32 scale bytes, then rope
constexpr int kScaleBytes = kDim / 32;

__host__ __device__ constexpr int record_bytes(bool fp4, int rope) {
  return fp4 ? kCodeBytes + kScaleBytes + 2 * rope : 2 * (kDim + rope);
}

// 2^(b - 127) for a UE8M0 byte: a normal binary32 power of two for 1 .. 254, the
// subnormal 2^-127 for 0, NaN for 255.
__device__ __forceinline__ float ue8m0(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : (b == 255 ? 0x7FC00000u : b << 23));
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A softmax scale: the kernels multiply it by log2 e, which has to stay finite.
inline bool good_scale(float scale) { return scale > 0.f && scale < 0x1p127f; }

inline csa_status check_cache(const csa_latent_cache& c) {
  if (!c.pages || c.num_pages < 1 || c.num_pages > INT32_MAX) return CSA_ERR_INVALID_ARG;
  const int64_t rec = csa_latent_record_bytes(c.record_format, c.rope_dim);
  if (rec == 0) return CSA_ERR_UNSUPPORTED;
  if (c.page_stride_bytes < kPageRecs * rec) return CSA_ERR_INVALID_ARG;
  if (c.page_stride_bytes % 16 != 0 || !aligned(c.pages, 16)) return CSA_ERR_ALIGNMENT;
  return CSA_OK;
}

// The current device and its SM count (which is asked for once a device and kept, like a kernel's occupancy:
// each query costs about a microsecond of a small call).
constexpr int kMaxDevices = 64;

// What the host code keeps for each device, 0 until it is known. Two threads may both find it out, with the same
// answer; it stands alone, so no order with other memory is needed.
struct Kept {
  std::atomic<int> of[kMaxDevices];
  int get(int dev) const { return of[dev].load(std::memory_order_relaxed); }
  void set(int dev, int v) { of[dev].store(v, std::memory_order_relaxed); }
};

inline csa_status sm_count(int* sms, int* device = nullptr) {
  static Kept kept;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return CSA_ERR_CUDA;
  int n = kept.get(dev);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return CSA_ERR_CUDA;
    kept.set(dev, n);
  }
  *sms = n;
  if (device) *device = dev;
  return CSA_OK;
}

}  // namespace csa_latent
