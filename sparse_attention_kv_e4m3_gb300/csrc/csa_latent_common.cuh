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

// Four e2m1 codes (the low 16 bits of `sel`) as bf16 values times `s2`. The magnitudes
// 0 1/2 1 3/2 2 3 4 6 are looked up as the two bytes of their bf16 by byte permutes; a permute
// in its sign-replicating mode spreads the codes' sign bits. The product with a power of two is
// exact.
__device__ __forceinline__ void mxfp4_four(uint32_t sel, __nv_bfloat162 s2, uint32_t* lo, uint32_t* hi) {
  const uint32_t mag = sel & 0x7777u;
  const uint32_t h = __byte_perm(0x3F3F3F00u, 0x40404040u, mag), l = __byte_perm(0xC0800000u, 0xC0804000u, mag);
  // bytes 0x80 where the sign bit is clear, 0xFF where it is set: bit 6 is the sign
  uint32_t sg;
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(sg) : "r"(0x80808080u), "r"(sel));
  const uint32_t hs = h | ((sg << 1) & 0x80808080u);
  uint32_t a = __byte_perm(l, hs, 0x5140), b = __byte_perm(l, hs, 0x7362);
  const __nv_bfloat162 x = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), s2);
  const __nv_bfloat162 y = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&b), s2);
  *lo = *reinterpret_cast<const uint32_t*>(&x);
  *hi = *reinterpret_cast<const uint32_t*>(&y);
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A softmax scale: the kernels multiply it by log2 e, which has to stay finite.
inline bool good_scale(float scale) { return scale > 0.f && scale < 0x1p127f; }

// The factor c (the scale, times log2 e) of a row's exponents S c - m c, for its reference m. The rounding of m c that is left in them is 2^-25 of it:
// above 2^30 it could be more than an exponent holds. Scores that differ at all differ by 2^-24 of theirs, though, so that weights there are 1
// or 0 as well with the power of two below c, whose product with m is exact.
__device__ __forceinline__ float exponent_factor(float mc, float c) {
  return fabsf(mc) > 0x1p30f ? __uint_as_float(__float_as_uint(c) & 0x7F800000u) : c;
}

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
