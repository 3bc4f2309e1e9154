// csa_latent_rows.cuh — rows of values as a warp holds them, and as records of the latent cache: what the
// cache's writer and the rotating writer share.
#pragma once

#include <cuda_fp4.h>

#include "csa_latent_common.cuh"

namespace csa_latent {
namespace {

constexpr int kCopyThreads = 256;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Two e2m1 codes, a in the low nibble: nearest, ties to the even mantissa, saturating at 6.
__device__ __forceinline__ uint32_t e2m1_pair(float a, float b) {
  return __nv_cvt_float2_to_fp4x2(make_float2(a, b), __NV_E2M1, cudaRoundNearest);
}

template <bool kBf16In>
struct RowIn {
  float v[16], r[2];
  __device__ __forceinline__ void load(const void* row, int lane, int rope) {
    if constexpr (kBf16In) {
      const uint4* p = reinterpret_cast<const uint4*>(row) + 2 * lane;
      const uint4 a = p[0], b = p[1];
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[2 * k] = bf16_lo(w[k]);
        v[2 * k + 1] = bf16_hi(w[k]);
      }
      const uint32_t t = rope ? reinterpret_cast<const uint32_t*>(row)[kDim / 2 + lane] : 0u;
      r[0] = bf16_lo(t);
      r[1] = bf16_hi(t);
    } else {
      const float4* p = reinterpret_cast<const float4*>(row) + 4 * lane;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 a = p[k];
        v[4 * k] = a.x;
        v[4 * k + 1] = a.y;
        v[4 * k + 2] = a.z;
        v[4 * k + 3] = a.w;
      }
      const float2 t = rope ? reinterpret_cast<const float2*>(row)[kDim / 2 + lane] : make_float2(0.f, 0.f);
      r[0] = t.x;
      r[1] = t.y;
    }
  }
};

__device__ __forceinline__ uint32_t nonfinite_bf16x2(uint32_t w) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// A lane's 16 latent values as its part of a record: bf16 words, or e2m1 codes and the block's exponent.
template <bool kFp4>
struct Coded {
  uint32_t w[kFp4 ? 2 : 8];
  int e;
  bool bad;  // a value that is not finite (after rounding to bf16, where bf16 is stored)
};

// floor(log2 amax) - 2 of a magnitude's bits, held at -127: a subnormal amax (below 2^-126) lands there too.
__device__ __forceinline__ int block_exponent(uint32_t amax) { return max(static_cast<int>(amax >> 23) - 129, -127); }

// 2^-e is 2^-125 .. 2^127, a normal number; x 2^-e is exact where it can reach a nonzero code.
__device__ __forceinline__ float block_up(int e) { return __uint_as_float(static_cast<uint32_t>(min(-e, 127) + 127) << 23); }

template <bool kFp4>
__device__ __forceinline__ Coded<kFp4> encode(const float (&v)[16]) {
  Coded<kFp4> c;
  if constexpr (!kFp4) {
    uint32_t bad = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      c.w[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
      bad |= nonfinite_bf16x2(c.w[k]);
    }
    c.bad = bad != 0;
    c.e = 0;
  } else {
    uint32_t amax = 0;  // magnitude bits order like the magnitudes
#pragma unroll
    for (int k = 0; k < 16; ++k) amax = max(amax, __float_as_uint(v[k]) & 0x7FFFFFFFu);
    c.bad = amax >= 0x7F800000u;
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    c.e = block_exponent(amax);
    const float up = block_up(c.e);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      c.w[h] = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) c.w[h] |= e2m1_pair(v[8 * h + 2 * k] * up, v[8 * h + 2 * k + 1] * up) << (8 * k);
    }
  }
  return c;
}

// A whole warp's record to its slot (which is in the cache).
template <bool kFp4>
__device__ __forceinline__ void put_record(const csa_latent_cache& cache, int64_t slot, const Coded<kFp4>& c, uint32_t rope_word, int lane) {
  const int rope = cache.rope_dim, rec_bytes = record_bytes(kFp4, rope);
  uint8_t* rec = cache.pages + (slot / kPageRecs) * cache.page_stride_bytes + (slot % kPageRecs) * rec_bytes;
  if constexpr (!kFp4) {
    uint4* p = reinterpret_cast<uint4*>(rec) + 2 * lane;
    p[0] = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
    p[1] = make_uint4(c.w[4], c.w[5], c.w[6], c.w[7]);
  } else {
    reinterpret_cast<uint2*>(rec)[lane] = make_uint2(c.w[0], c.w[1]);
    // four blocks' scale bytes gathered into one word by lanes 0, 8, 16, 24
    uint32_t sb = static_cast<uint32_t>(c.e + 127) << (8 * ((lane >> 1) & 3));
    sb |= __shfl_xor_sync(0xFFFFFFFFu, sb, 2);
    sb |= __shfl_xor_sync(0xFFFFFFFFu, sb, 4);
    if ((lane & 7) == 0) reinterpret_cast<uint32_t*>(rec + kCodeBytes)[lane >> 3] = sb;
  }
  if (rope) reinterpret_cast<uint32_t*>(rec + rec_bytes - 2 * rope)[lane] = rope_word;
}

// At most one full wave of blocks, each taking `per_block` rows at a time. `kept` (or null): the kernel's resident
// blocks an SM on each device, asked for once.
template <typename K>
csa_status wave_grid(K kernel, int threads, size_t smem, Kept* kept, int64_t rows, int64_t per_block, unsigned* grid) {
  int sms = 0, dev = 0;
  if (sm_count(&sms, &dev) != CSA_OK) return CSA_ERR_CUDA;
  int per_sm = kept ? kept->get(dev) : 0;
  if (per_sm == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess || per_sm < 1)
      return CSA_ERR_CUDA;
    if (kept) kept->set(dev, per_sm);
  }
  const int64_t want = (rows + per_block - 1) / per_block, cap = static_cast<int64_t>(sms) * per_sm;
  *grid = static_cast<unsigned>(want < 1 ? 1 : (want < cap ? want : cap));
  return CSA_OK;
}

}  // namespace
}  // namespace csa_latent
