// csa_latent_maps.h — tensor maps of the latent attention kernels' operands (host).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace csa_latent {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult got;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &got) != cudaSuccess ||
        got != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// bf16 in boxes of 64 values wide, 128-byte swizzle; dims and boxes innermost first, strides in bytes of dims 1 ...
inline bool encode_map(CUtensorMap* map, const void* base, uint32_t rank, const cuuint64_t* dims, const cuuint64_t* strides,
                       const cuuint32_t* boxes) {
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  return encode_tiled() &&
         encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, boxes, steps,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [rows][heads][width] (strides in elements), or [rows][width] where heads is 0, in boxes of 64 values, `box_heads`
// heads and `box_rows` rows.
inline bool encode_bf16(CUtensorMap* map, const void* base, int64_t width, int64_t heads, int64_t rows, int64_t head_stride,
                        int64_t row_stride, uint32_t box_heads, uint32_t box_rows) {
  const bool flat = heads == 0;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(flat ? rows : heads),
                              static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(2 * (flat ? row_stride : head_stride)),
                                 static_cast<cuuint64_t>(2 * row_stride)};
  const cuuint32_t boxes[3] = {64, flat ? box_rows : box_heads, box_rows};
  return encode_map(map, base, flat ? 2 : 3, dims, strides, boxes);
}

}  // namespace csa_latent
