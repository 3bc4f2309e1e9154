// csa_latent_attend.cu — latent attention, absorbed form (include/csa_latent.h).
#include <cuda_fp4.h>

#include "csa_latent_common.cuh"

namespace csa_latent {
namespace {

constexpr int kThreads = 128;

// What a query row sees: its request's page table row and its length.
struct RowView {
  const int32_t* table;  // null: an empty row
  int32_t len;
};

__device__ __forceinline__ RowView row_view(const csa_latent_attend_args& A, int b, int32_t* flags) {
  const int32_t req = A.row_req ? A.row_req[b] : b;
  if (req < 0 || req >= A.num_req) {
    *flags |= CSA_DEV_BAD_REQUEST;
    return {nullptr, 0};
  }
  const int32_t n = A.row_len[b], cap = kPageRecs * A.pt_stride, len = min(max(n, 0), cap);
  if (len != n) *flags |= CSA_DEV_LEN_OOB;
  return {A.page_table + static_cast<int64_t>(req) * A.pt_stride, len};
}

// The record of the row's j-th entry (of the listed positions or of the history),
// or null where nothing is visible.
__device__ __forceinline__ const uint8_t* record_of(const csa_latent_attend_args& A, const RowView& R, int b, int j,
                                                    int rec_bytes, int32_t* flags) {
  int32_t pos = j;
  if (A.idx) {
    pos = A.idx[b * A.idx_stride + j];
    if (pos == -1) return nullptr;
    if (pos < 0 || pos >= R.len) {
      *flags |= CSA_DEV_LEN_OOB;
      return nullptr;
    }
  }
  const int32_t page = R.table[pos / kPageRecs];
  if (page < 0 || page >= A.cache.num_pages) {
    *flags |= CSA_DEV_PAGE_OOB;
    return nullptr;
  }
  return A.cache.pages + page * A.cache.page_stride_bytes + static_cast<int64_t>(pos % kPageRecs) * rec_bytes;
}

// Lane l's 16 latent values (16 l ..) and 2 rope values (2 l, 2 l + 1) of a record.
template <bool kFp4>
__device__ __forceinline__ void lane_values(const uint8_t* rec, int lane, int rope, float (&v)[18]) {
  if constexpr (kFp4) {
    const uint2 c = reinterpret_cast<const uint2*>(rec)[lane];
    const float s = ue8m0(rec[kCodeBytes + (lane >> 1)]);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t byte = ((k < 4 ? c.x : c.y) >> (8 * (k & 3))) & 0xFFu;
      const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte), __NV_E2M1);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[2 * k] = f.x * s;
      v[2 * k + 1] = f.y * s;
    }
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(rec) + 8 * lane;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  }
  const uint32_t t = rope ? reinterpret_cast<const uint32_t*>(rec + record_bytes(kFp4, 0))[lane] : 0u;
  v[16] = __uint_as_float(t << 16);
  v[17] = __uint_as_float(t & 0xFFFF0000u);
}

// One block per (row, head): each warp takes every fourth visible record, the dot
// product split over its lanes, and keeps its own running maximum, sum and
// weighted sum of values in registers; the warps are joined at the end.
template <bool kFp4>
__global__ void __launch_bounds__(kThreads) attend_kernel(const csa_latent_attend_args A) {
  const int h = blockIdx.x % A.num_heads, b = blockIdx.x / A.num_heads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rope = A.cache.rope_dim, rec_bytes = record_bytes(kFp4, rope);
  __shared__ float s_o[kThreads / 32][kDim];
  __shared__ float s_m[kThreads / 32], s_l[kThreads / 32];
  int32_t flags = 0;
  const RowView R = row_view(A, b, &flags);
  const __nv_bfloat16* qp =
      static_cast<const __nv_bfloat16*>(A.q) + b * A.q_row_stride + static_cast<int64_t>(h) * A.q_head_stride;
  float q[18], o[16] = {}, m = -INFINITY, l = 0.f;
  lane_values<false>(reinterpret_cast<const uint8_t*>(qp), lane, rope, q);
  const int n = R.table ? (A.idx ? A.top : R.len) : 0;
  for (int j = warp; j < n; j += kThreads / 32) {
    const uint8_t* rec = record_of(A, R, b, j, rec_bytes, &flags);
    if (!rec) continue;
    float v[18], s = 0.f;
    lane_values<kFp4>(rec, lane, rope, v);
#pragma unroll
    for (int k = 0; k < 18; ++k) s = fmaf(q[k], v[k], s);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    s *= A.scale;
    const float top = fmaxf(m, s), keep = expf(m - top), p = expf(s - top);
    m = top;
    l = fmaf(l, keep, p);
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = fmaf(o[k], keep, p * v[k]);
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) s_o[warp][16 * lane + k] = o[k];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.f, w[kThreads / 32];
  for (int k = 0; k < kThreads / 32; ++k) top = fmaxf(top, s_m[k]);
  for (int k = 0; k < kThreads / 32; ++k) {
    w[k] = s_m[k] == -INFINITY ? 0.f : expf(s_m[k] - top);
    sum = fmaf(s_l[k], w[k], sum);
  }
  const int64_t row = static_cast<int64_t>(b) * A.num_heads + h;
  for (int d = threadIdx.x; d < kDim; d += kThreads) {
    float a = 0.f;
    for (int k = 0; k < kThreads / 32; ++k) a = fmaf(s_o[k][d], w[k], a);
    static_cast<__nv_bfloat16*>(A.out)[row * kDim + d] = __float2bfloat16_rn(sum > 0.f ? a / sum : 0.f);
  }
  if (A.lse && threadIdx.x == 0) A.lse[row] = sum > 0.f ? top + logf(sum) : -INFINITY;
  flags = static_cast<int32_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(flags)));
  if (flags && A.dev_status && lane == 0) atomicOr(A.dev_status, flags);
}

csa_status check_args(const csa_latent_attend_args* a) {
  if (!a || a->num_q < 0 || a->num_req < 0 || a->pt_stride < 0 || a->top < 0) return CSA_ERR_INVALID_ARG;
  if (a->num_heads < 1 || a->num_heads > CSA_LATENT_MAX_HEADS) return CSA_ERR_UNSUPPORTED;
  if (!std::isfinite(a->scale) || !(a->scale > 0.f)) return CSA_ERR_INVALID_ARG;
  if (a->num_q == 0) return CSA_OK;
  const csa_status st = check_cache(a->cache);
  if (st != CSA_OK) return st;
  const int wide = kDim + a->cache.rope_dim;
  if (!a->q || !a->page_table || !a->row_len || !a->out || a->num_req < 1 || a->pt_stride < 1)
    return CSA_ERR_INVALID_ARG;
  if (!a->row_req && a->num_req < a->num_q) return CSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(kPageRecs) * a->pt_stride > INT32_MAX) return CSA_ERR_INVALID_ARG;
  if (a->idx ? (a->top < 1 || a->idx_stride < a->top) : a->top != 0) return CSA_ERR_INVALID_ARG;
  if ((a->num_heads > 1 && a->q_head_stride < wide) || (a->num_q > 1 && a->q_row_stride < wide))
    return CSA_ERR_INVALID_ARG;
  if (!aligned(a->q, 16) || a->q_row_stride % 8 != 0 || a->q_head_stride % 8 != 0 || !aligned(a->page_table, 4) ||
      !aligned(a->row_req, 4) || !aligned(a->row_len, 4) || !aligned(a->idx, 4) || !aligned(a->out, 16) ||
      !aligned(a->lse, 4) || !aligned(a->dev_status, 4))
    return CSA_ERR_ALIGNMENT;
  return CSA_OK;
}

}  // namespace
}  // namespace csa_latent

using namespace csa_latent;

extern "C" size_t csa_latent_attend_workspace_bytes(const csa_latent_attend_args* a) {
  return a && a->num_q >= 0 && a->num_heads >= 1 && a->num_heads <= CSA_LATENT_MAX_HEADS ? 16 : 0;
}

extern "C" csa_status csa_latent_attend(const csa_latent_attend_args* a, void* ws, size_t ws_bytes, void* stream) {
  const csa_status st = check_args(a);
  if (st != CSA_OK) return st;
  if (a->num_q == 0) return CSA_OK;
  if (!ws || ws_bytes < csa_latent_attend_workspace_bytes(a)) return CSA_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return CSA_ERR_ALIGNMENT;
  const int64_t blocks = static_cast<int64_t>(a->num_q) * a->num_heads;
  if (blocks > INT32_MAX) return CSA_ERR_INVALID_ARG;
  const auto kernel = a->cache.record_format == CSA_LATENT_MXFP4 ? attend_kernel<true> : attend_kernel<false>;
  kernel<<<static_cast<unsigned>(blocks), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(*a);
  return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}
