// csa_draft_attend.cu — latent attention of drafted tokens (include/csa_draft.h).
#include "csa_draft.h"
#include "csa_latent_rows.cuh"

namespace csa_latent {
namespace {

struct Request {
  int32_t row0, drafts, base, total;  // total: records that there are, history and drafts
};

// Request r; false where its rows' bounds descend or leave the tensor.
__device__ __forceinline__ bool request_of(const csa_draft_attend_args& A, int r, Request* R, int32_t* flags) {
  const int32_t a = A.row_start[r], b = A.row_start[r + 1], n = A.base_len[r];
  if (a < 0 || b < a || b > A.num_q) {
    *flags |= CSA_DEV_LEN_OOB;
    return false;
  }
  const int64_t cap = static_cast<int64_t>(kPageRecs) * A.pt_stride;
  const int64_t base = min(max(static_cast<int64_t>(n), int64_t(0)), cap), total = min(base + (b - a), cap);
  if (base != n || total != base + (b - a)) *flags |= CSA_DEV_LEN_OOB;
  *R = {a, b - a, static_cast<int32_t>(base), static_cast<int32_t>(total)};
  return true;
}

// Whether draft j (of row row0 + j) sees position p.
__device__ __forceinline__ bool sees(const csa_draft_attend_args& A, const Request& R, int j, int32_t p) {
  const int i = p - R.base;
  if (i < 0) return true;
  if (!A.mask) return i <= j;
  return i < 64 * A.mask_words && (A.mask[(R.row0 + j) * A.mask_stride + i / 64] >> (i % 64) & 1);
}

// A block a query row and head: scores of 64 records, the running maximum and sum, 512 / 128 output values a thread.
__global__ void __launch_bounds__(128) attend_simple(const csa_draft_attend_args A) {
  __shared__ float q[kDim + 64], s[kPageRecs];
  __shared__ int32_t found;
  __shared__ Request R;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.x % A.num_heads, b = blockIdx.x / A.num_heads;
  const bool fp4 = A.cache.record_format == CSA_LATENT_MXFP4;
  const int rope = A.cache.rope_dim, rec_bytes = record_bytes(fp4, rope);
  int32_t flags = 0;
  if (tid == 0) found = -1;
  __syncthreads();
  for (int r = tid; r < A.num_req; r += 128) {
    Request X;
    if (request_of(A, r, &X, &flags) && b >= X.row0 && b < X.row0 + X.drafts) found = r;
  }
  __syncthreads();
  if (flags && A.dev_status) atomicOr(A.dev_status, flags);
  flags = 0;
  const int r = found;
  if (r < 0) return;
  if (tid == 0) request_of(A, r, &R, &flags);
  const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(A.q) + b * A.q_row_stride + h * A.q_head_stride;
  for (int i = tid; i < kDim + rope; i += 128) q[i] = __bfloat162float(qp[i]);
  __syncthreads();
  const int j = b - R.row0;
  float m = -INFINITY, l = 0.f, o[4] = {};
  auto value = [&](const uint8_t* rec, int i) {
    if (!fp4) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(rec)[i]);
    if (i >= kDim) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(rec + kCodeBytes + kScaleBytes)[i - kDim]);
    const uint32_t code = rec[i / 2] >> (4 * (i & 1)) & 15, mag = code & 7;
    const float v = mag < 2 ? 0.5f * mag : ldexpf(1.f + 0.5f * (mag & 1), (mag >> 1) - 1);
    return (code & 8 ? -v : v) * ue8m0(rec[kCodeBytes + i / 32]);
  };
  for (int p0 = 0; p0 < R.total; p0 += kPageRecs) {
    const int32_t page = A.page_table[static_cast<int64_t>(r) * A.pt_stride + p0 / kPageRecs];
    if (page < 0 || page >= A.cache.num_pages) {
      flags |= CSA_DEV_PAGE_OOB;
      continue;
    }
    const uint8_t* recs = A.cache.pages + page * A.cache.page_stride_bytes;
    for (int n = warp; n < kPageRecs; n += 4) {
      float sum = 0.f;
      const bool live = p0 + n < R.total && sees(A, R, j, p0 + n);
      if (live)
        for (int i = lane; i < kDim + rope; i += 32) sum = fmaf(q[i], value(recs + n * rec_bytes, i), sum);
      for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, k);
      if (lane == 0) s[n] = live ? sum * A.scale : -INFINITY;
    }
    __syncthreads();
    float top = m;
    for (int n = 0; n < kPageRecs; ++n) top = fmaxf(top, s[n]);
    if (top > -INFINITY) {
      const float keep = expf(m - top);
      l *= keep;
      for (int k = 0; k < 4; ++k) o[k] *= keep;
      for (int n = 0; n < kPageRecs; ++n) {
        if (s[n] == -INFINITY) continue;
        const float p = expf(s[n] - top);
        l += p;
        for (int k = 0; k < 4; ++k) o[k] = fmaf(p, value(recs + n * rec_bytes, tid + 128 * k), o[k]);
      }
      m = top;
    }
    __syncthreads();
  }
  const int64_t row = static_cast<int64_t>(b) * A.num_heads + h;
  for (int k = 0; k < 4; ++k) static_cast<__nv_bfloat16*>(A.out)[row * kDim + tid + 128 * k] = __float2bfloat16(l > 0.f ? o[k] / l : l);
  if (tid == 0 && A.lse) A.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
  if (flags && A.dev_status) atomicOr(A.dev_status, flags);
}

csa_status check_args(const csa_draft_attend_args* a) {
  if (!a || a->num_q < 0 || a->num_req < 0 || a->pt_stride < 0 || a->mask_words < 0) return CSA_ERR_INVALID_ARG;
  if (a->num_heads < 1 || a->num_heads > CSA_LATENT_MAX_HEADS || a->mask_words > CSA_DRAFT_MAX_WORDS) return CSA_ERR_UNSUPPORTED;
  if (!good_scale(a->scale)) return CSA_ERR_INVALID_ARG;
  if (a->num_q == 0 || a->num_req == 0) return CSA_OK;
  const csa_status st = check_cache(a->cache);
  if (st != CSA_OK) return st;
  const int wide = kDim + a->cache.rope_dim;
  if (!a->q || !a->page_table || !a->base_len || !a->row_start || !a->out || a->pt_stride < 1) return CSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(kPageRecs) * a->pt_stride > INT32_MAX) return CSA_ERR_INVALID_ARG;
  if (a->mask ? (a->mask_words < 1 || (a->num_q > 1 && a->mask_stride < a->mask_words)) : a->mask_words != 0) return CSA_ERR_INVALID_ARG;
  if ((a->num_heads > 1 && a->q_head_stride < wide) || (a->num_q > 1 && a->q_row_stride < wide)) return CSA_ERR_INVALID_ARG;
  if (!aligned(a->q, 16) || a->q_row_stride % 8 != 0 || a->q_head_stride % 8 != 0 || !aligned(a->page_table, 4) || !aligned(a->base_len, 4) ||
      !aligned(a->row_start, 4) || !aligned(a->mask, 8) || !aligned(a->out, 16) || !aligned(a->lse, 4) || !aligned(a->dev_status, 4))
    return CSA_ERR_ALIGNMENT;
  return CSA_OK;
}

}  // namespace
}  // namespace csa_latent

using namespace csa_latent;

extern "C" size_t csa_draft_attend_workspace_bytes(const csa_draft_attend_args* a) {
  if (!a || a->num_q < 0 || a->num_req < 0 || a->num_heads < 1 || a->num_heads > CSA_LATENT_MAX_HEADS) return 0;
  return 16;
}

extern "C" csa_status csa_draft_attend(const csa_draft_attend_args* a, void* ws, size_t ws_bytes, void* stream) {
  const csa_status st = check_args(a);
  if (st != CSA_OK) return st;
  if (a->num_q == 0 || a->num_req == 0) return CSA_OK;
  if (!ws || ws_bytes < csa_draft_attend_workspace_bytes(a)) return CSA_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return CSA_ERR_ALIGNMENT;
  if (static_cast<int64_t>(a->num_q) * a->num_heads > INT32_MAX) return CSA_ERR_INVALID_ARG;
  attend_simple<<<static_cast<unsigned>(a->num_q * a->num_heads), 128, 0, static_cast<cudaStream_t>(stream)>>>(*a);
  return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}
