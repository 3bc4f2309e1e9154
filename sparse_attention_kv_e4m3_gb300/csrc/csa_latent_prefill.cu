// csa_latent_prefill.cu — latent attention, expanded form (include/csa_latent.h).
#include "csa_latent_common.cuh"

namespace csa_latent {
namespace {

constexpr int kThreads = 128;
constexpr int kV = CSA_PREFILL_V;

__device__ __forceinline__ float2 pair_of(const void* base, int64_t off, int k) {
  const uint32_t w = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(base) + off)[k];
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Bounds of request r, false where they descend or leave the tensors.
__device__ __forceinline__ bool request_bounds(const csa_latent_prefill_args& A, int r, int32_t* q0, int32_t* q1,
                                               int32_t* k0, int32_t* k1) {
  *q0 = A.q_start[r];
  *q1 = A.q_start[r + 1];
  *k0 = A.kv_start[r];
  *k1 = A.kv_start[r + 1];
  return *q0 >= 0 && *q1 >= *q0 && *q1 <= A.total_q && *k0 >= 0 && *k1 >= *k0 && *k1 <= A.total_k;
}

// One block per (query row, head): each warp takes every fourth visible key.
__global__ void __launch_bounds__(kThreads) prefill_kernel(const csa_latent_prefill_args A) {
  const int h = blockIdx.x % A.num_heads;
  const int64_t i = blockIdx.x / A.num_heads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ float s_o[kThreads / 32][kV];
  __shared__ float s_m[kThreads / 32], s_l[kThreads / 32];
  int32_t q0 = 0, q1 = 0, k0 = 0, k1 = 0;
  bool mine = false, bad = false;
  for (int r = 0; r < A.num_req && !mine; ++r) {
    const bool ok = request_bounds(A, r, &q0, &q1, &k0, &k1);
    bad |= !ok;
    mine = ok && i >= q0 && i < q1;
  }
  if (bad && A.dev_status && threadIdx.x == 0) atomicOr(A.dev_status, CSA_DEV_LEN_OOB);
  if (!mine) return;
  const int64_t past = static_cast<int64_t>(k1 - k0) - (q1 - q0);
  const int64_t seen = A.causal ? min(max(i - q0 + past + 1, int64_t(0)), int64_t(k1 - k0)) : k1 - k0;
  const int64_t q_off = i * A.q_row_stride + h * A.q_head_stride;
  float2 q[3], o[2] = {};
#pragma unroll
  for (int t = 0; t < 3; ++t) q[t] = pair_of(A.q, q_off, 32 * t + lane);
  float m = -INFINITY, l = 0.f;
  for (int64_t j = warp; j < seen; j += kThreads / 32) {
    const int64_t row = k0 + j, k_off = row * A.k_row_stride + h * A.k_head_stride;
    const float2 a = pair_of(A.k_nope, k_off, lane), c = pair_of(A.k_nope, k_off, 32 + lane);
    const float2 e = pair_of(A.k_rope, row * A.rope_row_stride, lane);
    float s = q[0].x * a.x + q[0].y * a.y + q[1].x * c.x + q[1].y * c.y + q[2].x * e.x + q[2].y * e.y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    s *= A.scale;
    const float top = fmaxf(m, s), keep = expf(m - top), p = expf(s - top);
    m = top;
    l = fmaf(l, keep, p);
    const int64_t v_off = row * A.v_row_stride + h * A.v_head_stride;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float2 v = pair_of(A.v, v_off, 32 * t + lane);
      o[t].x = fmaf(o[t].x, keep, p * v.x);
      o[t].y = fmaf(o[t].y, keep, p * v.y);
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) reinterpret_cast<float2*>(s_o[warp])[32 * t + lane] = o[t];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.f, w[kThreads / 32], acc = 0.f;
  for (int k = 0; k < kThreads / 32; ++k) top = fmaxf(top, s_m[k]);
  for (int k = 0; k < kThreads / 32; ++k) {
    w[k] = s_m[k] == -INFINITY ? 0.f : expf(s_m[k] - top);
    sum = fmaf(s_l[k], w[k], sum);
    acc = fmaf(s_o[k][threadIdx.x], w[k], acc);
  }
  const int64_t row = i * A.num_heads + h;
  static_cast<__nv_bfloat16*>(A.out)[row * kV + threadIdx.x] = __float2bfloat16_rn(sum > 0.f ? acc / sum : 0.f);
  if (A.lse && threadIdx.x == 0) A.lse[row] = sum > 0.f ? top + logf(sum) : -INFINITY;
}

csa_status check_args(const csa_latent_prefill_args* a) {
  if (!a || a->num_req < 0 || a->total_q < 0 || a->total_k < 0 || (a->causal != 0 && a->causal != 1))
    return CSA_ERR_INVALID_ARG;
  if (a->num_heads < 1 || a->num_heads > 65535) return CSA_ERR_UNSUPPORTED;
  if (!std::isfinite(a->scale) || !(a->scale > 0.f)) return CSA_ERR_INVALID_ARG;
  if (a->total_q > INT32_MAX || a->total_k > INT32_MAX || a->total_q * a->num_heads > INT32_MAX)
    return CSA_ERR_INVALID_ARG;
  if (a->num_req == 0 || a->total_q == 0) return CSA_OK;
  if (!a->q || !a->q_start || !a->kv_start || !a->out) return CSA_ERR_INVALID_ARG;
  if (a->total_k > 0 && (!a->k_nope || !a->k_rope || !a->v)) return CSA_ERR_INVALID_ARG;
  const int64_t row[] = {a->q_row_stride, a->k_row_stride, a->rope_row_stride, a->v_row_stride};
  const int64_t head[] = {a->q_head_stride, a->k_head_stride, a->v_head_stride};
  for (int64_t s : row)
    if (s < 1) return CSA_ERR_INVALID_ARG;
  for (int64_t s : head)
    if (s < 1) return CSA_ERR_INVALID_ARG;
  for (int64_t s : row)
    if (s % 8 != 0) return CSA_ERR_ALIGNMENT;
  for (int64_t s : head)
    if (s % 8 != 0) return CSA_ERR_ALIGNMENT;
  if (!aligned(a->q, 16) || !aligned(a->k_nope, 16) || !aligned(a->k_rope, 16) || !aligned(a->v, 16) ||
      !aligned(a->out, 16) || !aligned(a->lse, 4) || !aligned(a->q_start, 4) || !aligned(a->kv_start, 4) ||
      !aligned(a->dev_status, 4))
    return CSA_ERR_ALIGNMENT;
  return CSA_OK;
}

}  // namespace
}  // namespace csa_latent

using namespace csa_latent;

extern "C" csa_status csa_latent_prefill(const csa_latent_prefill_args* a, void* stream) {
  const csa_status st = check_args(a);
  if (st != CSA_OK) return st;
  if (a->num_req == 0 || a->total_q == 0) return CSA_OK;
  prefill_kernel<<<static_cast<unsigned>(a->total_q * a->num_heads), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(*a);
  return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}
