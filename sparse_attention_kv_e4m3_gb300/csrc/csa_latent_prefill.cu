// csa_latent_prefill.cu — latent attention, expanded form (include/csa_latent.h).
#include <cuda.h>

#include "csa_latent_common.cuh"
#include "csa_latent_ptx.cuh"

namespace csa_latent {
namespace {

using csa::mbar_arrive;
using csa::mbar_wait;
using csa::smem_u32;

// The kernel. A CTA takes 256 query rows of one request and head as two tiles of 128, and
// runs over tiles of 128 keys: S = Q K^T (128 x 128 over 192), p = 2^(S c - m c) with
// c = scale log2 e, O = O + P V, l = sum p, out = O / l, lse = ln 2 (m c + log2 l). m is the
// first key tile's maximum of the row and moves only when a tile exceeds it by 2^8 (any reference is
// right; a stale one only scales O and l alike), so that O is rarely rescaled.
//
// Bound by the tensor cores (20 MMAs of 64 clocks a tile pair) while the exponentials of one query
// tile run under the MMAs of the other: the order of issue is S0(j), O1(j - 1), S1(j), O0(j), so
// each softmax has 1280 clocks. A row of S is a TMEM lane and belongs to one thread, P goes back over
// S in TMEM as the A operand of O, V is read from shared memory as it lies (N-major).
//
// Shared memory: Q 2 x 48 KB, K 2 x 48 KB, V 32 KB (in two halves of 64 keys, each handed back as soon as
// the last query tile has read it): 224 KB, one CTA an SM. TMEM: S0, S1, O0, O1, all 512 columns.
// Warps 0-3 and 4-7: softmax and output of the two tiles. Warp 8: one thread issues the MMAs.
// Warp 9: TMA; it also zeroes the value rows past a request's last key, which belong to
// others and may hold NaN (P is 0 there, but 0 x NaN is not).
constexpr int kNope = CSA_PREFILL_NOPE, kRope = CSA_PREFILL_ROPE, kV = CSA_PREFILL_V;
constexpr int kTile = 128;                            // query rows, keys
constexpr int kColBytes = kTile * 128;                // 64 values of 128 rows
constexpr int kQCols = (kNope + kRope) / 64, kVCols = kV / 64;
constexpr int kQBytes = kQCols * kColBytes, kVBytes = kVCols * kColBytes;
constexpr int kSoftmaxWarps = 8, kMmaWarp = 8;
constexpr int kThreads = 32 * 10;
constexpr uint32_t kTmemCols = 512, kTmemO = 256;     // S of tile t at 128 t, O at 256 + 128 t
constexpr float kGrow = 8.0f;                         // log2 of how far p may exceed 1

struct Maps {
  CUtensorMap q, k, rope, v;
};

struct Smem {
  uint8_t q[2][kQBytes];
  uint8_t k[2][kQBytes];
  uint8_t v[kVBytes];
  uint64_t bars[20];
  int32_t warp_pairs[kThreads / 32];
  int32_t total, request, first;  // of the item: its request and its first query row there
  uint32_t tmem;
  int abort;
};
enum { kBarQFull = 0, kBarKFull = 1, kBarKEmpty = 3, kBarVFull = 5, kBarVEmpty = 7, kBarVLand = 9, kBarSFull = 10,
       kBarPFull = 12, kBarOFull = 14, kBarDrain = 16 };

// Bounds of request r, false where they descend or leave the tensors.
struct Request {
  int32_t q0, k0, nq, nk;
};

__device__ __forceinline__ bool request_of(const csa_latent_prefill_args& A, int r, Request* R) {
  const int32_t q0 = A.q_start[r], q1 = A.q_start[r + 1], k0 = A.kv_start[r], k1 = A.kv_start[r + 1];
  if (q0 < 0 || q1 < q0 || q1 > A.total_q || k0 < 0 || k1 < k0 || k1 > A.total_k) return false;
  *R = {q0, k0, q1 - q0, k1 - k0};
  return true;
}

__device__ __forceinline__ int pairs_of(const csa_latent_prefill_args& A, int r, bool* bad) {
  Request R;
  if (!request_of(A, r, &R)) {
    *bad = true;
    return 0;
  }
  return (R.nq + 2 * kTile - 1) / (2 * kTile);
}

// Item `at` (from the last pair of query tiles backwards: the longest first, where requests are causal).
__device__ void find_item(const csa_latent_prefill_args& A, Smem& S, int at, bool* bad) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (A.num_req + kThreads - 1) / kThreads;
  const int r0 = min(tid * per, A.num_req), r1 = min(r0 + per, A.num_req);
  int mine = 0;
  for (int r = r0; r < r1; ++r) mine += pairs_of(A, r, bad);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) S.warp_pairs[warp] = incl;
  __syncthreads();
  int before = incl - mine, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += S.warp_pairs[w];
    total += S.warp_pairs[w];
  }
  if (tid == 0) S.total = total;
  const int want = total - 1 - at;
  if (want >= before && want < before + mine) {
    for (int r = r0; r < r1; ++r) {
      bool ignore = false;
      const int n = pairs_of(A, r, &ignore);
      if (want < before + n) {
        S.request = r;
        S.first = (want - before) * 2 * kTile;
        break;
      }
      before += n;
    }
  }
  __syncthreads();
}

// A whole warp's bounded wait, with one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* stop) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, stop));
}

// Key tiles that query tile t (rows first + 128 t ..) sees any key of.
__device__ __forceinline__ int key_tiles(const csa_latent_prefill_args& A, const Request& R, int first, int t) {
  const int row = first + t * kTile;
  if (row >= R.nq) return 0;
  int64_t seen = R.nk;
  if (A.causal) seen = min(seen, static_cast<int64_t>(min(row + kTile, R.nq)) + R.nk - R.nq);
  return seen <= 0 ? 0 : static_cast<int>((seen + kTile - 1) / kTile);
}

__device__ void role_load(const csa_latent_prefill_args& A, const Maps& M, Smem& S, const Request& R, int first, int head) {
  const int lane = threadIdx.x & 31;
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars);
  const int n = max(key_tiles(A, R, first, 0), key_tiles(A, R, first, 1));
  if (n == 0) return;
  if (lane == 0) {
    csa::mbar_arrive_expect_tx(bars + 8 * kBarQFull, 2 * kQBytes);
    for (int t = 0; t < 2; ++t)
      for (int c = 0; c < kQCols; ++c)
        csa::tma_tile_3d(smem_u32(S.q[t]) + c * kColBytes, &M.q, 64 * c, head, R.q0 + first + t * kTile, bars + 8 * kBarQFull);
  }
  bool ok = true;
  int k_done = 0, v_done = 0, landed = 0;
  auto load_k = [&](int j) {
    const uint32_t s = j & 1;
    ok = ok && warp_wait(bars + 8 * (kBarKEmpty + s), ((j >> 1) & 1) ^ 1, stop);
    if (!ok) return;
    if (lane == 0) {
      const uint32_t bar = bars + 8 * (kBarKFull + s), dst = smem_u32(S.k[s]);
      csa::mbar_arrive_expect_tx(bar, kQBytes);
      for (int c = 0; c < kNope / 64; ++c) csa::tma_tile_3d(dst + c * kColBytes, &M.k, 64 * c, head, R.k0 + j * kTile, bar);
      csa::tma_tile_2d(dst + kNope / 64 * kColBytes, &M.rope, 0, R.k0 + j * kTile, bar);
    }
    k_done = j + 1;
  };
  auto load_v = [&](int j) {
    for (int half = 0; half < 2; ++half) {
      ok = ok && warp_wait(bars + 8 * (kBarVEmpty + half), (j & 1) ^ 1, stop);
      if (!ok) return;
      // rows of the half that are this request's; the others become zeros before the half is handed over
      const int rows = min(64, R.nk - j * kTile - 64 * half);
      const bool whole = rows == 64;
      const uint32_t full = bars + 8 * (kBarVFull + half), land = whole ? full : bars + 8 * kBarVLand;
      if (rows > 0 && lane == 0) {
        csa::mbar_arrive_expect_tx(land, kVBytes / 2);
        for (int c = 0; c < kVCols; ++c)
          csa::tma_tile_3d(smem_u32(S.v) + c * kColBytes + half * (kColBytes / 2), &M.v, 64 * c, head,
                           R.k0 + j * kTile + 64 * half, land);
      }
      if (whole) continue;
      if (rows > 0) {
        ok = ok && warp_wait(land, landed & 1, stop);
        ++landed;
      }
      for (int c = 0; c < kVCols; ++c)
        for (int b = max(rows, 0) * 128 + 16 * lane; b < kColBytes / 2; b += 512)
          csa::st_shared_v4(smem_u32(S.v) + c * kColBytes + half * (kColBytes / 2) + b, 0, 0, 0, 0);
      csa::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
    }
    v_done = j + 1;
  };
  // in the order in which the MMAs give the buffers back
  load_k(0);
  load_v(0);
  if (n > 1) load_k(1);
  for (int j = 1; ok && j < n; ++j) {
    if (j + 1 < n) load_k(j + 1);
    if (ok) load_v(j);
  }
  // no copy of this CTA is in flight when it leaves
  if (lane == 0) {
    csa::mbar_wait_drain(bars + 8 * kBarQFull, 0);
    for (int j = max(k_done - 2, 0); j < k_done; ++j) csa::mbar_wait_drain(bars + 8 * (kBarKFull + (j & 1)), (j >> 1) & 1);
    if (ok) {
      for (int half = 0; half < 2; ++half) csa::mbar_wait_drain(bars + 8 * (kBarVFull + half), (v_done - 1) & 1);
    } else {  // gave up: whatever was begun for V lands within the time limit
      for (int half = 0; half < 2; ++half) csa::mbar_wait_drain(bars + 8 * (kBarVFull + half), v_done & 1);
      csa::mbar_wait_drain(bars + 8 * kBarVLand, landed & 1);
    }
  }
  __syncwarp();
}

__device__ void role_mma(const csa_latent_prefill_args& A, Smem& S, const Request& R, int first) {
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars), tmem = S.tmem;
  const int n[2] = {key_tiles(A, R, first, 0), key_tiles(A, R, first, 1)}, most = max(n[0], n[1]);
  constexpr uint32_t idesc_s = csa::idesc_bf16_f32(kTile, kTile);
  constexpr uint32_t idesc_o = csa::idesc_bf16_f32(kTile, kV) | csa::kIdescBMnMajor;
  const csa::Desc q[2] = {csa::Desc(csa::sdesc_kmajor_sw128(smem_u32(S.q[0]))), csa::Desc(csa::sdesc_kmajor_sw128(smem_u32(S.q[1])))};
  const csa::Desc k[2] = {csa::Desc(csa::sdesc_kmajor_sw128(smem_u32(S.k[0]))), csa::Desc(csa::sdesc_kmajor_sw128(smem_u32(S.k[1])))};
  const csa::Desc v(csa::sdesc_mn_sw128_b16(smem_u32(S.v), kColBytes));
  bool ok = most == 0 || mbar_wait(bars + 8 * kBarQFull, 0, stop);
  auto issue_s = [&](int t, int j) {
    const csa::Desc a = t ? q[1] : q[0], b = (j & 1) ? k[1] : k[0];
#pragma unroll
    for (int x = 0; x < kNope + kRope; x += 16) {
      const uint32_t bytes = x / 64 * kColBytes + x % 64 * 2;
      if (x == 0) csa::mma_f16_ss<false>(tmem + t * kTile, a, bytes, b, bytes, idesc_s);
      else csa::mma_f16_ss<true>(tmem + t * kTile, a, bytes, b, bytes, idesc_s);
    }
    csa::mma_commit(bars + 8 * (kBarSFull + t));
  };
  // O of tile t over key tile j; `frees`: the last to read V
  auto issue_o = [&](int t, int j, bool frees) {
    ok = ok && mbar_wait(bars + 8 * (kBarPFull + t), j & 1, stop);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      ok = ok && mbar_wait(bars + 8 * (kBarVFull + half), j & 1, stop);
      if (!ok) return;
      csa::tc_fence_after();
#pragma unroll
      for (int x = 64 * half; x < 64 * half + 64; x += 16) {
        if (j == 0 && x == 0) csa::mma_f16_ts<false>(tmem + kTmemO + t * kTile, tmem + t * kTile + x / 2, v, x * 128, idesc_o);
        else csa::mma_f16_ts<true>(tmem + kTmemO + t * kTile, tmem + t * kTile + x / 2, v, x * 128, idesc_o);
      }
      if (frees) csa::mma_commit(bars + 8 * (kBarVEmpty + half));
    }
    if (j + 1 == n[t]) csa::mma_commit(bars + 8 * (kBarOFull + t));
  };
  for (int j = 0; ok && j < most; ++j) {
    ok = mbar_wait(bars + 8 * (kBarKFull + (j & 1)), (j >> 1) & 1, stop);
    if (!ok) break;
    csa::tc_fence_after();
    if (j < n[0]) issue_s(0, j);
    if (j > 0 && j - 1 < n[1]) issue_o(1, j - 1, true);
    if (!ok) break;
    if (j < n[1]) issue_s(1, j);
    csa::mma_commit(bars + 8 * (kBarKEmpty + (j & 1)));
    if (j < n[0]) issue_o(0, j, j >= n[1]);
  }
  if (ok && n[1] == most && most > 0) issue_o(1, most - 1, true);
  csa::mma_commit(bars + 8 * kBarDrain);
  csa::mbar_wait_drain(bars + 8 * kBarDrain, 0);
}

__device__ void role_softmax(const csa_latent_prefill_args& A, Smem& S, const Request& R, int first, int head) {
  const int t = threadIdx.x >> 7, warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars);
  const uint32_t s_at = S.tmem + t * kTile + (static_cast<uint32_t>(32 * warp) << 16);
  const uint32_t o_at = s_at + kTmemO;
  const int n = key_tiles(A, R, first, t);
  const int row = first + t * kTile + 32 * warp + lane;
  // keys that this row sees, and that every row of the warp sees
  const int64_t past = static_cast<int64_t>(R.nk) - R.nq;
  const int64_t seen = A.causal ? min(max(row + past + 1, int64_t(0)), static_cast<int64_t>(R.nk)) : R.nk;
  const int64_t all_see = A.causal ? min(max(row - lane + past + 1, int64_t(0)), static_cast<int64_t>(R.nk)) : R.nk;
  const float c = A.scale * 1.4426950408889634f, grow = kGrow / c;
  float m = -INFINITY, l = 0.f;
  bool ok = true;
  for (int j = 0; j < n; ++j) {
    ok = ok && warp_wait(bars + 8 * (kBarSFull + t), j & 1, stop);
    if (!ok) break;
    csa::tc_fence_after();
    float s[4][32];
#pragma unroll
    for (int k = 0; k < 4; ++k) csa::tmem_ld32(s_at + 32 * k, reinterpret_cast<uint32_t(&)[32]>(s[k]));
    csa::tmem_wait_ld();
    if (static_cast<int64_t>(j + 1) * kTile > all_see) {
      const int lim = static_cast<int>(min(seen - static_cast<int64_t>(j) * kTile, static_cast<int64_t>(kTile)));
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int x = 0; x < 32; ++x)
          if (32 * k + x >= lim) s[k][x] = -INFINITY;
    }
    float top4[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      top4[k] = s[k][0];
#pragma unroll
      for (int x = 1; x < 32; ++x) top4[k] = fmaxf(top4[k], s[k][x]);
    }
    const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
    const bool up = top > m + grow;
    if (__any_sync(0xFFFFFFFFu, up)) {
      const float keep = up ? csa::ex2((m - top) * c) : 1.f;  // 0 when there was nothing
      if (up) m = top;
      l *= keep;
      if (j > 0) {  // S of this tile is complete, so O of the one before is
#pragma unroll 1
        for (int k = 0; k < kV; k += 32) {
          uint32_t v[32];
          csa::tmem_ld32(o_at + k, v);
          csa::tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * keep);
          csa::tmem_st32(o_at + k, v);
        }
      }
    }
    const float mc = m == -INFINITY ? 0.f : m * c;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t w[32];
#pragma unroll
      for (int x = 0; x < 64; x += 2) {
        const float p0 = csa::ex2(fmaf(s[2 * k + x / 32][x % 32], c, -mc));
        const float p1 = csa::ex2(fmaf(s[2 * k + x / 32][x % 32 + 1], c, -mc));
        sum[x / 2 % 4] += p0 + p1;
        // rounded to bf16 here, the tensor cores' operand type; l sums p unrounded
        const __nv_bfloat162 two = __floats2bfloat162_rn(p0, p1);
        w[x / 2] = *reinterpret_cast<const uint32_t*>(&two);
      }
      csa::tmem_st32(s_at + 32 * k, w);
    }
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    csa::tmem_wait_st();
    csa::tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * (kBarPFull + t));
  }
  if (n > 0) ok = ok && warp_wait(bars + 8 * (kBarOFull + t), 0, stop);
  csa::tc_fence_after();
  const float inv = l > 0.f ? 1.f / l : l;  // a NaN stays one
  const bool there = row < R.nq;
  const int64_t at = static_cast<int64_t>(R.q0 + row) * A.num_heads + head;
  if (there && A.lse) A.lse[at] = l == 0.f ? -INFINITY : (m * c + log2f(l)) * 0.6931471805599453f;
  uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(A.out) + (there ? at : 0) * kV);
#pragma unroll 1
  for (int k = 0; k < kV; k += 32) {
    uint32_t v[32] = {};
    if (n > 0) {
      csa::tmem_ld32(o_at + k, v);
      csa::tmem_wait_ld();
    }
    if (there) {
#pragma unroll
      for (int x = 0; x < 32; x += 8) {
        uint32_t w[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const __nv_bfloat162 two =
              __floats2bfloat162_rn(__uint_as_float(v[x + 2 * y]) * inv, __uint_as_float(v[x + 2 * y + 1]) * inv);
          w[y] = *reinterpret_cast<const uint32_t*>(&two);
        }
        out[(k + x) / 8] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ csa_latent_prefill_args A, const __grid_constant__ Maps M) {
  extern __shared__ uint8_t smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = smem_u32(S.bars);
  const int head = blockIdx.x % A.num_heads;
  bool bad = false;
  find_item(A, S, blockIdx.x / A.num_heads, &bad);
  if (bad && A.dev_status && blockIdx.x == 0) atomicOr(A.dev_status, CSA_DEV_LEN_OOB);
  if (static_cast<int>(blockIdx.x / A.num_heads) >= S.total) return;
  Request R;
  request_of(A, S.request, &R);
  const int first = S.first;
  if (threadIdx.x == 0) {
    csa::mbar_init(bars + 8 * kBarQFull, 1);
    csa::mbar_init(bars + 8 * kBarVLand, 1);
    csa::mbar_init(bars + 8 * kBarDrain, 1);
    for (int k = 0; k < 2; ++k) {
      csa::mbar_init(bars + 8 * (kBarKFull + k), 1);
      csa::mbar_init(bars + 8 * (kBarKEmpty + k), 1);
      csa::mbar_init(bars + 8 * (kBarVFull + k), 1);
      csa::mbar_init(bars + 8 * (kBarVEmpty + k), 1);
      csa::mbar_init(bars + 8 * (kBarSFull + k), 1);
      csa::mbar_init(bars + 8 * (kBarPFull + k), 4);
      csa::mbar_init(bars + 8 * (kBarOFull + k), 1);
    }
    csa::mbar_init_fence();
    S.abort = 0;
  }
  if (warp == kMmaWarp) {
    csa::tmem_alloc(smem_u32(&S.tmem), kTmemCols);
    csa::tmem_relinquish();
  }
  csa::tc_fence_before();
  __syncthreads();
  csa::tc_fence_after();
  if (warp < kSoftmaxWarps) {
    role_softmax(A, S, R, first, head);
  } else if (warp == kMmaWarp) {
    if (lane == 0) role_mma(A, S, R, first);
    __syncwarp();
  } else {
    role_load(A, M, S, R, first, head);
  }
  csa::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    csa::tc_fence_after();
    csa::tmem_dealloc(S.tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && S.abort && A.dev_status) atomicOr(A.dev_status, CSA_DEV_TIMEOUT);
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

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
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

// bf16 [rows][heads][width] in boxes of 64 values of one head and `box` rows, 128-byte swizzle.
bool encode(CUtensorMap* map, const void* base, int64_t width, int64_t heads, int64_t rows, int64_t head_stride,
            int64_t row_stride, uint32_t box) {
  const bool flat = heads == 0;  // [rows][width]
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(flat ? rows : heads),
                              static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(2 * (flat ? row_stride : head_stride)),
                                 static_cast<cuuint64_t>(2 * row_stride)};
  const cuuint32_t boxes[3] = {64, flat ? box : 1, box}, steps[3] = {1, 1, 1};
  return encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, flat ? 2 : 3, const_cast<void*>(base), dims, strides, boxes,
                        steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace csa_latent

using namespace csa_latent;

extern "C" csa_status csa_latent_prefill(const csa_latent_prefill_args* a, void* stream) {
  const csa_status st = check_args(a);
  if (st != CSA_OK) return st;
  if (a->num_req == 0 || a->total_q == 0) return CSA_OK;
  // pairs of query tiles: at most one a request beyond the whole ones
  const int64_t pairs = a->total_q / (2 * kTile) + (a->num_req < a->total_q ? a->num_req : a->total_q);
  if (pairs * a->num_heads > INT32_MAX) return CSA_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CSA_ERR_CUDA;
  static bool ready[64];  // the kernel's shared memory size is set on each device once
  constexpr size_t smem = sizeof(Smem) + 1024;
  static_assert(smem <= 232448, "shared memory of one CTA");
  if (!ready[dev]) {
    if (cudaFuncSetAttribute(prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
      return CSA_ERR_CUDA;
    ready[dev] = true;
  }
  if (!encode_tiled()) return CSA_ERR_CUDA;
  Maps M;
  const bool keys = a->total_k > 0;  // without keys no map of theirs is used: any valid one does
  const int64_t rows = keys ? a->total_k : a->total_q, heads = a->num_heads;
  if (!encode(&M.q, a->q, kNope + kRope, heads, a->total_q, a->q_head_stride, a->q_row_stride, kTile) ||
      !encode(&M.k, keys ? a->k_nope : a->q, kNope, heads, rows, keys ? a->k_head_stride : a->q_head_stride,
              keys ? a->k_row_stride : a->q_row_stride, kTile) ||
      !encode(&M.rope, keys ? a->k_rope : a->q, kRope, 0, rows, 0, keys ? a->rope_row_stride : a->q_row_stride, kTile) ||
      !encode(&M.v, keys ? a->v : a->q, kV, heads, rows, keys ? a->v_head_stride : a->q_head_stride,
              keys ? a->v_row_stride : a->q_row_stride, kTile / 2))
    return CSA_ERR_INVALID_ARG;
  prefill_kernel<<<static_cast<unsigned>(pairs * heads), kThreads, smem, static_cast<cudaStream_t>(stream)>>>(*a, M);
  return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}
