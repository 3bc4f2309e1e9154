// csa_latent_prefill.cu — latent attention, expanded form (include/csa_latent.h).
#include <type_traits>

#include "csa_latent_common.cuh"
#include "csa_latent_maps.h"
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
// tile run under the MMAs of the other. A row of S is a TMEM lane and belongs to one thread, P goes back over
// S in TMEM as the A operand of O, V is read from shared memory as it lies (N-major).
//
// Shared memory: Q 2 x 48 KB and a ring of eight 16 KB chunks through which K(0), V(0), K(1), V(1), ... go in
// turn (K(j) takes the place of K(j - 2)'s end and V(j - 2), V(j) that of K(j - 1)'s beginning), so that V has two
// and a half of the MMAs' rounds to arrive and K one: 224 KB, one CTA an SM. TMEM: S0, S1, O0, O1, all 512 columns.
// Warps 0-3 and 4-7: softmax and output of the two tiles. Warp 8 issues the MMAs.
// Warp 9: TMA; it also zeroes the value rows past a request's last key, which belong to
// others and may hold NaN (P is 0 there, but 0 x NaN is not).
constexpr int kNope = CSA_PREFILL_NOPE, kRope = CSA_PREFILL_ROPE, kV = CSA_PREFILL_V;
constexpr int kTile = 128;                            // query rows, keys
constexpr int kColBytes = kTile * 128;                // 64 values of 128 rows
constexpr int kQCols = (kNope + kRope) / 64;
constexpr int kQBytes = kQCols * kColBytes;
constexpr int kRing = 8;                              // chunks of 16 KB: K is 3 (64 values of 128 keys each), V 2 (64 keys each)
constexpr int kTileChunks = kQCols + 2;
constexpr int kSoftmaxWarps = 8, kMmaWarp = 8;
constexpr int kThreads = 32 * 10;
constexpr uint32_t kTmemCols = 512, kTmemO = 256;     // S of tile t at 128 t, O at 256 + 128 t
constexpr float kGrow = 8.0f;                         // log2 of how far p may exceed 1

struct Maps {
  CUtensorMap q, k, rope, v;
};

struct Smem {
  uint8_t q[2][kQBytes];
  uint8_t ring[kRing][kColBytes];
  uint64_t bars[24];
  int32_t warp_pairs[kThreads / 32];
  int32_t total, request, first;  // of the item: its request and its first query row there
  uint32_t tmem;
  int abort;
};
// K, V: by the key tile's parity (V also by half: 2 * parity + half); S, P, O, Q: by query tile
enum { kBarQFull = 0, kBarKFull = 2, kBarKEmpty = 4, kBarVFull = 6, kBarVEmpty = 10, kBarSFull = 12, kBarPFull = 14,
       kBarOFull = 16, kBarVLand = 18, kBarDrain };

// Where chunk i of key tile j lies: K 0 .. 2, V 3, 4.
__device__ __forceinline__ uint32_t ring_slot(int j, int i) { return static_cast<uint32_t>(kTileChunks * j + i) % kRing; }

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
  const int nt[2] = {key_tiles(A, R, first, 0), key_tiles(A, R, first, 1)}, n = max(nt[0], nt[1]);
  if (n == 0) return;
  auto load_q = [&](int t) {
    if (lane != 0 || nt[t] == 0) return;
    csa::mbar_arrive_expect_tx(bars + 8 * (kBarQFull + t), kQBytes);
    for (int c = 0; c < kQCols; ++c)
      csa::tma_tile_3d(smem_u32(S.q[t]) + c * kColBytes, &M.q, 64 * c, head, R.q0 + first + t * kTile, bars + 8 * (kBarQFull + t));
  };
  csa::test_delay();
  bool ok = true, landing = false;  // landing: a copy to kBarVLand is in flight
  int k_done = 0, v_done[2] = {0, 0}, landed = 0;  // tiles loaded, of V by halves
  const uint32_t ring = smem_u32(S.ring[0]);
  auto freed = [&](int bar, int j) {  // what tile j held there has been read (nothing held it where j < 0)
    ok = ok && (j < 0 || warp_wait(bars + 8 * (bar + (j & 1)), (j >> 1) & 1, stop));
    return ok;
  };
  auto load_k = [&](int j) {
    if (!freed(kBarKEmpty, j - 2)) return;
    const uint32_t bar = bars + 8 * (kBarKFull + (j & 1));
    const int row = R.k0 + j * kTile;
    if (lane == 0) {
      csa::mbar_arrive_expect_tx(bar, kColBytes);
      csa::tma_tile_3d(ring + ring_slot(j, 0) * kColBytes, &M.k, 0, head, row, bar);
    }
    k_done = j + 1;
    if (!freed(kBarVEmpty, j - 2)) {
      if (lane == 0) mbar_arrive(bar);  // no more is coming: the first chunk's landing can be waited for
      return;
    }
    if (lane == 0) {
      csa::mbar_arrive_expect_tx(bar, 2 * kColBytes);
      csa::tma_tile_3d(ring + ring_slot(j, 1) * kColBytes, &M.k, 64, head, row, bar);
      csa::tma_tile_2d(ring + ring_slot(j, 2) * kColBytes, &M.rope, 0, row, bar);
    }
  };
  auto load_v = [&](int j) {
    if (!freed(kBarKEmpty, j - 1)) return;
    for (int half = 0; half < 2; ++half) {
      // rows of the half that are this request's; the others become zeros before the half is handed over
      const int rows = min(64, R.nk - j * kTile - 64 * half);
      const bool whole = rows == 64;
      const uint32_t full = bars + 8 * (kBarVFull + 2 * (j & 1) + half), land = whole ? full : bars + 8 * kBarVLand;
      const uint32_t dst = ring + ring_slot(j, kQCols + half) * kColBytes;
      if (rows > 0 && lane == 0) {
        csa::mbar_arrive_expect_tx(land, kColBytes);
        for (int c = 0; c < kV / 64; ++c)
          csa::tma_tile_3d(dst + c * (kColBytes / 2), &M.v, 64 * c, head, R.k0 + j * kTile + 64 * half, land);
      }
      if (whole) v_done[half] = j + 1;
      if (whole) continue;
      if (rows > 0) {
        landing = true;
        ok = ok && warp_wait(land, landed & 1, stop);
        if (!ok) return;
        landing = false;
        ++landed;
      }
      for (int c = 0; c < kV / 64; ++c)
        for (int b = max(rows, 0) * 128 + 16 * lane; b < kColBytes / 2; b += 512) csa::st_shared_v4(dst + c * (kColBytes / 2) + b, 0, 0, 0, 0);
      csa::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
      v_done[half] = j + 1;
    }
  };
  // in the order in which the MMAs give the chunks back
  load_q(0);
  load_k(0);
  load_q(1);
  load_v(0);
  if (n > 1) load_k(1);
  for (int j = 1; ok && j < n; ++j) {
    load_v(j);
    if (ok && j + 1 < n) load_k(j + 1);
  }
  // no copy of this CTA is in flight when it leaves
  if (lane == 0) {
    for (int t = 0; t < 2; ++t)
      if (nt[t] > 0) csa::mbar_wait_drain(bars + 8 * (kBarQFull + t), 0);
    for (int j = max(k_done - 2, 0); j < k_done; ++j) csa::mbar_wait_drain(bars + 8 * (kBarKFull + (j & 1)), (j >> 1) & 1);
    for (int half = 0; half < 2; ++half)
      for (int j = max(v_done[half] - 2, 0); j < v_done[half]; ++j)
        csa::mbar_wait_drain(bars + 8 * (kBarVFull + 2 * (j & 1) + half), (j >> 1) & 1);
    if (landing) csa::mbar_wait_drain(bars + 8 * kBarVLand, landed & 1);
  }
  __syncwarp();
}

// One warp issues all MMAs, S0(j), O1(j - 1), S1(j), O0(j) in turn, with as few waits and commits in
// between as the buffers need: each costs the tensor cores some 80 clocks, and a thread of its own for
// each query tile costs more (their MMAs interleave, and every softmax waits longer for its S).
__device__ void role_mma(const csa_latent_prefill_args& A, Smem& S, const Request& R, int first) {
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars), tmem = csa::uniform(S.tmem), lead = csa::elect_lane();
  const int n[2] = {static_cast<int>(csa::uniform(key_tiles(A, R, first, 0))), static_cast<int>(csa::uniform(key_tiles(A, R, first, 1)))};
  const int most = max(n[0], n[1]);
  constexpr uint32_t idesc_s = csa::idesc_bf16_f32(kTile, kTile);
  constexpr uint32_t idesc_o = csa::idesc_bf16_f32(kTile, kV) | csa::kIdescBMnMajor;
  const csa::Desc q[2] = {csa::Desc(csa::sdesc_kmajor_sw128(smem_u32(S.q[0]))), csa::Desc(csa::sdesc_kmajor_sw128(smem_u32(S.q[1])))};
  const csa::Desc k_ring(csa::sdesc_kmajor_sw128(smem_u32(S.ring[0])));
  const csa::Desc v_ring(csa::sdesc_mn_sw128_b16(smem_u32(S.ring[0]), kColBytes / 2));
  bool ok = true;
  auto need = [&](int bar, uint32_t parity) {
    ok = ok && warp_wait(bars + 8 * bar, parity, stop);
    csa::tc_fence_after();
  };
  // S of tile t over key tile j. `ahead` looks, while these MMAs run, whether what comes after is there.
  auto issue_s = [&](auto tile, int j, auto ahead) {
    constexpr int t = decltype(tile)::value;
    if (!ok) return;
#pragma unroll
    for (int c = 0; c < kQCols; ++c) {
      const csa::Desc b = k_ring.at(ring_slot(j, c) * kColBytes);
#pragma unroll
      for (int x = 0; x < 4; ++x)
        csa::mma_f16_ss(lead, tmem + t * kTile, q[t].at(c * kColBytes + 32 * x), b.at(32 * x), idesc_s, c > 0 || x > 0);
      if (c == 1) ahead();
    }
    csa::mma_commit_if(lead, bars + 8 * (kBarSFull + t));
  };
  // O of tile t over key tile j. `last_reader`: V is free afterwards
  auto issue_o = [&](auto tile, int j, bool last_reader, auto ahead) {
    constexpr int t = decltype(tile)::value;
    if (!ok) return;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const csa::Desc b = v_ring.at(ring_slot(j, kQCols + half) * kColBytes);
#pragma unroll
      for (int x = 0; x < 4; ++x)
        csa::mma_f16_ts(lead, tmem + kTmemO + t * kTile, tmem + t * kTile + 32 * half + 8 * x, b.at(2048 * x), idesc_o,
                        j > 0 || half > 0 || x > 0);
      if (half == 0) ahead();
    }
    if (last_reader) csa::mma_commit_if(lead, bars + 8 * (kBarVEmpty + (j & 1)));
    if (j + 1 == n[t]) csa::mma_commit_if(lead, bars + 8 * (kBarOFull + t));
  };
  const std::integral_constant<int, 0> t0;
  const std::integral_constant<int, 1> t1;
  const auto nothing = [] {};
  // What O of tile t over key tile j needs. A first look that finds it costs nothing: MMAs are still queued.
  auto there = [&](int bar, uint32_t parity) { return static_cast<bool>(__all_sync(0xFFFFFFFFu, csa::mbar_test(bars + 8 * bar, parity))); };
  auto look_o = [&](int t, int j) {
    const int seen = there(kBarPFull + t, j & 1) + 2 * there(kBarVFull + 2 * (j & 1), (j >> 1) & 1) +
                     4 * there(kBarVFull + 2 * (j & 1) + 1, (j >> 1) & 1);
    csa::tc_fence_after();
    return seen;
  };
  auto need_o = [&](int t, int j, int seen) {
    if (!(seen & 2)) need(kBarVFull + 2 * (j & 1), (j >> 1) & 1);
    if (!(seen & 4)) need(kBarVFull + 2 * (j & 1) + 1, (j >> 1) & 1);
    if (!(seen & 1)) need(kBarPFull + t, j & 1);
  };
  if (most > 0) need(kBarKFull, 0);
  if (n[0] > 0) need(kBarQFull, 0);
  for (int j = 0; ok && j < most; ++j) {
    const bool s0 = j < n[0], s1 = j < n[1], o1 = j > 0 && j - 1 < n[1];
    int seen1 = 0, seen0 = 0;
    bool seen_k = false;
    if (s0)
      issue_s(t0, j, [&] {
        if (o1) seen1 = look_o(1, j - 1);
      });
    if (o1) {
      need_o(1, j - 1, seen1);
      issue_o(t1, j - 1, true, nothing);
    }
    if (j == 0 && s1) need(kBarQFull + 1, 0);
    if (s1)
      issue_s(t1, j, [&] {
        if (s0) seen0 = look_o(0, j);
      });
    csa::mma_commit_if(lead, bars + 8 * (kBarKEmpty + (j & 1)));
    const int k_bar = kBarKFull + ((j + 1) & 1);
    const uint32_t k_parity = ((j + 1) >> 1) & 1;
    if (s0) {
      need_o(0, j, seen0);
      issue_o(t0, j, !s1, [&] {
        if (j + 1 < most) {
          seen_k = there(k_bar, k_parity);
          csa::tc_fence_after();
        }
      });
    }
    if (j + 1 < most && !seen_k) need(k_bar, k_parity);
  }
  if (ok && n[1] == most && most > 0) {
    need_o(1, most - 1, 0);
    issue_o(t1, most - 1, true, nothing);
  }
  csa::mma_commit_if(lead, bars + 8 * kBarDrain);  // nothing of this thread's is in flight when it leaves
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
    const csa::F2 c2(c, c), mc2(-mc, -mc);
    csa::F2 sum[4];
    // the exponentials of 32 keys ahead of the rounding of the 32 before them
    auto exps = [&](int k) {
#pragma unroll
      for (int x = 0; x < 32; x += 2) {
        csa::fma2(csa::F2(s[k][x], s[k][x + 1]), c2, mc2).get(s[k][x], s[k][x + 1]);
        s[k][x] = csa::ex2(s[k][x]);
        s[k][x + 1] = csa::ex2(s[k][x + 1]);
      }
    };
    exps(0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k < 3) exps(k + 1);
      uint32_t w[16];
#pragma unroll
      for (int x = 0; x < 32; x += 2) {
        sum[x / 2 % 4] = csa::add2(sum[x / 2 % 4], csa::F2(s[k][x], s[k][x + 1]));
        // rounded to bf16 here, the tensor cores' operand type; l sums p unrounded
        const __nv_bfloat162 two = __floats2bfloat162_rn(s[k][x], s[k][x + 1]);
        w[x / 2] = *reinterpret_cast<const uint32_t*>(&two);
      }
      csa::tmem_st16(s_at + 16 * k, w);
    }
    float l0, l1;
    csa::add2(csa::add2(sum[0], sum[1]), csa::add2(sum[2], sum[3])).get(l0, l1);
    l += l0 + l1;
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
  // through this tile's Q (its last S is done), so that a row is written as 256 contiguous bytes: row r of the warp at 256 r, its
  // 16-byte chunks exchanged by r so that neither side has lanes on one bank
  const uint32_t stage = smem_u32(S.q[t]) + warp * 32 * 256;
#pragma unroll 1
  for (int k = 0; k < kV; k += 32) {
    uint32_t v[32] = {};
    if (n > 0) {
      csa::tmem_ld32(o_at + k, v);
      csa::tmem_wait_ld();
    }
#pragma unroll
    for (int x = 0; x < 32; x += 8) {
      uint32_t w[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const __nv_bfloat162 two = __floats2bfloat162_rn(__uint_as_float(v[x + 2 * y]) * inv, __uint_as_float(v[x + 2 * y + 1]) * inv);
        w[y] = *reinterpret_cast<const uint32_t*>(&two);
      }
      csa::st_shared_v4(stage + lane * 256 + ((((k + x) / 8) ^ (lane & 15)) << 4), w[0], w[1], w[2], w[3]);
    }
  }
  __syncwarp();
  const int rows = min(32, R.nq - (first + t * kTile + 32 * warp));  // of this warp's
  uint8_t* out = static_cast<uint8_t*>(A.out) +
                 2 * ((static_cast<int64_t>(R.q0 + first + t * kTile + 32 * warp) * A.num_heads + head) * kV) + 16 * (lane & 15);
#pragma unroll 4
  for (int r = lane >> 4; r < rows; r += 2) {
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "r"(stage + r * 256 + (((lane & 15) ^ (r & 15)) << 4))
                 : "memory");
    *reinterpret_cast<uint4*>(out + static_cast<int64_t>(r) * A.num_heads * (2 * kV)) = x;
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ csa_latent_prefill_args A, const __grid_constant__ Maps M) {
  extern __shared__ uint8_t smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
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
    csa::mbar_init(bars + 8 * kBarVLand, 1);
    csa::mbar_init(bars + 8 * kBarDrain, 1);
    for (int k = 0; k < 2; ++k) {
      csa::mbar_init(bars + 8 * (kBarQFull + k), 1);
      csa::mbar_init(bars + 8 * (kBarKFull + k), 2);  // K comes in two parts
      csa::mbar_init(bars + 8 * (kBarKEmpty + k), 1);
      csa::mbar_init(bars + 8 * (kBarVFull + 2 * k), 1);
      csa::mbar_init(bars + 8 * (kBarVFull + 2 * k + 1), 1);
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
    role_mma(A, S, R, first);
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
  int sms = 0, dev = 0;
  if (sm_count(&sms, &dev) != CSA_OK) return CSA_ERR_CUDA;
  static bool ready[kMaxDevices];  // the kernel's shared memory size is set on each device once
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
  if (!encode_bf16(&M.q, a->q, kNope + kRope, heads, a->total_q, a->q_head_stride, a->q_row_stride, 1, kTile) ||
      !encode_bf16(&M.k, keys ? a->k_nope : a->q, kNope, heads, rows, keys ? a->k_head_stride : a->q_head_stride,
                   keys ? a->k_row_stride : a->q_row_stride, 1, kTile) ||
      !encode_bf16(&M.rope, keys ? a->k_rope : a->q, kRope, 0, rows, 0, keys ? a->rope_row_stride : a->q_row_stride, 1, kTile) ||
      !encode_bf16(&M.v, keys ? a->v : a->q, kV, heads, rows, keys ? a->v_head_stride : a->q_head_stride,
                   keys ? a->v_row_stride : a->q_row_stride, 1, kTile / 2))
    return CSA_ERR_INVALID_ARG;
  prefill_kernel<<<static_cast<unsigned>(pairs * heads), kThreads, smem, static_cast<cudaStream_t>(stream)>>>(*a, M);
  return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}
