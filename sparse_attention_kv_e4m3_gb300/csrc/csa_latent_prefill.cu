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

// The kernel. An item is 256 query rows of one request and head, as two tiles of 128; it runs over tiles of 128 keys:
// S = Q K^T (128 x 128 over 192), p = 2^(S c - m c) with c = scale log2 e, O = O + P V, l = sum p, out = O / l,
// lse = ln 2 (m c + log2 l). m is the first key tile's maximum of the row and moves only when a tile exceeds it by 2^8 (any
// reference is right; a stale one only scales O and l alike), so that O is rarely rescaled.
//
// Bound by the tensor cores (20 MMAs of 64 clocks a tile pair) while the exponentials of one query
// tile run under the MMAs of the other. A row of S is a TMEM lane and belongs to one thread, P goes back over
// S in TMEM as the A operand of O, V is read from shared memory as it lies (N-major).
// 4096 rows over 16384 keys, 16 heads: 430 us, 1.40 PFLOP/s. 8 prompts of 130 to 2048, 32 heads: 150 us, 0.93 PFLOP/s:
// there items are 1 to 16 key tiles, and what is lost is their ends, where the softmax warps write 64 KB (5 k clocks a tile).
//
// One block an item, but a block that is at the end of its item takes the place of one that has not started yet, so that the next
// item's Q and K come in and its first S is computed while the softmax warps write the last one's output (171 us with a block
// for each item: its start, the first loads and the last O were 42% of the time; the longer case lost 1% then).
//
// Shared memory: Q 2 x 48 KB and a ring of eight 16 KB chunks through which K(0), V(0), K(1), V(1), ... go in
// turn (K(g) takes the place of K(g - 2)'s end and V(g - 2), V(g) that of K(g - 1)'s beginning), so that V has two
// and a half of the MMAs' rounds to arrive and K one: 224 KB, one CTA an SM. TMEM: S0, S1, O0, O1, all 512 columns.
// Warps 0-3 and 4-7: softmax and output of the two tiles. Warp 8 issues the MMAs.
// Warp 9: TMA; it also zeroes the value rows past a request's last key, which belong to
// others and may hold NaN (P is 0 there, but 0 x NaN is not). Warp 10 finds the items.
constexpr int kNope = CSA_PREFILL_NOPE, kRope = CSA_PREFILL_ROPE, kV = CSA_PREFILL_V;
constexpr int kTile = 128;                            // query rows, keys
constexpr int kColBytes = kTile * 128;                // 64 values of 128 rows
constexpr int kQCols = (kNope + kRope) / 64;
constexpr int kQBytes = kQCols * kColBytes;
constexpr int kRing = 8;                              // chunks of 16 KB: K is 3 (64 values of 128 keys each), V 2 (64 keys each)
constexpr int kTileChunks = kQCols + 2;
constexpr int kSoftmaxWarps = 8, kMmaWarp = 8, kLoadWarp = 9;  // and warp 10: role_next
constexpr int kThreads = 32 * 11;
constexpr int kAhead = 3;                             // key tiles before an item's last at which the next one is looked for
constexpr uint32_t kTmemCols = 512, kTmemO = 256;     // S of tile t at 128 t, O at 256 + 128 t
constexpr float kGrow = 8.0f;                         // log2 of how far p may exceed 1

struct Maps {
  CUtensorMap q, k, rope, v;
};

// Bounds of a request.
struct Request {
  int32_t q0, k0, nq, nk;
};

struct Item {
  Request r;
  int32_t first, head;  // first query row in the request, negative after the last item
  int32_t n[2];         // key tiles that each query tile sees any key of
};

struct Smem {
  uint8_t q[2][kQBytes];
  uint8_t ring[kRing][kColBytes];
  uint64_t bars[28];
  alignas(16) uint8_t next[16];          // the answer to a request for another block's place
  Item items[2];
  int32_t before[kThreads];              // pairs of query tiles before each thread's requests
  int32_t warp_pairs[kThreads / 32];
  int32_t total;
  uint32_t tmem;
  int abort;
};
// K, V: by the key tile's parity (V also by half: 2 * parity + half); S, P, O, Q: by query tile
enum { kBarQFull = 0, kBarKFull = 2, kBarKEmpty = 4, kBarVFull = 6, kBarVEmpty = 10, kBarSFull = 12, kBarPFull = 14,
       kBarOFull = 16, kBarVLand = 18, kBarDrain, kBarQEmpty = 20, kBarItemFull = 22, kBarItemEmpty = 24, kBarNext = 26, kBarAsk };

// Where chunk i of the CTA's key tile g lies: K 0 .. 2, V 3, 4.
__device__ __forceinline__ uint32_t ring_slot(uint32_t g, int i) { return (kTileChunks * g + i) % kRing; }

// False where request r's bounds descend or leave the tensors.
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

// Key tiles that query tile t (rows first + 128 t ..) sees any key of.
__device__ __forceinline__ int key_tiles(const csa_latent_prefill_args& A, const Request& R, int first, int t) {
  const int row = first + t * kTile;
  if (row >= R.nq) return 0;
  int64_t seen = R.nk;
  if (A.causal) seen = min(seen, static_cast<int64_t>(min(row + kTile, R.nq)) + R.nk - R.nq);
  return seen <= 0 ? 0 : static_cast<int>((seen + kTile - 1) / kTile);
}

__device__ __forceinline__ int running_sum(int x) {  // over the lanes
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if ((threadIdx.x & 31) >= o) x += up;
  }
  return x;
}

__device__ __forceinline__ int requests_a_thread(const csa_latent_prefill_args& A) { return (A.num_req + kThreads - 1) / kThreads; }

// Sums of the requests' pairs of query tiles, a run of requests a thread.
__device__ void sum_pairs(const csa_latent_prefill_args& A, Smem& S, bool* bad) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, per = requests_a_thread(A);
  const int r0 = min(tid * per, A.num_req), r1 = min(r0 + per, A.num_req);
  int mine = 0;
  for (int r = r0; r < r1; ++r) mine += pairs_of(A, r, bad);
  const int incl = running_sum(mine);
  if (lane == 31) S.warp_pairs[warp] = incl;
  __syncthreads();
  int before = incl - mine, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += S.warp_pairs[w];
    total += S.warp_pairs[w];
  }
  S.before[tid] = before;
  if (tid == 0) S.total = total;
}

// Item of block `at`, by one warp: pairs from the last backwards (the longest first, where requests are causal),
// the heads of a pair next to one another. False past the last.
__device__ bool find_item(const csa_latent_prefill_args& A, Smem& S, uint32_t at, Item* I) {
  const int lane = threadIdx.x & 31, per = requests_a_thread(A);
  const int pair = static_cast<int>(at / A.num_heads), want = S.total - 1 - pair;
  if (want < 0) return false;
  int run = 0;  // the last run of requests that begins at or before the pair
  for (int k = lane; k < kThreads; k += 32)
    if (S.before[k] <= want) run = k;
  run = __reduce_max_sync(0xFFFFFFFFu, run);
  int before = S.before[run];
  bool ignore = false;
  for (int r0 = run * per; r0 < A.num_req; r0 += 32) {
    const int n = r0 + lane < A.num_req ? pairs_of(A, r0 + lane, &ignore) : 0, incl = before + running_sum(n);
    const uint32_t here = __ballot_sync(0xFFFFFFFFu, want < incl);
    if (here) {
      const int who = __ffs(here) - 1;
      const int start = __shfl_sync(0xFFFFFFFFu, incl - n, who);
      if (!request_of(A, r0 + who, &I->r)) return false;
      I->first = (want - start) * 2 * kTile;
      I->head = static_cast<int>(at % A.num_heads);
      for (int t = 0; t < 2; ++t) I->n[t] = key_tiles(A, I->r, I->first, t);
      return true;
    }
    before = __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  return false;
}

// A whole warp's bounded wait, with one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* stop) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, stop));
}

// The same, with a limit for each 2^18 of the key tiles that others may be busy with meanwhile (they take a quarter of it).
__device__ __forceinline__ bool patient_wait(uint32_t bar, uint32_t parity, volatile int* stop, int tiles) {
  for (int k = tiles >> 18; k > 0 && !*stop; --k) {
    volatile int over = 0;
    if (warp_wait(bar, parity, &over)) return true;
  }
  return warp_wait(bar, parity, stop);
}

// Waits for the item at `at`; false after the last one.
__device__ __forceinline__ bool next_item(Smem& S, uint32_t at, int idle) {
  return patient_wait(smem_u32(S.bars) + 8 * (kBarItemFull + (at & 1)), (at >> 1) & 1, &S.abort, idle) && S.items[at & 1].first >= 0;
}

__device__ __forceinline__ void done_with_item(Smem& S, uint32_t at) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(S.bars) + 8 * (kBarItemEmpty + (at & 1)));
}

// Hands out the items: the block's own, then those of blocks that have not started yet, whose places it asks for,
// one at a time, when little of the last item is left to load. What the next item begins with is on its way to L2
// before it is handed out.
__device__ void role_next(const csa_latent_prefill_args& A, const Maps& M, Smem& S) {
  const int lane = threadIdx.x & 31;
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars), next = smem_u32(S.next);
  Item I;
  bool ok = true, more = find_item(A, S, blockIdx.x, &I);
  for (uint32_t at = 0;; ++at) {
    if (!more) I.first = -1;
    ok = ok && (at < 2 || warp_wait(bars + 8 * (kBarItemEmpty + (at & 1)), ((at - 2) >> 1) & 1, stop));
    if (!ok) return;
    if (lane == 0) {
      S.items[at & 1] = I;
      mbar_arrive(bars + 8 * (kBarItemFull + (at & 1)));
    }
    __syncwarp();
    if (!more || !patient_wait(bars + 8 * kBarAsk, at & 1, stop, max(I.n[0], I.n[1]))) return;
    if (lane == 0) {
      csa::mbar_arrive_expect_tx(bars + 8 * kBarNext, 16);
      csa::cancel_next_block(next, bars + 8 * kBarNext);
    }
    __syncwarp();
    if (!warp_wait(bars + 8 * kBarNext, at & 1, stop)) {
      csa::mbar_wait_drain(bars + 8 * kBarNext, at & 1);
      return;
    }
    uint32_t block = 0;
    more = csa::cancelled_block(next, &block) && find_item(A, S, block, &I);
    csa::fence_proxy_async_smem();  // the answer is read before the next one is asked for
    __syncwarp();
    if (more && lane == 0) {
      for (int t = 0; t < 2; ++t)
        for (int c = 0; I.n[t] > 0 && c < kQCols; ++c) csa::tma_prefetch_3d(&M.q, 64 * c, I.head, I.r.q0 + I.first + t * kTile);
      if (max(I.n[0], I.n[1]) > 0) {
        for (int c = 0; c < 2; ++c) csa::tma_prefetch_3d(&M.k, 64 * c, I.head, I.r.k0);
        csa::tma_prefetch_2d(&M.rope, 0, I.r.k0);
        for (int c = 0; c < 2; ++c) csa::tma_prefetch_3d(&M.v, 64 * c, I.head, I.r.k0);
      }
    }
  }
}

__device__ void role_load(const csa_latent_prefill_args& A, const Maps& M, Smem& S) {
  const int lane = threadIdx.x & 31;
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars);
  Item I;
  csa::test_delay();
  bool ok = true, landing = false;  // landing: a copy to kBarVLand is in flight
  // over all items: tiles of Q loaded, key tiles loaded (of V by halves), copies landed
  uint32_t q_done[2] = {0, 0}, k_done = 0, v_done[2] = {0, 0}, landed = 0;
  const uint32_t ring = smem_u32(S.ring[0]);
  uint32_t base = 0;  // key tiles of the items before
  auto freed = [&](int bar, uint32_t g, uint32_t back) {  // what key tile g - back held there has been read
    ok = ok && (g < back || warp_wait(bars + 8 * (bar + ((g - back) & 1)), ((g - back) >> 1) & 1, stop));
    return ok;
  };
  auto load_q = [&](int t) {
    ok = ok && (q_done[t] == 0 || warp_wait(bars + 8 * (kBarQEmpty + t), (q_done[t] - 1) & 1, stop));
    if (!ok) return;
    if (lane == 0) {
      const uint32_t bar = bars + 8 * (kBarQFull + t);
      csa::mbar_arrive_expect_tx(bar, kQBytes);
      for (int c = 0; c < kQCols; ++c)
        csa::tma_tile_3d(smem_u32(S.q[t]) + c * kColBytes, &M.q, 64 * c, I.head, I.r.q0 + I.first + t * kTile, bar);
    }
    ++q_done[t];
  };
  auto load_k = [&](int j) {
    const uint32_t g = base + j;
    if (!freed(kBarKEmpty, g, 2)) return;
    const uint32_t bar = bars + 8 * (kBarKFull + (g & 1));
    const int row = I.r.k0 + j * kTile;
    if (lane == 0) {
      csa::mbar_arrive_expect_tx(bar, kColBytes);
      csa::tma_tile_3d(ring + ring_slot(g, 0) * kColBytes, &M.k, 0, I.head, row, bar);
    }
    k_done = g + 1;
    if (!freed(kBarVEmpty, g, 2)) {
      if (lane == 0) mbar_arrive(bar);  // no more is coming: the first chunk's landing can be waited for
      return;
    }
    if (lane == 0) {
      csa::mbar_arrive_expect_tx(bar, 2 * kColBytes);
      csa::tma_tile_3d(ring + ring_slot(g, 1) * kColBytes, &M.k, 64, I.head, row, bar);
      csa::tma_tile_2d(ring + ring_slot(g, 2) * kColBytes, &M.rope, 0, row, bar);
    }
  };
  auto load_v = [&](int j) {
    const uint32_t g = base + j;
    if (!ok || !freed(kBarKEmpty, g, 1)) return;
    for (int half = 0; half < 2; ++half) {
      // rows of the half that are this request's; the others become zeros before the half is handed over
      const int rows = min(64, I.r.nk - j * kTile - 64 * half);
      const bool whole = rows == 64;
      const uint32_t full = bars + 8 * (kBarVFull + 2 * (g & 1) + half), land = whole ? full : bars + 8 * kBarVLand;
      const uint32_t dst = ring + ring_slot(g, kQCols + half) * kColBytes;
      if (rows > 0 && lane == 0) {
        csa::mbar_arrive_expect_tx(land, kColBytes);
        for (int c = 0; c < kV / 64; ++c)
          csa::tma_tile_3d(dst + c * (kColBytes / 2), &M.v, 64 * c, I.head, I.r.k0 + j * kTile + 64 * half, land);
      }
      if (whole) v_done[half] = g + 1;
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
      v_done[half] = g + 1;
    }
  };
  auto ask = [&] {  // for the next item
    if (lane == 0) mbar_arrive(bars + 8 * kBarAsk);
  };
  for (uint32_t at = 0; ok && next_item(S, at, 0); ++at) {
    I = S.items[at & 1];
    done_with_item(S, at);
    const int n = max(I.n[0], I.n[1]);
    // in the order in which the MMAs give the chunks back
    if (I.n[0] > 0) load_q(0);
    if (n > 0) load_k(0);
    if (I.n[1] > 0) load_q(1);
    if (n <= kAhead) ask();
    if (n > 0) load_v(0);
    if (n > 1) load_k(1);
    for (int j = 1; ok && j < n; ++j) {
      if (j + kAhead == n) ask();
      load_v(j);
      if (ok && j + 1 < n) load_k(j + 1);
    }
    base += n;
  }
  // no copy of this CTA is in flight when it leaves
  if (lane == 0) {
    for (int t = 0; t < 2; ++t)
      if (q_done[t] > 0) csa::mbar_wait_drain(bars + 8 * (kBarQFull + t), (q_done[t] - 1) & 1);
    for (uint32_t g = k_done - min(k_done, 2u); g < k_done; ++g) csa::mbar_wait_drain(bars + 8 * (kBarKFull + (g & 1)), (g >> 1) & 1);
    for (int half = 0; half < 2; ++half)
      for (uint32_t g = v_done[half] - min(v_done[half], 2u); g < v_done[half]; ++g)
        csa::mbar_wait_drain(bars + 8 * (kBarVFull + 2 * (g & 1) + half), (g >> 1) & 1);
    if (landing) csa::mbar_wait_drain(bars + 8 * kBarVLand, landed & 1);
  }
  __syncwarp();
}

// One warp issues all MMAs, S0(j), O1(j - 1), S1(j), O0(j) in turn, with as few waits and commits in
// between as the buffers need: each costs the tensor cores some 80 clocks, and a thread of its own for
// each query tile costs more (their MMAs interleave, and every softmax waits longer for its S).
// O1 of an item's last key tile waits for the next item's S0, if what that needs is there.
__device__ void role_mma(const csa_latent_prefill_args& A, Smem& S) {
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars), tmem = csa::uniform(S.tmem), lead = csa::elect_lane();
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
  // Over the items before: key tiles, and of each query tile those that it sees and its loads of Q.
  uint32_t base = 0, seen_by[2] = {0, 0}, loads[2] = {0, 0};
  // S of tile t over key tile g. `ahead` looks, while these MMAs run, whether what comes after is there.
  auto issue_s = [&](auto tile, uint32_t g, bool last, auto ahead) {
    constexpr int t = decltype(tile)::value;
    if (!ok) return;
#pragma unroll
    for (int c = 0; c < kQCols; ++c) {
      const csa::Desc b = k_ring.at(ring_slot(g, c) * kColBytes);
#pragma unroll
      for (int x = 0; x < 4; ++x)
        csa::mma_f16_ss(lead, tmem + t * kTile, q[t].at(c * kColBytes + 32 * x), b.at(32 * x), idesc_s, c > 0 || x > 0);
      if (c == 1) ahead();
    }
    csa::mma_commit_if(lead, bars + 8 * (kBarSFull + t));
    if (last) csa::mma_commit_if(lead, bars + 8 * (kBarQEmpty + t));
  };
  // O of a query tile over key tile g, its p-th there. frees: V is free afterwards
  struct Value {
    uint32_t g, p;
    bool begin, last, frees;
  };
  auto issue_o = [&](auto tile, const Value& o, auto ahead) {
    constexpr int t = decltype(tile)::value;
    if (!ok) return;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const csa::Desc b = v_ring.at(ring_slot(o.g, kQCols + half) * kColBytes);
#pragma unroll
      for (int x = 0; x < 4; ++x)
        csa::mma_f16_ts(lead, tmem + kTmemO + t * kTile, tmem + t * kTile + 32 * half + 8 * x, b.at(2048 * x), idesc_o,
                        !o.begin || half > 0 || x > 0);
      if (half == 0) ahead();
    }
    if (o.frees) csa::mma_commit_if(lead, bars + 8 * (kBarVEmpty + (o.g & 1)));
    if (o.last) csa::mma_commit_if(lead, bars + 8 * (kBarOFull + t));
  };
  const std::integral_constant<int, 0> t0;
  const std::integral_constant<int, 1> t1;
  const auto nothing = [] {};
  // What O of tile t needs. A first look that finds it costs nothing: MMAs are still queued.
  auto there = [&](int bar, uint32_t parity) { return static_cast<bool>(__all_sync(0xFFFFFFFFu, csa::mbar_test(bars + 8 * bar, parity))); };
  auto look_o = [&](int t, const Value& o) {
    const int seen = there(kBarPFull + t, o.p & 1) + 2 * there(kBarVFull + 2 * (o.g & 1), (o.g >> 1) & 1) +
                     4 * there(kBarVFull + 2 * (o.g & 1) + 1, (o.g >> 1) & 1);
    csa::tc_fence_after();
    return seen;
  };
  auto need_o = [&](int t, const Value& o, int seen) {
    if (!(seen & 2)) need(kBarVFull + 2 * (o.g & 1), (o.g >> 1) & 1);
    if (!(seen & 4)) need(kBarVFull + 2 * (o.g & 1) + 1, (o.g >> 1) & 1);
    if (!(seen & 1)) need(kBarPFull + t, o.p & 1);
  };
  Value late{};  // O1 that is still to be issued
  bool is_late = false;
  auto issue_late = [&](int seen) {
    need_o(1, late, seen);
    issue_o(t1, late, nothing);
    is_late = false;
  };
  for (uint32_t at = 0; ok; ++at) {
    if (is_late && !there(kBarItemFull + (at & 1), (at >> 1) & 1)) issue_late(0);
    if (!ok || !next_item(S, at, 0)) break;
    const Item& I = S.items[at & 1];
    const int n[2] = {static_cast<int>(csa::uniform(I.n[0])), static_cast<int>(csa::uniform(I.n[1]))};
    const int most = max(n[0], n[1]);
    done_with_item(S, at);
    if (most == 0) continue;
    if (is_late && !(there(kBarKFull + (base & 1), (base >> 1) & 1) && (n[0] == 0 || there(kBarQFull, loads[0] & 1)))) issue_late(0);
    need(kBarKFull + (base & 1), (base >> 1) & 1);
    if (n[0] > 0) need(kBarQFull, loads[0] & 1);
    for (int j = 0; ok && j < most; ++j) {
      const uint32_t g = base + j;
      const bool s0 = j < n[0], s1 = j < n[1];
      const Value o0{g, seen_by[0] + j, j == 0, j + 1 == n[0], !s1};
      int seen1 = 0, seen0 = 0;
      bool seen_k = false;
      if (s0)
        issue_s(t0, g, o0.last, [&] {
          if (is_late) seen1 = look_o(1, late);
        });
      if (is_late) issue_late(seen1);
      if (s1) {
        if (j == 0) need(kBarQFull + 1, loads[1] & 1);
        issue_s(t1, g, j + 1 == n[1], [&] {
          if (s0) seen0 = look_o(0, o0);
        });
        late = {g, seen_by[1] + j, j == 0, j + 1 == n[1], true};
        is_late = true;
      }
      csa::mma_commit_if(lead, bars + 8 * (kBarKEmpty + (g & 1)));
      const int k_bar = kBarKFull + ((g + 1) & 1);
      const uint32_t k_parity = ((g + 1) >> 1) & 1;
      if (s0) {
        need_o(0, o0, seen0);
        issue_o(t0, o0, [&] {
          if (j + 1 < most) {
            seen_k = there(k_bar, k_parity);
            csa::tc_fence_after();
          }
        });
      }
      if (j + 1 < most && !seen_k) need(k_bar, k_parity);
    }
    base += most;
    for (int t = 0; t < 2; ++t) {
      seen_by[t] += n[t];
      loads[t] += n[t] > 0;
    }
  }
  if (is_late) issue_late(0);
  csa::mma_commit_if(lead, bars + 8 * kBarDrain);  // nothing of this thread's is in flight when it leaves
  csa::mbar_wait_drain(bars + 8 * kBarDrain, 0);
}

// Softmax and output of query tile t of an item; `n`: its key tiles there, `seen_by` and `items`: its key tiles and its items
// with any so far. What is needed only at the ends is read from shared memory there: registers are short in between.
__device__ __forceinline__ bool softmax_item(const csa_latent_prefill_args& A, Smem& S, uint32_t which, int n, uint32_t seen_by,
                                             uint32_t items) {
  const Item& I = S.items[which & 1];
  const int t = threadIdx.x >> 7, warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars);
  const uint32_t s_at = S.tmem + t * kTile + (static_cast<uint32_t>(32 * warp) << 16);
  int seen;  // keys from tile j on that this row sees
  {
    const int row = I.first + t * kTile + 32 * warp + lane;
    const int64_t past = static_cast<int64_t>(I.r.nk) - I.r.nq;
    seen = A.causal ? static_cast<int>(min(max(row + past + 1, int64_t(0)), static_cast<int64_t>(I.r.nk))) : I.r.nk;
  }
  const float c = A.scale * 1.4426950408889634f;
  float m = -INFINITY, l = 0.f;
  bool ok = true;
  for (int j = 0; j < n; ++j) {
    ok = ok && warp_wait(bars + 8 * (kBarSFull + t), (seen_by + j) & 1, stop);
    if (!ok) break;
    csa::tc_fence_after();
    float s[4][32];
#pragma unroll
    for (int k = 0; k < 4; ++k) csa::tmem_ld32(s_at + 32 * k, reinterpret_cast<uint32_t(&)[32]>(s[k]));
    csa::tmem_wait_ld();
    if (__any_sync(0xFFFFFFFFu, seen < kTile)) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int x = 0; x < 32; ++x)
          if (32 * k + x >= seen) s[k][x] = -INFINITY;
    }
    seen -= kTile;
    float top4[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      top4[k] = s[k][0];
#pragma unroll
      for (int x = 1; x < 32; ++x) top4[k] = fmaxf(top4[k], s[k][x]);
    }
    const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
    const bool up = (top - m) * c > kGrow;  // also when there was nothing; not where there is still nothing
    if (__any_sync(0xFFFFFFFFu, up)) {
      const float keep = up ? csa::ex2((m - top) * c) : 1.f;  // 0 when there was nothing
      if (up) m = top;
      l *= keep;
      if (j > 0) {  // S of this tile is complete, so O of the one before is
#pragma unroll 1
        for (int k = 0; k < kV; k += 32) {
          uint32_t v[32];
          csa::tmem_ld32(s_at + kTmemO + k, v);
          csa::tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * keep);
          csa::tmem_st32(s_at + kTmemO + k, v);
        }
      }
    }
    const float mc = m == -INFINITY ? 0.f : m * c;
    const csa::F2 c2(c, c), mc2(-mc, -mc);
    csa::F2 sum[2];
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
        sum[x / 2 % 2] = csa::add2(sum[x / 2 % 2], csa::F2(s[k][x], s[k][x + 1]));
        // rounded to bf16 here, the tensor cores' operand type; l sums p unrounded
        const __nv_bfloat162 two = __floats2bfloat162_rn(s[k][x], s[k][x + 1]);
        w[x / 2] = *reinterpret_cast<const uint32_t*>(&two);
      }
      csa::tmem_st16(s_at + 16 * k, w);
    }
    float l0, l1;
    csa::add2(sum[0], sum[1]).get(l0, l1);
    l += l0 + l1;
    csa::tmem_wait_st();
    csa::tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * (kBarPFull + t));
  }
  if (n > 0) ok = ok && warp_wait(bars + 8 * (kBarOFull + t), items & 1, stop);
  if (!ok) return false;
  csa::tc_fence_after();
  const float inv = l > 0.f ? 1.f / l : l;  // a NaN stays one
  const int row0 = I.first + t * kTile + 32 * warp, rows = I.r.nq - row0;  // of this warp, and how many are left from there
  const int64_t at0 = static_cast<int64_t>(I.r.q0 + row0) * A.num_heads + I.head;
  done_with_item(S, which);  // before the stores, whose completion an arrival waits for
  float o[4][32] = {};
  if (n > 0) {  // all of a row before the first wait: a load takes 700 clocks beside the MMAs
#pragma unroll
    for (int k = 0; k < 4; ++k) csa::tmem_ld32(s_at + kTmemO + 32 * k, reinterpret_cast<uint32_t(&)[32]>(o[k]));
    csa::tmem_wait_ld();
  }
  if (l == 0.f) {  // the row sees no key; its O is 0 times the values of keys that other rows see, NaN where those are not finite
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int x = 0; x < 32; ++x) o[k][x] = 0.f;
  }
  if (lane >= rows) return true;
  const int64_t at = at0 + static_cast<int64_t>(lane) * A.num_heads;
  if (A.lse) A.lse[at] = l == 0.f ? -INFINITY : (m * c + log2f(l)) * 0.6931471805599453f;
  // Each lane writes its row, 32 bytes (a sector) at a time: staged through Q's place the rows would be whole lines, but
  // that is being loaded with the next item's rows meanwhile, and lines made by exchanges between lanes are no faster.
  uint8_t* out = static_cast<uint8_t*>(A.out) + 2 * kV * at;
  const bool wide = (reinterpret_cast<uintptr_t>(A.out) & 31) == 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t w[16];
#pragma unroll
    for (int x = 0; x < 32; x += 2) {
      const __nv_bfloat162 two = __floats2bfloat162_rn(o[k][x] * inv, o[k][x + 1] * inv);
      w[x / 2] = *reinterpret_cast<const uint32_t*>(&two);
    }
#pragma unroll
    for (int x = 0; x < 16; x += 8) csa::st_global_v8(out + 64 * k + 4 * x, &w[x], wide);
  }
  return true;
}

__device__ void role_softmax(const csa_latent_prefill_args& A, Smem& S) {
  const int t = threadIdx.x >> 7;
  uint32_t seen_by = 0, items = 0;
  int idle = 0;  // key tiles that the other query tile has more than this one
  for (uint32_t at = 0;; ++at) {
    if (!next_item(S, at, idle)) return;
    const int n = S.items[at & 1].n[t];
    idle = max(S.items[at & 1].n[t ^ 1] - n, 0);
    if (!softmax_item(A, S, at, n, seen_by, items)) return;
    seen_by += n;
    items += n > 0;
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ csa_latent_prefill_args A, const __grid_constant__ Maps M) {
  extern __shared__ uint8_t smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const uint32_t bars = smem_u32(S.bars);
  bool bad = false;
  sum_pairs(A, S, &bad);
  if (bad && A.dev_status) atomicOr(A.dev_status, CSA_DEV_LEN_OOB);
  if (threadIdx.x == 0) {
    csa::mbar_init(bars + 8 * kBarVLand, 1);
    csa::mbar_init(bars + 8 * kBarDrain, 1);
    csa::mbar_init(bars + 8 * kBarNext, 1);
    csa::mbar_init(bars + 8 * kBarAsk, 1);
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
      csa::mbar_init(bars + 8 * (kBarQEmpty + k), 1);
      csa::mbar_init(bars + 8 * (kBarItemFull + k), 1);
      csa::mbar_init(bars + 8 * (kBarItemEmpty + k), kSoftmaxWarps + 2);
    }
    csa::mbar_init_fence();
    S.abort = 0;
  }
  __syncthreads();
  if (static_cast<int>(blockIdx.x / A.num_heads) >= S.total) return;
  if (warp == kMmaWarp) {
    csa::tmem_alloc(smem_u32(&S.tmem), kTmemCols);
    csa::tmem_relinquish();
  }
  csa::tc_fence_before();
  __syncthreads();
  csa::tc_fence_after();
  if (warp < kSoftmaxWarps) {
    role_softmax(A, S);
  } else if (warp == kMmaWarp) {
    role_mma(A, S);
    __syncwarp();
  } else if (warp == kLoadWarp) {
    role_load(A, M, S);
  } else {
    role_next(A, M, S);
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
  if (!good_scale(a->scale)) return CSA_ERR_INVALID_ARG;
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
  static Kept ready;  // the kernel's shared memory size is set on each device once
  constexpr size_t smem = sizeof(Smem) + 1024;
  static_assert(smem <= 232448, "shared memory of one CTA");
  if (!ready.get(dev)) {
    if (cudaFuncSetAttribute(prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
      return CSA_ERR_CUDA;
    ready.set(dev, 1);
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
