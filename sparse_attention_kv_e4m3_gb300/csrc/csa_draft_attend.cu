// csa_draft_attend.cu — latent attention of drafted tokens (include/csa_draft.h).
#include <cfloat>
#include <type_traits>

#include "csa_draft.h"
#include "csa_latent_maps.h"
#include "csa_latent_ptx.cuh"
#include "csa_latent_rows.cuh"

namespace csa_latent {
namespace {

using csa::smem_u32;

// The kernel. Per query row i (a draft and a head) and record n that its draft sees, with S = q_i . c_n:
//   p_n = 2^((S_n - m) c), c = scale log2 e,  O = sum p_n c_n[0:512],  l = sum p_n,  out = O / l, lse = scale m + ln l,
// for any reference m a row (the running maximum, moved only when a tile exceeds it by 2^8). The difference comes before the product with c:
// S c - m c is off by a rounding of m c, which from scores of 2^31 on is more than fp32's exponents hold.
//
// All rows of a request read the same records, so they are taken together, 128 rows (drafts times heads, whatever either is) over
// tiles of 128 records, by a pair of CTAs. 128 rows of O, 512 values each, would fill one SM's TMEM and leave S no room; the pair
// has 64 rows each, of S and of O, and the tensor cores of both work on all 128 (cta_group::2, M 128): a CTA's rows lie twice in
// the 128 lanes, with half of the columns each, so O takes 256 columns and S 64 a tile. As operands a CTA has its 64 rows of Q
// (72 KB) and of P (16 KB), the keys of one of the tile's two pages (all their values: half of S's columns) and 256 of the values of
// both (half of O's columns), in a ring of eight slots of 16 KB: keys and values take four each, tile by tile.
//
// Shared memory is what bounds long histories: a tile's MMAs read 245 KB of operands at 128 bytes a clock and its copies write
// 136 KB, 3.0 k clocks, where the tensor cores need 2.18 k (1152 for S, 1024 for O, which they reach with nothing else going on). The
// values of a CTA's own page come in a second time because both CTAs' operands of an MMA lie at the same place. Two requests of 65536 and more records,
// 16 drafts, 64 heads: 330 us, 1.34 PFLOP/s (the absorbed form's own kernel, 64 rows high, reaches 0.68). 32 requests of 8192 to
// 32768, 16 heads, up to 8 drafts, whose records are 783 MB: 172 us, 4.6 TB/s. 4-bit records, 16 requests of 7001 to 16384, up to
// 13 drafts: 308 us, 0.68 PFLOP/s, bound by the conversion to bf16: 10 k warp instructions a tile, at half of the issue rate.
constexpr int kTile = 128;                     // records a tile: two pages, one for each CTA's keys
constexpr int kRows = 64;                      // query rows (draft and head) of a CTA; a unit is the pair's 128
constexpr int kSlots = 8;                      // of the ring: 64 records x 128 values each, two 8 KB columns of 64 values
constexpr int kColBytes = kRows * 128, kSlotBytes = 2 * kColBytes;
constexpr int kSoftmaxWarps = 8, kMmaWarp = kSoftmaxWarps;
// The loaders: of bf16 records one warp, by TMA, and two for queries that TMA does not reach; of 4-bit records four for the keys
// (and the queries) and four for the values, through registers.
template <bool kFp4>
struct Warps {
  static constexpr int kQuery = kMmaWarp + (kFp4 ? 1 : 2), kQueries = kFp4 ? 4 : 2, kValues = kQuery + kQueries;
  static constexpr int kThreads = 32 * (kFp4 ? kValues + 4 : kValues);
  static constexpr int kFills = kFp4 ? 4 : 1;  // arrivals of a CTA that make a slot full
};
constexpr int kLoadWarp = kMmaWarp + 1;
constexpr uint32_t kTmemCols = 512, kTmemS = 256;  // O in columns 0 .. 255, S of even and odd tiles in 256 and 320
constexpr float kGrow = 8.0f;                  // log2 of how far p may exceed 1
constexpr int kMaxPairs = 80;                  // CTA pairs at most: sizes the workspace
constexpr int kParts = 4;                      // cut pieces of a run at most, see Walk
constexpr int kBarRows = 1;                    // named barriers 1, 2: the four warps of rows 0 .. 31, and of 32 .. 63
constexpr int kBarAll = 3;                     // of all softmax warps

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

// ------------------------------------------------------------- work
//
// A unit is 128 query rows (drafts times heads, in that order) of a request; its tiles are the request's. The tiles of
// all units are put in an order and cut into equal runs, one a pair. A request of many tiles is cut into segments of about
// a run's length first, and the order is request, segment, unit, tile: the units of a request read the same segment at
// about the same time, so its records come from HBM once and from L2 for the others. What a run has of one unit's segment is
// a piece; a unit that is not one whole piece leaves parts, which a second kernel joins in their order.

// a / b of numbers that are not negative: most fit in 32 bits, whose division takes a fifth of the time and little code.
__device__ __noinline__ int64_t wide_quotient(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return wide_quotient(a, b);
}

struct Work {
  Request R;
  int32_t units, tiles, segments;
};

__device__ __forceinline__ void set_segments(Work& w, int64_t run) {  // tiles / run, rounded
  w.segments = run >= 2 * static_cast<int64_t>(w.tiles) ? 1 : max(1, static_cast<int32_t>(quotient(2 * static_cast<int64_t>(w.tiles) + run, 2 * run)));
}

// Request r's share; units 0 where it has no rows.
__device__ __forceinline__ Work work_of(const csa_draft_attend_args& A, int r, int64_t run, int32_t* flags) {
  Work w = {{0, 0, 0, 0}, 0, 1, 1};
  if (!request_of(A, r, &w.R, flags) || w.R.drafts == 0) return w;
  w.units = static_cast<int32_t>((static_cast<int64_t>(w.R.drafts) * A.num_heads + 2 * kRows - 1) / (2 * kRows));
  w.tiles = (w.R.total + kTile - 1) / kTile;
  set_segments(w, run);
  return w;
}

__device__ __forceinline__ int64_t run_start(int64_t total, int p, int pairs) { return quotient(total * p, pairs); }

__device__ __forceinline__ int32_t segment_start(const Work& w, int s) { return static_cast<int32_t>(quotient(static_cast<int64_t>(w.tiles) * s, w.segments)); }

struct Kernel {
  csa_draft_attend_args A;
  struct Part* parts_of;  // [pairs][kParts]
  float* parts;
  int32_t pairs;
  int32_t even;  // the rows of q (draft and head) are q_head_stride apart throughout
};

// A cut piece: where its rows begin among all rows (draft and head), how many there are (0 where there is no piece), and
// whether it has the unit's first tile.
struct Part {
  int64_t first;
  int32_t rows, begins;
};
constexpr size_t kPartFloats = 2 * kRows * (static_cast<size_t>(kDim) + 2);  // O, then m and l of its rows

// Walks a run piece by piece. A segment has at least 3/4 of a run's tiles (segments = tiles / run rounded, 2 at least), so a run
// meets at most two whole ones, or one and the ends of two others: kParts are enough for its cut pieces. (A unit of a
// request with one segment is cut at a run's ends only.)
struct Walk {
  Work w;
  int64_t left, run;
  int32_t request, segment, unit, first, n;  // the piece: its first tile in the request, its tiles
  bool cut;
  // The run of `tiles` tiles from tile x of request r's, whose work is `of`.
  __device__ __forceinline__ void start(const Work& of, int32_t r, int64_t x, int64_t tiles, int64_t run_tiles) {
    left = tiles;
    run = run_tiles;
    request = r;
    w = of;
    set_segments(w, run);
    const int32_t t = static_cast<int32_t>(quotient(x, w.units));
    segment = static_cast<int32_t>(quotient((static_cast<int64_t>(t) + 1) * w.segments - 1, w.tiles));
    const int32_t s0 = segment_start(w, segment), len = segment_start(w, segment + 1) - s0;
    const int64_t y = x - static_cast<int64_t>(s0) * w.units;
    unit = static_cast<int32_t>(quotient(y, len));
    size(s0, len, static_cast<int32_t>(y - static_cast<int64_t>(unit) * len));
  }
  __device__ __forceinline__ void size(int32_t s0, int32_t len, int32_t off) {
    first = s0 + off;
    n = static_cast<int32_t>(min(left, static_cast<int64_t>(len - off)));
    cut = n < w.tiles;
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next(const csa_draft_attend_args& A) {
    left -= n;
    if (left <= 0) return;
    int32_t s0 = segment_start(w, segment), len = segment_start(w, segment + 1) - s0;
    if (first + n == s0 + len && ++unit == w.units) {
      unit = 0;
      if (++segment == w.segments) {
        segment = 0;
        int32_t ignore = 0;
        do w = work_of(A, ++request, run, &ignore);
        while (w.units == 0);
      }
      s0 = segment_start(w, segment);
      len = segment_start(w, segment + 1) - s0;
    }
    size(s0, len, 0);
  }
  __device__ __forceinline__ int64_t first_row(const csa_draft_attend_args& A) const {  // of the unit, among all rows
    return static_cast<int64_t>(w.R.row0) * A.num_heads + static_cast<int64_t>(unit) * 2 * kRows;
  }
  __device__ __forceinline__ int32_t rows(const csa_draft_attend_args& A) const {
    return static_cast<int32_t>(min(static_cast<int64_t>(2 * kRows), static_cast<int64_t>(w.R.drafts) * A.num_heads - static_cast<int64_t>(unit) * 2 * kRows));
  }
};

template <bool kFp4, int kRope>
struct Smem {
  using W = Warps<kFp4>;
  static constexpr int kCols = (kDim + kRope) / 64;
  uint8_t q[kCols * kColBytes];
  uint8_t ring[kSlots][kSlotBytes];
  uint8_t rope[kRope ? kColBytes : 16];
  alignas(1024) uint8_t p[2 * kColBytes];  // 64 rows x 128 keys, two columns of 64 keys
  uint64_t bars[32];
  float quarter[4][kRows];             // maxima, or sums, of the quarters of a row's keys
  uint32_t fills[3];                   // by TMA: slots and rope columns that this CTA filled, and Q
  int64_t scan[W::kThreads / 32];
  Walk walk;  // at the run's first piece
  Walk at;    // at the softmax warps' piece: theirs together, to spare their registers
  uint32_t theirs[4];                  // the other CTA's fills, and whether a wait of its ran out
  uint32_t tmem;
  int abort;
};
enum { kBarFull = 0, kBarEmpty = kSlots, kBarRopeFull = 2 * kSlots, kBarRopeEmpty, kBarSFull, kBarSEmpty = kBarSFull + 2,
       kBarPFull = kBarSEmpty + 2, kBarODone, kBarQFull, kBarQEmpty, kBarOEmpty, kBarLand, kBarDrain,
       kBarFirstKeys, kBarLastValues, kBars };
static_assert(kBars <= 32, "barriers");

// The run of this pair: the requests' tiles are summed by the block.
template <bool kFp4, int kRope>
__device__ void make_plan(const Kernel& K, Smem<kFp4, kRope>& S, int32_t* flags) {
  constexpr int kThreads = Warps<kFp4>::kThreads;
  const csa_draft_attend_args& A = K.A;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, pair = blockIdx.x >> 1;
  const int per = (A.num_req + kThreads - 1) / kThreads, r0 = min(tid * per, A.num_req), r1 = min(r0 + per, A.num_req);
  constexpr int64_t kNoSegments = INT64_MAX / 4;
  int64_t mine = 0;
  Work w;
  for (int r = r0; r < r1; ++r) {
    w = work_of(A, r, kNoSegments, flags);
    mine += static_cast<int64_t>(w.units) * w.tiles;
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) S.scan[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += S.scan[w];
    total += S.scan[w];
  }
  const int64_t at = run_start(total, pair, K.pairs), end = run_start(total, pair + 1, K.pairs);
  if (tid == 0 && at == end) S.walk.left = 0;
  if (at < end && at >= before && at < before + mine) {
    int32_t ignore = 0;
    for (int r = r0; r < r1; ++r) {
      if (per > 1) w = work_of(A, r, kNoSegments, &ignore);
      const int64_t all = static_cast<int64_t>(w.units) * w.tiles;
      if (at < before + all) {
        S.walk.start(w, r, at - before, end - at, max(quotient(total, K.pairs), int64_t(1)));
        break;
      }
      before += all;
    }
  }
  __syncthreads();
}

// ------------------------------------------------------------- the pair's barriers
//
// Operands that the MMAs of a pair read lie in both CTAs; what makes them full is counted at the first one's barriers,
// whose MMA warp issues for both. What gives them back is told to both by the MMAs' commits.

// What they order are a CTA's own writes before its own tensor core's reads (a fence to the async proxy, then the arrival, then the
// MMA that the other CTA issues for both), so the arrivals and waits need no memory order between the CTAs: with cluster
// scope each cost several hundred clocks, and 16 drafts of two long histories took 1165 us instead of 359.

// A whole warp's bounded wait, with one answer for all lanes. A first look that finds the phase complete costs the MMA warp
// nothing, where a wait that may park costs it 130 clocks, of which the MMAs already issued cover 100.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* stop) {
  return __all_sync(0xFFFFFFFFu, csa::mbar_test(bar, parity)) || __all_sync(0xFFFFFFFFu, csa::mbar_wait(bar, parity, stop));
}

// The same, with a limit for each 2^18 tiles that others may be busy with meanwhile (they take about half of it).
__device__ __forceinline__ bool patient_wait(uint32_t bar, uint32_t parity, volatile int* stop, int tiles) {
  for (int k = tiles >> 18; k > 0 && !*stop; --k) {
    volatile int over = 0;
    if (warp_wait(bar, parity, &over)) return true;
  }
  return warp_wait(bar, parity, stop);
}

__device__ __forceinline__ void arrive_at(uint32_t remote) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}

__device__ __forceinline__ void arrive_expect_at(uint32_t remote, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(remote), "r"(bytes) : "memory");
}

// A tile to this CTA's shared memory that completes at either CTA's barrier.
__device__ __forceinline__ void tma_pair_4d(uint32_t dst, const void* map, int32_t x, int32_t y, int32_t z, int32_t w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_pair_2d(uint32_t dst, const void* map, int32_t x, int32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// D[tmem] (+)= A[smem] B[smem]^T over the pair: 128 rows of A, 64 in each CTA, and N columns, half of B in each. A CTA's D
// are its 64 rows: the first CTA's columns in lanes 0 .. 63, the second one's in lanes 64 .. 127.
__device__ __forceinline__ void mma_pair(uint32_t lead, uint32_t d, csa::Desc a, csa::Desc b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.u32 q, %7, 0;\n\tsetp.ne.u32 p, %6, 0;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
      "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(lead)
      : "memory");
}

// Arrives at the barrier in both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n\t}" ::"r"(bar),
      "r"(lead), "h"(static_cast<uint16_t>(3))
      : "memory");
}

__device__ __forceinline__ void st_peer_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

struct Maps {  // [page][column of 64 values][record][value]: boxes of a page's two columns, and of one
  CUtensorMap two, one;
  CUtensorMap q;  // [row (draft and head)][value], boxes of a column of 64 rows
};

// ------------------------------------------------------------- roles

// Makes 0 of what is not finite in the 8 values at `addr` of shared memory.
__device__ __forceinline__ void keep_finite(uint32_t addr) {
  const uint4 v = csa::ld_shared_v4(addr);
  if (!(nonfinite_bf16x2(v.x) | nonfinite_bf16x2(v.y) | nonfinite_bf16x2(v.z) | nonfinite_bf16x2(v.w))) return;
  auto clean = [](uint32_t w) { return ((w & 0x7F80u) == 0x7F80u ? 0u : w & 0xFFFFu) | ((w & 0x7F800000u) == 0x7F800000u ? 0u : w & 0xFFFF0000u); };
  csa::st_shared_v4(addr, clean(v.x), clean(v.y), clean(v.z), clean(v.w));
}

// The records, through the ring in the order in which the MMAs take them: the keys of tile 0, then keys of tile i + 1
// and values of tile i. A CTA loads its page's 64 records whole as keys, and its 256 values' columns of both pages.
// The values of a page with drafts or with an end in it are looked at before they are handed over: rows past the end
// become 0, and so do values of drafts that are not finite (0 x NaN is not 0; a row that sees the draft has the NaN of its score).
template <int kRope>
__device__ void role_load(const Kernel& K, const Maps& M, Smem<false, kRope>& S, uint32_t rank, int32_t* flags) {
  const csa_draft_attend_args& A = K.A;
  const int lane = threadIdx.x & 31;
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars), lead_bars = csa::peer_smem(bars, 0), ring = smem_u32(S.ring[0]);
  csa::test_delay();
  uint32_t q = 0, ropes = 0, landed = 0;  // slots filled, rope columns filled, landings
  bool ok = true;
  auto free_slot = [&](uint32_t k) { return ok = ok && warp_wait(bars + 8 * (kBarEmpty + k % kSlots), (k / kSlots & 1) ^ 1, stop); };
  for (Walk W = S.walk; ok && W.more(); W.next(A)) {
    const int32_t* table = A.page_table + static_cast<int64_t>(W.request) * A.pt_stride;
    auto page_of = [&](int32_t p) {  // of the request's page p, or -1
      if (p * kPageRecs >= W.w.R.total) return -1;
      const int32_t page = __ldg(table + p);
      if (page >= 0 && page < A.cache.num_pages) return page;
      *flags |= CSA_DEV_PAGE_OOB;
      return -1;
    };
    auto keys = [&](int32_t tile) {
      const int32_t page = page_of(2 * tile + static_cast<int32_t>(rank));
      if (kRope != 0) {
        ok = ok && warp_wait(bars + 8 * kBarRopeEmpty, (ropes & 1) ^ 1, stop);
        if (!ok) return;
        ++ropes;
        if (lane == 0) {
          const uint32_t full = lead_bars + 8 * kBarRopeFull;
          if (page >= 0) {
            arrive_expect_at(full, kColBytes);
            tma_pair_4d(smem_u32(S.rope), &M.one, 0, 0, kDim / 64, page, full);
          } else {
            arrive_at(full);
          }
        }
      }
#pragma unroll 1
      for (int d = 0; d < kDim / 128; ++d) {
        if (!free_slot(q)) return;
        if (lane == 0) {
          const uint32_t full = lead_bars + 8 * (kBarFull + q % kSlots);
          if (page >= 0) {
            arrive_expect_at(full, kSlotBytes);
            tma_pair_4d(ring + q % kSlots * kSlotBytes, &M.two, 0, 0, 2 * d, page, full);
          } else {
            arrive_at(full);
          }
        }
        ++q;
      }
    };
    auto values = [&](int32_t tile) {
      for (int half = 0; half < 2; ++half) {
        const int32_t p = 2 * tile + half, page = page_of(p), p0 = p * kPageRecs;
        const int rows = page < 0 ? 0 : min(kPageRecs, W.w.R.total - p0);
        const bool plain = rows == kPageRecs && p0 + kPageRecs <= W.w.R.base;
        const uint32_t q0 = q;
        if (plain) {
          for (int b = 0; b < 2; ++b, ++q) {
            if (!free_slot(q)) return;
            if (lane == 0) {
              const uint32_t full = lead_bars + 8 * (kBarFull + q % kSlots);
              arrive_expect_at(full, kSlotBytes);
              tma_pair_4d(ring + q % kSlots * kSlotBytes, &M.two, 0, 0, 4 * static_cast<int>(rank) + 2 * b, page, full);
            }
          }
          continue;
        }
        if (!free_slot(q) || !free_slot(q + 1)) return;
        if (lane == 0 && rows > 0) {
          const uint32_t land = bars + 8 * kBarLand;
          csa::mbar_arrive_expect_tx(land, 2 * kSlotBytes);
          for (int b = 0; b < 2; ++b) csa::tma_tile_4d(ring + (q0 + b) % kSlots * kSlotBytes, &M.two, 0, 0, 4 * static_cast<int>(rank) + 2 * b, page, land);
        }
        q += 2;
        if (rows > 0) {
          if (!warp_wait(bars + 8 * kBarLand, landed & 1, stop)) {
            ok = false;
            csa::mbar_wait_drain(bars + 8 * kBarLand, landed & 1);  // no copy of this CTA is in flight when it leaves
            return;
          }
          ++landed;
        }
        for (int b = 0; b < 2; ++b) {
          const uint32_t slot = ring + (q0 + b) % kSlots * kSlotBytes;
          const int drafts = min(rows, max(0, W.w.R.base - p0));  // the first draft's row
          for (int at = 8 * drafts + lane; at < 2 * 8 * kPageRecs; at += 32) {  // 16 bytes each, of 2 columns of 64 rows
            const int row = at / 8 % kPageRecs;
            if (row < drafts) continue;
            const uint32_t addr = slot + 16 * at;
            if (row < rows) keep_finite(addr);
            else csa::st_shared_v4(addr, 0, 0, 0, 0);
          }
        }
        csa::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
          for (int b = 0; b < 2; ++b) arrive_at(lead_bars + 8 * (kBarFull + (q0 + b) % kSlots));
      }
    };
    keys(W.first);
    for (int i = 0; ok && i < W.n; ++i) {
      if (i + 1 < W.n) keys(W.first + i + 1);
      if (ok) values(W.first + i);
    }
  }
  __syncwarp();
  // for the drain, should a wait have run out: how often each slot was filled
  if (lane == 0) {
    S.fills[0] = q;
    S.fills[1] = ropes;
  }
}

// Q of a run's piece-th piece (`tiles_before`: how much of the one before may still be to come): row i of this CTA's 64 is row
// 64 rank + i of the unit. Past the unit's last lie zeros, or rows that nothing comes of. By TMA where all rows lie evenly, else by the
// threads of the warps that call it.
template <bool kFp4, int kRope>
__device__ bool load_query(const Kernel& K, const Maps& M, Smem<kFp4, kRope>& S, const Walk& W, uint32_t piece, uint32_t rank, int tiles_before) {
  constexpr int kCols = Smem<kFp4, kRope>::kCols;
  const csa_draft_attend_args& A = K.A;
  const int t = threadIdx.x - 32 * Warps<kFp4>::kQuery, lane = t & 31;
  const uint32_t bars = smem_u32(S.bars), full = csa::peer_smem(bars, 0) + 8 * kBarQFull;
  if (K.even && t >= 32) return true;
  if (!patient_wait(bars + 8 * kBarQEmpty, (piece & 1) ^ 1, &S.abort, tiles_before)) return false;
  if (K.even) {
    if (t == 0) {
      arrive_expect_at(full, sizeof(S.q));
#pragma unroll 1
      for (int c = 0; c < kCols; ++c)
        tma_pair_2d(smem_u32(S.q) + c * kColBytes, &M.q, 64 * c, static_cast<int32_t>(W.first_row(A)) + kRows * static_cast<int32_t>(rank), full);
      S.fills[2] = piece + 1;
    }
    __syncwarp();
    return true;
  }
  const int64_t first = static_cast<int64_t>(W.unit) * 2 * kRows + kRows * rank, draft = quotient(first, A.num_heads);  // of the request's rows
  const int head = static_cast<int>(first - draft * A.num_heads), rows = W.rows(A) - kRows * static_cast<int>(rank);
#pragma unroll 2
  for (int i = t >> 3; i < kRows; i += 4 * Warps<kFp4>::kQueries) {
    const uint32_t x = head + i, j = x / static_cast<uint32_t>(A.num_heads), h = x - j * A.num_heads;
    const uint8_t* q = static_cast<const uint8_t*>(A.q) + 16 * (t & 7);
    if (i < rows) q += 2 * ((W.w.R.row0 + draft + j) * A.q_row_stride + h * A.q_head_stride);
#pragma unroll
    for (int c = 0; c < kCols; ++c) csa::cp_async16(smem_u32(S.q) + c * kColBytes + i * 128 + (((t & 7) ^ (i & 7)) << 4), i < rows ? q + 128 * c : A.q, i < rows);
  }
  csa::cp_async_wait_all();
  csa::fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) arrive_at(full);
  return true;
}

// The queries of bf16 records' kernels, whose records come by another warp.
template <int kRope>
__device__ void role_query(const Kernel& K, const Maps& M, Smem<false, kRope>& S, uint32_t rank) {
  uint32_t piece = 0;
  int before = 0;  // tiles of the piece before
  for (Walk W = S.walk; W.more(); before = W.n, W.next(K.A), ++piece)
    if (!load_query<false, kRope>(K, M, S, W, piece, rank, before)) return;
}

// 4-bit records, four lanes a record. A slot is 128 values of 64 records, four blocks of 32 each: two blocks a thread (16 code
// bytes and a scale byte become 64 bytes of bf16, exactly). The codes of the next two slots are on their way while one is
// converted (of four, their registers and the code for them made it slower), and the page of the tile after the next one is
// on its way to L2. Keys and values have four warps each, so that neither waits for the other's turn in the ring; the values of the
// CTA's own page are read and converted a second time, because there is no room to keep them.
struct Codes {
  uint4 code[2];
  uint32_t scale[2];
};

// To the slot at `slot`, as records t / 4 and t / 4 + 32, block t % 4.
__device__ __forceinline__ void store_codes(const Codes& x, uint32_t slot, int t) {
  const int s = t & 3;
  const bool swap = s >= 2;  // lanes 2, 3 of a record store their words in another order: no two on one bank
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = (t >> 2) + 32 * k;
    const uint32_t sb = x.scale[k], bits = sb == 0 ? 0x0040u : (sb == 255 ? 0x7FC0u : sb << 7), two = bits | (bits << 16);
    const __nv_bfloat162 s2 = *reinterpret_cast<const __nv_bfloat162*>(&two);
    const uint4 c = x.code[k];
    const uint32_t word[4] = {swap ? c.z : c.x, swap ? c.w : c.y, swap ? c.x : c.z, swap ? c.y : c.w};
    const uint32_t row = slot + (s >> 1) * kColBytes + r * 128;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t v[4];
      mxfp4_four(word[j], s2, &v[0], &v[1]);
      mxfp4_four(word[j] >> 16, s2, &v[2], &v[3]);
      const int chunk = 4 * (s & 1) + (swap ? j ^ 2 : j);
      csa::st_shared_v4(row + ((chunk ^ (r & 7)) << 4), v[0], v[1], v[2], v[3]);
    }
  }
}

// What a thread has stored of a tile's values (four slots, two of each page), in records `first` and after, without what is not finite: a
// scale byte of 255 is NaN, and of 253 and 254 (2^126, 2^127; the writers' end at 252) the larger codes are infinite in bf16. Once a
// tile that has drafts, out of the loop's way (4-bit trees 311 us; with a look at each slot 340, with a test of the codes 370).
__device__ __noinline__ void keep_finite_codes(uint32_t slots, int first, int t) {
#pragma unroll 1
  for (int i = 0; i < 32; ++i) {
    const int half = i >> 4, r = (t >> 2) + 32 * (i >> 2 & 1), chunk = 4 * (t & 1) + (i & 3);
    if (kPageRecs * half + r >= first) keep_finite(slots + (i >> 3) * kSlotBytes + (t >> 1 & 1) * kColBytes + r * 128 + ((chunk ^ (r & 7)) << 4));
  }
}

// A page of a piece, as the loaders of 4-bit records see it.
struct PageView {
  const uint8_t* records;  // null: none of it is there
  int32_t rows;            // of its records, that there are
};

__device__ __forceinline__ PageView page_view(const csa_draft_attend_args& A, const Request& R, int32_t p, int32_t page, int32_t* flags) {
  if (p * kPageRecs >= R.total) return {nullptr, 0};
  if (page < 0 || page >= A.cache.num_pages) {
    *flags |= CSA_DEV_PAGE_OOB;
    return {nullptr, 0};
  }
  return {A.cache.pages + page * A.cache.page_stride_bytes, min(kPageRecs, R.total - p * kPageRecs)};
}

template <int kRope>
__device__ __forceinline__ void fetch_codes(Codes& x, const PageView& P, int block, int t) {
  constexpr int kRec = record_bytes(true, kRope);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = (t >> 2) + 32 * k;
    const uint8_t* rec = P.records + r * kRec;
    const bool there = r < P.rows;
    x.code[k] = there ? __ldg(reinterpret_cast<const uint4*>(rec) + block) : make_uint4(0, 0, 0, 0);
    x.scale[k] = there ? __ldg(rec + kCodeBytes + block) : 0u;
  }
}

// Hands over four slots, whose barriers begin at `full`, and what else there is a barrier for. All at once: the fence to the
// tensor cores' proxy holds a warp up longer than the slots' coming one by one gains (4-bit trees: a fence a slot 341 us, for
// two 317, for four 304).
__device__ __forceinline__ void handed_over(uint32_t full, uint32_t other) {
  csa::fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) != 0) return;
  for (int k = 0; k < 4; ++k) arrive_at(full + 8 * k);
  if (other) arrive_at(other);
}

template <int kRope>
__device__ void role_keys_fp4(const Kernel& K, const Maps& M, Smem<true, kRope>& S, uint32_t rank, int32_t* flags) {
  const csa_draft_attend_args& A = K.A;
  const int t = threadIdx.x - 32 * Warps<true>::kQuery, s = t & 3;
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars), lead_bars = csa::peer_smem(bars, 0), ring = smem_u32(S.ring[0]);
  csa::test_delay();
  uint32_t q = 0, ropes = 0, piece = 0;  // q: slots of the pieces before
  bool ok = true;
  for (Walk W = S.walk; ok && W.more(); q += 8 * W.n, W.next(A), ++piece) {
    const int32_t* table = A.page_table + static_cast<int64_t>(W.request) * A.pt_stride;
    const Request& R = W.w.R;
    const int32_t past = W.first + W.n;
    auto page_at = [&](int32_t tile) { return tile < past && (2 * tile + static_cast<int>(rank)) * kPageRecs < R.total ? __ldg(table + 2 * tile + rank) : -1; };
    auto view = [&](int32_t tile, int32_t page) { return tile < past ? page_view(A, R, 2 * tile + rank, page, flags) : PageView{nullptr, 0}; };
    int32_t page = page_at(W.first + 1);
    PageView now = view(W.first, page_at(W.first)), next;
    Codes x[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) fetch_codes<kRope>(x[c], now, 4 * c + s, t);
    ok = load_query<true, kRope>(K, M, S, W, piece, rank, 0);
    for (int i = 0; ok && i < W.n; ++i) {
      next = view(W.first + i + 1, page);
      page = page_at(W.first + i + 2);
      if (kRope != 0) {  // the rope values go straight to shared memory, while the first codes are converted
        if (!warp_wait(bars + 8 * kBarRopeEmpty, (ropes & 1) ^ 1, stop)) return;
        ++ropes;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = (t >> 3) + 16 * k;
          csa::cp_async16(smem_u32(S.rope) + r * 128 + (((t & 7) ^ (r & 7)) << 4),
                          r < now.rows ? now.records + r * record_bytes(true, kRope) + kCodeBytes + kScaleBytes + 16 * (t & 7) : A.cache.pages, r < now.rows);
        }
      }
      const uint32_t at = i == 0 ? q : q + 8 * i - 4;
      if (i == 0 && piece > 0) ok = warp_wait(bars + 8 * kBarLastValues, (piece - 1) & 1, stop);
#pragma unroll 1
      for (int c0 = 0; c0 < 4; c0 += 2) {
        const PageView from = c0 == 0 ? now : next;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t slot = (at + c0 + c) % kSlots;
          ok = ok && warp_wait(bars + 8 * (kBarEmpty + slot), (at / kSlots & 1) ^ 1, stop);
          if (ok) store_codes(x[c], ring + slot * kSlotBytes, t);
          if (c == 1 && c0 == 2) {
            if (kRope != 0) csa::cp_async_wait_all();
            if (ok) handed_over(lead_bars + 8 * (kBarFull + slot - 3), kRope != 0 ? lead_bars + 8 * kBarRopeFull : 0);
            if (ok && i == 0 && (t & 31) == 0) csa::mbar_arrive(bars + 8 * kBarFirstKeys);
          }
          fetch_codes<kRope>(x[c], from, 4 * (c0 == 0 ? c + 2 : c) + s, t);
        }
      }
      now = next;
      if (t == 0 && page >= 0 && page < A.cache.num_pages)
        csa::bulk_prefetch_l2(A.cache.pages + page * A.cache.page_stride_bytes, kPageRecs * record_bytes(true, kRope));
    }
  }
}

// What becomes of rows past the end, and of drafts' values that are not finite, is as in role_load.
template <int kRope>
__device__ void role_values_fp4(const Kernel& K, Smem<true, kRope>& S, uint32_t rank, int32_t* flags) {
  const csa_draft_attend_args& A = K.A;
  const int t = threadIdx.x - 32 * Warps<true>::kValues, s = t & 3;
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars), lead_bars = csa::peer_smem(bars, 0), ring = smem_u32(S.ring[0]);
  csa::test_delay();
  uint32_t q = 0, piece = 0;
  for (Walk W = S.walk; W.more(); q += 8 * W.n, W.next(A), ++piece) {
    const int32_t* table = A.page_table + static_cast<int64_t>(W.request) * A.pt_stride;
    const Request& R = W.w.R;
    const int32_t past = W.first + W.n;
    auto page_at = [&](int32_t tile, int h) { return tile < past && (2 * tile + h) * kPageRecs < R.total ? __ldg(table + 2 * tile + h) : -1; };
    auto view = [&](int32_t tile, int h, int32_t page) { return tile < past ? page_view(A, R, 2 * tile + h, page, flags) : PageView{nullptr, 0}; };
    auto fetch = [&](Codes& x, const PageView& P, int b) { fetch_codes<kRope>(x, P, 8 * rank + 4 * b + s, t); };
    PageView other = view(W.first, 1, page_at(W.first, 1));  // the page whose turn is next but one
    int32_t page = page_at(W.first + 1, 0);                  // of the turn after it
    Codes x[2];
    {
      const PageView first = view(W.first, 0, page_at(W.first, 0));
      fetch(x[0], first, 0);
      fetch(x[1], first, 1);
    }
    if (!warp_wait(bars + 8 * kBarFirstKeys, piece & 1, stop)) return;
    for (int i = 0; i < W.n; ++i) {
      const uint32_t at = i + 1 < W.n ? q + 8 * i + 8 : q + 8 * W.n - 4;
      const int32_t drafts = R.base - (W.first + i) * kTile;  // the tile's first draft
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint32_t slot = (at + 2 * h + b) % kSlots;
          if (!warp_wait(bars + 8 * (kBarEmpty + slot), (at / kSlots & 1) ^ 1, stop)) return;
          store_codes(x[b], ring + slot * kSlotBytes, t);
          if (b == 1 && h == 1) {
            if (drafts < kTile) keep_finite_codes(ring + (slot - 3) * kSlotBytes, drafts, t);
            handed_over(lead_bars + 8 * (kBarFull + slot - 3), 0);
          }
          fetch(x[b], other, b);
        }
        other = view(W.first + i + 1, h, page);
        page = page_at(W.first + i + 1 + h, h ^ 1);
      }
    }
    if ((t & 31) == 0) csa::mbar_arrive(bars + 8 * kBarLastValues);
    __syncwarp();
  }
}

// One warp of the first CTA issues the pair's MMAs: S(0), then S(i + 1) and O(i) in turn.
template <bool kFp4, int kRope>
__device__ void role_mma(const Kernel& K, Smem<kFp4, kRope>& S) {
  const csa_draft_attend_args& A = K.A;
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars), tmem = csa::uniform(S.tmem), lead = csa::elect_lane();
  constexpr uint32_t idesc_s = csa::idesc_bf16_f32(2 * kRows, kTile), idesc_o = csa::idesc_bf16_f32(2 * kRows, 256) | csa::kIdescBMnMajor;
  const csa::Desc q_desc(csa::sdesc_kmajor_sw128(smem_u32(S.q))), p_desc(csa::sdesc_kmajor_sw128(smem_u32(S.p))),
      k_ring(csa::sdesc_kmajor_sw128(smem_u32(S.ring[0]))), k_rope(csa::sdesc_kmajor_sw128(smem_u32(S.rope))),
      v_ring(csa::sdesc_mn_sw128_b16(smem_u32(S.ring[0]), kColBytes));
  uint32_t q = 0, ropes = 0, g = 0, done = 0, piece = 0;  // slots and rope columns taken; tiles of which S, O was issued
  bool ok = true;
  auto need = [&](int bar, uint32_t parity) {
    ok = ok && warp_wait(bars + 8 * bar, parity, stop);
    csa::tc_fence_after();
    return ok;
  };
  auto scores = [&](bool last) {
    if (!need(kBarSEmpty + (g & 1), (g >> 1 & 1) ^ 1)) return;
    const uint32_t d = tmem + kTmemS + (g & 1) * (kTile / 2);
    if (kRope != 0) {
      if (!need(kBarRopeFull, ropes & 1)) return;
      ++ropes;
#pragma unroll
      for (int x = 0; x < 4; ++x) mma_pair(lead, d, q_desc.at(kDim / 64 * kColBytes + 32 * x), k_rope.at(32 * x), idesc_s, x > 0);
      commit_pair(lead, bars + 8 * kBarRopeEmpty);
    }
    const uint32_t at_slot = q % kSlots, parity = q / kSlots & 1;  // four slots at a time: 0 .. 3 or 4 .. 7
    const csa::Desc k = k_ring.at(at_slot * kSlotBytes);
#pragma unroll
    for (int c = 0; c < kDim / 128; ++c) {
      if (!need(kBarFull + at_slot + c, parity)) return;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const uint32_t at = c * kSlotBytes + x / 4 * kColBytes + x % 4 * 32;
        mma_pair(lead, d, q_desc.at(at), k.at(at), idesc_s, kRope != 0 || c > 0 || x > 0);
      }
      commit_pair(lead, bars + 8 * (kBarEmpty + at_slot + c));
    }
    q += kDim / 128;
    commit_pair(lead, bars + 8 * (kBarSFull + (g & 1)));
    if (last) commit_pair(lead, bars + 8 * kBarQEmpty);
    ++g;
  };
  auto outputs = [&](bool begin) {
    if (!need(kBarPFull, done & 1)) return;
    const uint32_t at_slot = q % kSlots, parity = q / kSlots & 1;
    const csa::Desc v = v_ring.at(at_slot * kSlotBytes);
#pragma unroll
    for (int c = 0; c < 4; ++c) {  // page c / 2, columns 128 (c % 2) .. of the CTAs' values
      if (!need(kBarFull + at_slot + c, parity)) return;
#pragma unroll
      for (int x = 0; x < 4; ++x)
        mma_pair(lead, tmem + 128 * (c & 1), p_desc.at(c / 2 * kColBytes + 32 * x), v.at(c * kSlotBytes + 2048 * x), idesc_o, !begin || c > 1 || x > 0);
      commit_pair(lead, bars + 8 * (kBarEmpty + at_slot + c));
    }
    q += 4;
    commit_pair(lead, bars + 8 * kBarODone);
    ++done;
  };
  for (Walk W = S.walk; ok && W.more(); W.next(A), ++piece) {
    const int n = static_cast<int>(csa::uniform(W.n));
    if (!need(kBarQFull, piece & 1)) break;
    scores(n == 1);
    for (int i = 0; ok && i < n; ++i) {
      if (i + 1 < n) scores(i + 2 == n);
      if (ok && i == 0) need(kBarOEmpty, (piece & 1) ^ 1);
      if (ok) outputs(i == 0);
    }
  }
  commit_pair(lead, bars + 8 * kBarDrain);  // nothing of the pair's MMAs is in flight when it leaves
  csa::mbar_wait_drain(bars + 8 * kBarDrain, 0);
  __syncwarp();
}

// Which of 64 records from position p0 on the row of draft j sees.
__device__ __forceinline__ uint64_t seen_bits(const csa_draft_attend_args& A, const Request& R, int32_t j, int32_t p0) {
  auto below = [](int64_t n) { return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1); };
  const uint64_t there = below(static_cast<int64_t>(R.total) - p0), history = below(static_cast<int64_t>(R.base) - p0);
  uint64_t drafts = 0;
  const int32_t i0 = p0 - R.base;  // the draft at p0, below 0 where that is history
  if (!A.mask) {
    drafts = below(static_cast<int64_t>(j) + 1 - i0);
  } else if (i0 > -64) {
    const uint64_t* words = A.mask + (R.row0 + static_cast<int64_t>(j)) * A.mask_stride;
    auto word = [&](int32_t w) { return w >= 0 && w < A.mask_words ? __ldg(reinterpret_cast<const unsigned long long*>(words) + w) : 0ull; };
    if (i0 < 0) drafts = word(0) << -i0;
    else drafts = i0 % 64 ? word(i0 / 64) >> (i0 % 64) | word(i0 / 64 + 1) << (64 - i0 % 64) : word(i0 / 64);
  }
  return there & (history | drafts);
}

// A thread has a row and a quarter of its tile's keys: warps 0, 1 half of the first page's (rows 0 .. 31, 32 .. 63), 2, 3 half of
// the second's, 4 .. 7 the other halves. For the output it has 128 of the row's values, half of its lane of TMEM. m is the
// row's reference, any: it moves only when a tile exceeds it by 2^8, so that O is rarely scaled.
template <bool kFp4, int kRope>
__device__ void role_softmax(const Kernel& K, Smem<kFp4, kRope>& S, uint32_t rank) {
  const csa_draft_attend_args& A = K.A;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = threadIdx.x & (kRows - 1);
  const int half = (warp >> 1) & 1, part = warp >> 2, mine = 2 * part + half, row_bar = kBarRows + (warp & 1);
  constexpr int kRowThreads = 32 * kSoftmaxWarps / 2, kKeys = kTile / 4, kValues = kDim / 4;
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars), lead_bars = csa::peer_smem(bars, 0);
  const uint32_t tmem = S.tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16), o_tmem = tmem + kValues * part;
  const float c = A.scale * 1.4426950408889634f;
  const float grow = fminf(kGrow / c, FLT_MAX);
  const uint32_t p_row = smem_u32(S.p) + half * kColBytes + row * 128;
  uint32_t g = 0;
  bool ok = true;  // once a wait has run out, the rest runs through without waiting: the warps meet at every barrier
  auto o_done = [&](uint32_t tiles) { return tiles == 0 || warp_wait(bars + 8 * kBarODone, (tiles - 1) & 1, stop); };
  uint32_t ordinal = 0;  // of the run's cut pieces
  const Walk& W = S.at;
  auto step = [&](bool first) {
    csa::named_bar_sync(kBarAll, 32 * kSoftmaxWarps);
    if (threadIdx.x == 0) {
      if (first) S.at = S.walk;
      else S.at.next(A);
    }
    csa::named_bar_sync(kBarAll, 32 * kSoftmaxWarps);
  };
  for (step(true); W.more(); step(false)) {
    const Request R = W.w.R;
    const int32_t* table = A.page_table + static_cast<int64_t>(W.request) * A.pt_stride;
    const int64_t flat = W.first_row(A) + kRows * rank + row;
    const bool there = kRows * static_cast<int>(rank) + row < W.rows(A);
    const int32_t j = there ? static_cast<int32_t>(quotient(flat, A.num_heads)) - R.row0 : 0;
    auto page_at = [&](int32_t tile) { return (2 * tile + half) * kPageRecs < R.total ? __ldg(table + 2 * tile + half) : 0; };
    const int32_t first = W.first, n = W.n;
    int32_t page = page_at(first);
    float m = -INFINITY, l = 0.f;  // l: of this thread's quarter of the keys
    for (int i = 0; i < n; ++i, ++g) {
      const int32_t p0 = (2 * (first + i) + half) * kPageRecs;
      const bool good = page >= 0 && page < A.cache.num_pages;
      if (i + 1 < n) page = page_at(first + i + 1);
      ok = ok && warp_wait(bars + 8 * (kBarSFull + (g & 1)), g >> 1 & 1, stop);
      csa::tc_fence_after();
      float s[kKeys];
      {
        uint32_t raw[kKeys];
        csa::tmem_ld32(tmem + kTmemS + (g & 1) * (kTile / 2) + kKeys * part, raw);
        csa::tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < kKeys; ++x) s[x] = __uint_as_float(raw[x]);
      }
      csa::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(lead_bars + 8 * (kBarSEmpty + (g & 1)));
      if (!(good && p0 + kPageRecs <= R.base && there)) {
        const uint32_t seen = good && there ? static_cast<uint32_t>(seen_bits(A, R, j, p0) >> (kKeys * part)) : 0;
#pragma unroll
        for (int x = 0; x < kKeys; ++x)
          if (!(seen >> x & 1)) s[x] = -INFINITY;
      }
      float top = s[0];
#pragma unroll
      for (int x = 1; x < kKeys; ++x) top = fmaxf(top, s[x]);
      if (csa::named_bar_any(row_bar, kRowThreads, top > m + grow)) {  // also when there was nothing (-infinity), not where there is still nothing
        S.quarter[mine][row] = top;
        csa::named_bar_sync(row_bar, kRowThreads);
        top = fmaxf(fmaxf(S.quarter[0][row], S.quarter[1][row]), fmaxf(S.quarter[2][row], S.quarter[3][row]));
        csa::named_bar_sync(row_bar, kRowThreads);
        float keep = 1.f;
        if (top > m + grow) {
          keep = csa::ex2((m - top) * c);  // 0 when there was nothing
          m = top;
          l *= keep;
        }
        if (i > 0) {
          ok = ok && o_done(g);
          csa::tc_fence_after();
#pragma unroll 1
          for (int at = 0; at < kValues; at += 16) {
            uint32_t v[16];
            csa::tmem_ld16(o_tmem + at, v);
            csa::tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * keep);
            csa::tmem_st16(o_tmem + at, v);
          }
          csa::tmem_wait_st();
          csa::tc_fence_before();
        }
      }
      // p is rounded to bf16 here, the tensor cores' operand type; l sums it unrounded
      const float ref = m == -INFINITY ? 0.f : m;
      const csa::F2 minus_ref(-ref, -ref), c2(c, c), zero;
      uint32_t w[kKeys / 2];
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int x = 0; x < kKeys / 2; ++x) {
        float a, b;
        csa::fma2(csa::add2(csa::F2(s[2 * x], s[2 * x + 1]), minus_ref), c2, zero).get(a, b);
        a = csa::ex2(a), b = csa::ex2(b);
        sum[x & 1] += a + b;
        w[x] = pack_bf16(a, b);
      }
      l += sum[0] + sum[1];
      ok = ok && o_done(g);  // the tile before has been read
#pragma unroll
      for (int x = 0; x < 4; ++x)
        csa::st_shared_v4(p_row + (((4 * part + x) ^ (row & 7)) << 4), w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
      csa::fence_proxy_async_smem();
      csa::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(lead_bars + 8 * kBarPFull);
    }
    // the piece's output
    S.quarter[mine][row] = l;
    csa::named_bar_sync(row_bar, kRowThreads);
    l = (S.quarter[0][row] + S.quarter[1][row]) + (S.quarter[2][row] + S.quarter[3][row]);
    csa::named_bar_sync(row_bar, kRowThreads);
    ok = ok && o_done(g);
    csa::tc_fence_after();
    // 64 bytes of each of the warp's 32 rows at a time go through its 2 KB of P (which is not in use between a piece's last
    // O and the next one's first P) and out in runs of them.
    const int rows_here = W.rows(A) - kRows * static_cast<int>(rank) - 32 * (warp & 1);  // of the warp's, that there are
    const uint32_t stage = smem_u32(S.p) + 2048 * warp, r0 = lane >> 2, chunk = lane & 3;
    auto lines_in = [&](const uint32_t (&v)[16]) {
      __syncwarp();
#pragma unroll
      for (int x = 0; x < 4; ++x) csa::st_shared_v4(stage + lane * 64 + ((x ^ ((lane >> 1) & 3)) << 4), v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
      __syncwarp();
    };
    auto lines_out = [&](uint8_t* to, int64_t row_bytes) {  // `to`: the warp's first row
      uint4 y[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) y[x] = csa::ld_shared_v4(stage + (r0 + 8 * x) * 64 + ((chunk ^ (((r0 + 8 * x) >> 1) & 3)) << 4));
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (static_cast<int>(r0) + 8 * x < rows_here) *reinterpret_cast<uint4*>(to + (r0 + 8 * x) * row_bytes + 16 * chunk) = y[x];
    };
    const int first_value = 256 * half + kValues * part;
    if (!W.cut) {
      const float inv = l > 0.f ? 1.f / l : l;  // 0 for an empty row; a NaN stays one
      if (there && mine == 0 && A.lse) A.lse[flat] = l == 0.f ? -INFINITY : fmaf(m, A.scale, log2f(l) * 0.6931471805599453f);
      uint8_t* out = static_cast<uint8_t*>(A.out) + 2 * ((W.first_row(A) + kRows * rank + 32 * (warp & 1)) * kDim + first_value);
      uint32_t v[32];
      csa::tmem_ld32(o_tmem, v);
#pragma unroll 1
      for (int at = 0; at < kValues; at += 32) {
        uint32_t y[16];
        csa::tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 16; ++x) y[x] = pack_bf16(__uint_as_float(v[2 * x]) * inv, __uint_as_float(v[2 * x + 1]) * inv);
        lines_in(y);
        if (at + 32 < kValues) csa::tmem_ld32(o_tmem + at + 32, v);  // the next ones, while these go out
        lines_out(out + 2 * at, 2 * kDim);
      }
    } else {
      float* part_out = K.parts + (static_cast<size_t>(blockIdx.x >> 1) * kParts + ordinal) * kPartFloats;
      const int at_row = kRows * rank + row;
      if (mine == 0) {
        part_out[2 * kRows * kDim + at_row] = m;
        part_out[2 * kRows * (kDim + 1) + at_row] = l;
      }
      uint8_t* to = reinterpret_cast<uint8_t*>(part_out + static_cast<size_t>(kRows * rank + 32 * (warp & 1)) * kDim + first_value);
      uint32_t v[16];
      csa::tmem_ld16(o_tmem, v);
#pragma unroll 1
      for (int at = 0; at < kValues; at += 16) {
        csa::tmem_wait_ld();
        lines_in(v);
        if (at + 16 < kValues) csa::tmem_ld16(o_tmem + at + 16, v);
        lines_out(to + 4 * at, 4 * kDim);
      }
      ++ordinal;
    }
    csa::tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive_at(lead_bars + 8 * kBarOEmpty);
  }
}

template <bool kFp4, int kRope>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Warps<kFp4>::kThreads, 1) attend_kernel(const __grid_constant__ Kernel K, const __grid_constant__ Maps M) {
  extern __shared__ uint8_t smem_raw[];
  Smem<kFp4, kRope>& S = *reinterpret_cast<Smem<kFp4, kRope>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x & 1, bars = smem_u32(S.bars);
  if (threadIdx.x < kBars) {  // a barrier's arrivals
    const int k = threadIdx.x;
    int n = 1;
    if (k < kBarEmpty || k == kBarRopeFull) n = 2 * Warps<kFp4>::kFills;
    else if (k == kBarSEmpty || k == kBarSEmpty + 1 || k == kBarPFull || k == kBarOEmpty) n = 2 * kSoftmaxWarps;
    else if (k == kBarFirstKeys || k == kBarLastValues) n = 4;
    else if (k == kBarQFull) n = 2 * (K.even ? 1 : Warps<kFp4>::kQueries);
    csa::mbar_init(bars + 8 * k, n);
    csa::mbar_init_fence();
  }
  if (threadIdx.x == 0) S.abort = 0;
  if (threadIdx.x < 3) S.fills[threadIdx.x] = 0;
  if (threadIdx.x == 32 * kLoadWarp) {
    if (!kFp4) csa::prefetch_tensormap(&M.two);
    if (!kFp4 && kRope != 0) csa::prefetch_tensormap(&M.one);
    if (K.even) csa::prefetch_tensormap(&M.q);
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&S.tmem)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  int32_t flags = 0;
  csa::tc_fence_before();
  csa::cluster_arrive();
  make_plan(K, S, &flags);  // ends with a block barrier
  csa::cluster_wait();  // the other CTA's barriers are there
  csa::tc_fence_after();
  if (warp < kSoftmaxWarps) {
    role_softmax<kFp4, kRope>(K, S, rank);
  } else if (warp == kMmaWarp) {
    if (rank == 0) {
      role_mma<kFp4, kRope>(K, S);
    } else {  // what this run leaves for the join
      if (lane == 0) {
        Part* parts = K.parts_of + (blockIdx.x >> 1) * kParts;
        int k = 0;
        for (Walk W = S.walk; W.more(); W.next(K.A))
          if (W.cut) parts[k++] = {W.first_row(K.A), W.rows(K.A), W.first == 0};
        while (k < kParts) parts[k++] = {0, 0, 0};
      }
      __syncwarp();
    }
  } else {
    if constexpr (kFp4) {
      if (warp < Warps<kFp4>::kValues) role_keys_fp4<kRope>(K, M, S, rank, &flags);
      else role_values_fp4<kRope>(K, S, rank, &flags);
    } else if (warp == kLoadWarp) role_load<kRope>(K, M, S, rank, &flags);
    else role_query<kRope>(K, M, S, rank);
  }
  csa::tc_fence_before();
  __syncthreads();
  // The last commit has told this CTA too. Behind the block's barrier, because the wait has a limit and this warp nothing else to do: from the
  // start of a run it would end before runs of more than a second do.
  if (warp == kMmaWarp && rank == 1) csa::mbar_wait_drain(bars + 8 * kBarDrain, 0);
  __syncwarp();
  if (threadIdx.x < 4) st_peer_u32(csa::peer_smem(smem_u32(&S.theirs[threadIdx.x]), rank ^ 1), threadIdx.x < 3 ? S.fills[threadIdx.x] : static_cast<uint32_t>(S.abort));
  csa::cluster_arrive();
  csa::cluster_wait();
  // A wait that ran out may have left copies in flight, to be waited for before either CTA leaves. A slot's full barrier wants both
  // CTAs' arrival: the first CTA arrives for the one that did not fill the slot.
  if (S.abort || S.theirs[3]) {
    if (rank == 0 && threadIdx.x == 0) {
      auto drain = [&](int bar, uint32_t a, uint32_t b) {  // filled a and b times
        for (uint32_t k = min(a, b); k < max(a, b); ++k) csa::mbar_arrive(bars + 8 * bar);
        if (max(a, b) > 0) csa::mbar_wait_drain(bars + 8 * bar, (max(a, b) - 1) & 1);
      };
      for (uint32_t k = 0; k < kSlots; ++k) drain(kBarFull + k, (S.fills[0] + kSlots - 1 - k) / kSlots, (S.theirs[0] + kSlots - 1 - k) / kSlots);
      drain(kBarRopeFull, S.fills[1], S.theirs[1]);
      drain(kBarQFull, S.fills[2], S.theirs[2]);
    }
    __syncwarp();
    csa::cluster_arrive();
    csa::cluster_wait();
  }
  if (warp == kMmaWarp) {
    csa::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(S.tmem), "r"(kTmemCols));
  }
  if (threadIdx.x == 0 && S.abort) flags |= CSA_DEV_TIMEOUT;
  flags = static_cast<int32_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(flags)));
  if (flags && K.A.dev_status && lane == 0) atomicOr(K.A.dev_status, flags);
}

// A part's weight 2^x, x <= 0: as a square, so that it becomes subnormal before it becomes 0.
__device__ __forceinline__ float weight(float x) {
  const float h = csa::ex2(0.5f * x);
  return h * h;
}

// Joins the units that are in parts. Block (p, y) takes 8 rows of each unit whose first part is one of run p's; the unit's other
// parts come after it, in the order of its tiles, and are added in that order, so the result does not depend on timing. A
// warp a row, 16 values a lane.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const Kernel K) {
  const csa_draft_attend_args& A = K.A;
  constexpr int kMost = kMaxPairs * kParts;
  __shared__ Part parts[kMost];
  __shared__ uint16_t list[kParts][kMost];  // of each of the run's parts that a unit begins with: the unit's
  __shared__ int32_t count[kParts];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, row = blockIdx.y * kJoinWarps + warp, all = K.pairs * kParts;
  const int from = blockIdx.x * kParts;  // the unit's other parts are behind its first
  asm volatile("griddepcontrol.wait;" ::: "memory");
  bool any = false;
#pragma unroll
  for (int k = 0; k < kParts; ++k) any |= K.parts_of[from + k].begins && static_cast<int>(blockIdx.y) * kJoinWarps < K.parts_of[from + k].rows;
  if (!any) return;
  for (int k = from + tid; k < all; k += 32 * kJoinWarps) parts[k] = K.parts_of[k];
  __syncthreads();
  if (warp < kParts) {
    const int mine = from + warp;
    const Part P = parts[mine];
    int n = 0;
    if (P.begins && static_cast<int>(blockIdx.y) * kJoinWarps < P.rows) {
      for (int k0 = mine; k0 < all; k0 += 32) {
        const int k = k0 + lane;
        const bool is = k < all && parts[k].first == P.first && parts[k].rows > 0;
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, is);
        if (is) list[warp][n + __popc(who & ((1u << lane) - 1))] = static_cast<uint16_t>(k);
        n += __popc(who);
      }
    }
    if (lane == 0) count[warp] = n;
  }
  __syncthreads();
  for (int i = 0; i < kParts; ++i) {
    const int n = count[i];
    const Part P = parts[from + i];
    if (n == 0 || row >= P.rows) continue;
    auto part_of = [&](int k) { return K.parts + static_cast<size_t>(list[i][k]) * kPartFloats; };
    float top = -INFINITY;
    for (int k = lane; k < n; k += 32) top = fmaxf(top, part_of(k)[2 * kRows * kDim + row]);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, k));
    const float ref = top == -INFINITY ? 0.f : top, exponent = A.scale * 1.4426950408889634f;
    float l = 0.f;
    float4 v[4] = {};
    auto add = [&](auto step, int k) {
      constexpr int kStep = decltype(step)::value;
      float w[kStep], s[kStep];
      float4 x[kStep][4];
#pragma unroll
      for (int j = 0; j < kStep; ++j) {
        const float* part = part_of(k + j);
        w[j] = part[2 * kRows * kDim + row];
        s[j] = part[2 * kRows * (kDim + 1) + row];
#pragma unroll
        for (int c = 0; c < 4; ++c) x[j][c] = reinterpret_cast<const float4*>(part + static_cast<size_t>(row) * kDim)[lane + 32 * c];
      }
#pragma unroll
      for (int j = 0; j < kStep; ++j) {
        const float f = weight((w[j] - ref) * exponent);
        l = fmaf(s[j], f, l);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          v[c] = make_float4(fmaf(x[j][c].x, f, v[c].x), fmaf(x[j][c].y, f, v[c].y), fmaf(x[j][c].z, f, v[c].z), fmaf(x[j][c].w, f, v[c].w));
      }
    };
    int k = 0;
    for (; k + 4 <= n; k += 4) add(std::integral_constant<int, 4>(), k);
    for (; k < n; ++k) add(std::integral_constant<int, 1>(), k);
    const float inv = l > 0.f ? 1.f / l : l;
    uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(A.out) + (P.first + row) * kDim);
#pragma unroll
    for (int c = 0; c < 4; ++c) out[lane + 32 * c] = make_uint2(pack_bf16(v[c].x * inv, v[c].y * inv), pack_bf16(v[c].z * inv, v[c].w * inv));
    if (A.lse && lane == 0) A.lse[P.first + row] = l == 0.f ? -INFINITY : fmaf(top, A.scale, log2f(l) * 0.6931471805599453f);
  }
}

// Pairs of the call: one for every two SMs, fewer when there cannot be as many tiles.
int pairs_cap(const csa_draft_attend_args* a) {
  const int64_t rows = static_cast<int64_t>(a->num_q) * a->num_heads, units = rows / (2 * kRows) + a->num_req;
  const int64_t tiles = (static_cast<int64_t>(a->pt_stride) + 1) / 2;
  return static_cast<int>(units >= kMaxPairs || tiles >= kMaxPairs || units * tiles >= kMaxPairs ? kMaxPairs : units * tiles);
}

constexpr size_t kPartsOfBytes = (kMaxPairs * kParts * sizeof(Part) + 255) / 256 * 256;

template <bool kFp4, int kRope>
csa_status launch(Kernel& K, int dev, cudaStream_t stream) {
  static Kept ready;  // the kernel's shared memory size is set on each device once
  constexpr size_t smem = sizeof(Smem<kFp4, kRope>) + 1024;
  static_assert(smem <= 232448, "shared memory of one CTA");
  const csa_draft_attend_args& a = K.A;
  constexpr int64_t kRec = record_bytes(false, kRope);
  Maps M;
  if (!kFp4) {
    const cuuint64_t dims[4] = {64, kPageRecs, static_cast<cuuint64_t>(kRec / 128), static_cast<cuuint64_t>(a.cache.num_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(kRec), 128, static_cast<cuuint64_t>(a.cache.page_stride_bytes)};
    const cuuint32_t two[4] = {64, kPageRecs, 2, 1}, one[4] = {64, kPageRecs, 1, 1};
    if (!encode_map(&M.two, a.cache.pages, 4, dims, strides, two) || !encode_map(&M.one, a.cache.pages, 4, dims, strides, one)) return CSA_ERR_INVALID_ARG;
  }
  const int64_t rows = static_cast<int64_t>(a.num_q) * a.num_heads, step = a.num_heads > 1 ? a.q_head_stride : a.q_row_stride;
  K.even = rows <= INT32_MAX && (a.num_q == 1 || a.num_heads == 1 || a.q_row_stride == a.num_heads * a.q_head_stride) &&
           encode_bf16(&M.q, a.q, kDim + kRope, 0, rows, 0, rows > 1 ? step : kDim + kRope, 0, kRows);
  if (!ready.get(dev)) {
    if (cudaFuncSetAttribute(attend_kernel<kFp4, kRope>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
      return CSA_ERR_CUDA;
    ready.set(dev, 1);
  }
  attend_kernel<kFp4, kRope><<<2 * K.pairs, Warps<kFp4>::kThreads, smem, stream>>>(K, M);
  return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

csa_status check_args(const csa_draft_attend_args* a) {
  if (!a || a->num_q < 0 || a->num_req < 0 || a->pt_stride < 0 || a->mask_words < 0) return CSA_ERR_INVALID_ARG;
  if (a->num_heads < 1 || a->num_heads > CSA_LATENT_MAX_HEADS || a->mask_words > CSA_DRAFT_MAX_WORDS || a->num_req > CSA_DRAFT_MAX_REQ)
    return CSA_ERR_UNSUPPORTED;
  if (!good_scale(a->scale)) return CSA_ERR_INVALID_ARG;
  if (a->num_q == 0 || a->num_req == 0) return CSA_OK;
  const csa_status st = check_cache(a->cache);
  if (st != CSA_OK) return st;
  const int wide = kDim + a->cache.rope_dim;
  if (!a->q || !a->page_table || !a->base_len || !a->row_start || !a->out || a->pt_stride < 1) return CSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(kPageRecs) * a->pt_stride > INT32_MAX - 2 * kTile) return CSA_ERR_INVALID_ARG;  // a tile's end is an int32 too
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
  if (!a || a->num_q < 0 || a->num_req < 0 || a->pt_stride < 0 || a->num_heads < 1 || a->num_heads > CSA_LATENT_MAX_HEADS ||
      a->num_req > CSA_DRAFT_MAX_REQ)
    return 0;
  if (a->num_q > 0 && a->num_req > 0 && (a->pt_stride < 1 || static_cast<int64_t>(kPageRecs) * a->pt_stride > INT32_MAX - 2 * kTile)) return 0;
  return kPartsOfBytes + kParts * static_cast<size_t>(pairs_cap(a)) * kPartFloats * sizeof(float);
}

extern "C" csa_status csa_draft_attend(const csa_draft_attend_args* a, void* ws, size_t ws_bytes, void* stream) {
  const csa_status st = check_args(a);
  if (st != CSA_OK) return st;
  if (a->num_q == 0 || a->num_req == 0) return CSA_OK;
  if (!ws || ws_bytes < csa_draft_attend_workspace_bytes(a)) return CSA_ERR_WORKSPACE;
  if (!aligned(ws, 32)) return CSA_ERR_ALIGNMENT;
  const auto s = static_cast<cudaStream_t>(stream);
  int sms = 0, dev = 0;
  if (sm_count(&sms, &dev) != CSA_OK) return CSA_ERR_CUDA;
  Kernel K;
  K.A = *a;
  K.pairs = pairs_cap(a) < sms / 2 ? pairs_cap(a) : sms / 2;
  K.parts_of = static_cast<Part*>(ws);
  K.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kPartsOfBytes);
  const bool fp4 = a->cache.record_format == CSA_LATENT_MXFP4, rope = a->cache.rope_dim != 0;
  const csa_status ls = fp4 ? (rope ? launch<true, 64>(K, dev, s) : launch<true, 0>(K, dev, s)) : (rope ? launch<false, 64>(K, dev, s) : launch<false, 0>(K, dev, s));
  if (ls != CSA_OK || K.pairs == 1) return ls;
  cudaLaunchConfig_t cfg = {};
  const int64_t rows = static_cast<int64_t>(a->num_q) * a->num_heads;
  cfg.gridDim = dim3(K.pairs, static_cast<unsigned>(((rows < 2 * kRows ? rows : 2 * kRows) + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel, K) == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}
