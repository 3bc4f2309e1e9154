// csa_latent_attend.cu — latent attention, absorbed form (include/csa_latent.h).
#include <cfloat>

#include "csa_latent_common.cuh"
#include "csa_latent_maps.h"
#include "csa_latent_ptx.cuh"

namespace csa_latent {
namespace {

using csa::mbar_arrive;
using csa::mbar_wait;
using csa::smem_u32;

// The kernel. Per head h and visible record n, with S = q . c:
//   p_n = 2^(S_n c - m c), c = scale log2 e,  O = sum p_n c_n[0:512],  l = sum p_n,
// out = O / l, lse = ln 2 (m c + log2 l), for any reference m per head: m is the first tile's
// maximum and moves only when a tile exceeds it by 2^8, so that O is rarely rescaled and
// p stays below 2^8.
//
// A CTA takes 64 heads of one row and runs over tiles of 64 records. One tile in shared
// memory is both operands of the tensor cores: K-major as the keys (S = Q C^T, 64 heads x 64
// records over the record's 512 + rope values), MN-major as the values (O^T = C^T P^T, 512
// values x 64 heads over the 64 records), so a record is fetched once. S is kept with a head a
// TMEM lane, so that a softmax row belongs to one thread; O is kept transposed (128 values a
// lane block, a head a column), because 64 heads x 512 values with the heads in the lanes
// would fill all 512 columns of TMEM and leave S no room.
//
// Shared memory: Q (72 KB), two record tiles (72 KB each), P (8 KB): 224 KB, one CTA an SM.
// Four warps: softmax (S from TMEM, P to shared memory) and the output. Then the loaders: one
// warp and TMA where a tile is a page of whole bf16 records, else eight warps, which hold one more tile
// in registers, so that its global loads are in flight while both tiles in shared memory are in
// use; MXFP4 codes become bf16 values (exactly) on the way. Of the last two warps one issues the MMAs of S, the other
// those of O, so that neither waits for the other's operands and S of tile i + 1 runs during tile i's
// softmax. Of a tile 128 values move at a time: the next one comes in while O still reads the rest.
//
// Work is split over a long axis: the tiles of all (row, head group) units, in order, are
// cut into equal runs, one a CTA; a unit that is cut leaves unnormalised parts (O, m, l in
// fp32) in the workspace, which a second kernel joins in the order of the runs, so results do not
// depend on timing.
//
// 4 rows of 65536 to 131072 bf16 records, 64 heads: 96 us, 5.0 TB/s, bound by HBM. 32 rows of 32768 4-bit records, 64 heads: 233 us,
// 0.60 PFLOP/s, and 1024 rows of 512 positions, 128 heads: 281 us, 0.52 PFLOP/s: 4.0 k and 4.7 k clocks a tile, of which the tensor
// cores are active 1.66 k (S, 64 rows high and so at half rate, 1152, and O 512). What is full is shared memory: the
// MMAs read 240 KB of operands a tile (Q and the records for S, the records again and four times P for O), 1.9 k clocks at 128
// bytes a clock, and the roles' own loads and stores are 1.2 k wavefronts more; the second case adds the hand-over between units.
constexpr int kTile = 64, kHeads = 64;            // records a tile, heads a unit
constexpr int kColBytes = kTile * 128;            // 64 values of a tile's 64 records (or of Q's 64 heads)
constexpr int kSoftmaxWarps = 4;
// How records get to shared memory.
enum { kLoadTma = 0, kLoadFp4 = 1, kLoadBf16 = 2 };
template <int kLoad>
struct Warps {  // the softmax's, the loaders' (of which TMA uses one; all help in a cluster's join), S's and O's MMAs'
  static constexpr int kLoaders = kLoad == kLoadTma ? 4 : 8, kMma = kSoftmaxWarps + kLoaders, kThreads = 32 * (kMma + 2);
  static constexpr int kFills = kLoad == kLoadTma ? 1 : kLoaders;  // arrivals that make a buffer full
};
constexpr int kMaxGrid = 160;                     // CTAs at most: sizes the workspace
constexpr uint32_t kTmemCols = 512, kTmemS = 256;  // O^T in columns 0 .. 255, S in 256 .. 383
constexpr float kGrow = 8.0f;                     // log2 of how far p may exceed 1
constexpr int kBarSoftmax = 1;

template <int kRope>
struct Smem {
  static constexpr int kCols = (kDim + kRope) / 64;
  uint8_t q[kCols * kColBytes];
  uint8_t c[2][kCols * kColBytes];
  uint8_t p[kHeads * 128];
  uint64_t bars[20];
  uint8_t valid[2][kTile];  // 1 where the tile's record is visible
  alignas(16) float alpha[kHeads];
  float mc[kHeads], l[kHeads];  // cluster: this CTA's reference and sum per head
  int64_t total;
  int32_t unit, off;
  uint32_t tmem;
  int abort;
};
constexpr int kPairs = kDim / 128;  // a tile moves in 128 values at a time
// A tile is handed over in two halves of 256 values: barriers 2 * stage + half.
enum { kBarCFull = 0, kBarCEmpty = 4, kBarSFull = 8, kBarSEmpty = 10, kBarQFull = 12, kBarQEmpty, kBarPFull,
       kBarOEmpty, kBarDrainS, kBarDrainO, kBarLand };

// A part of a cut unit: O [64 heads][512], then m c and l of the 64 heads.
constexpr size_t kPartFloats = static_cast<size_t>(kHeads) * (kDim + 2);

// Where a unit begins, for the join: written by the run that holds its first tile, at the unit's index
// where there are at most as many units as runs, else at the run's (a run opens one cut unit at most).
struct Open {
  int64_t begin, total;  // the unit's first tile and all units' tiles, in the order of the runs
  int32_t unit, run, tiles, cut;
};

struct Kernel {
  csa_latent_attend_args A;
  Open* opens;
  float* parts;
  int32_t groups;  // head groups of 64: 1 or 2
  int32_t by_unit;  // opens are indexed by unit
  int32_t cluster;  // CTAs that share a unit and join it among themselves; 0: runs over all units
};

__device__ __forceinline__ int row_of(const Kernel& K, int unit) { return unit >> (K.groups - 1); }
__device__ __forceinline__ int group_of(const Kernel& K, int unit) { return unit & (K.groups - 1); }

// What a query row sees: its request's page table row and its length.
struct RowView {
  const int32_t* table;
  int32_t len;  // 0 for a row whose request is out of range
};

__device__ __forceinline__ RowView row_view(const csa_latent_attend_args& A, int b, int32_t* flags) {
  const int32_t req = A.row_req ? A.row_req[b] : b;
  if (req < 0 || req >= A.num_req) {
    *flags |= CSA_DEV_BAD_REQUEST;
    return {A.page_table, 0};
  }
  const int32_t n = A.row_len[b], cap = kPageRecs * A.pt_stride, len = min(max(n, 0), cap);
  if (len != n) *flags |= CSA_DEV_LEN_OOB;
  return {A.page_table + static_cast<int64_t>(req) * A.pt_stride, len};
}

// Tiles of row b; an empty row still has one, which writes its output.
__device__ __forceinline__ int tiles_of(const csa_latent_attend_args& A, int b) {
  if (A.idx) return (A.top + kTile - 1) / kTile;
  int32_t ignore = 0;
  return max(1, (row_view(A, b, &ignore).len + kTile - 1) / kTile);
}

// The position of entry j of the row (of the listed positions, or of the history); -1 for none.
__device__ __forceinline__ int32_t position_of(const csa_latent_attend_args& A, const RowView& R, int b, int j) {
  if (A.idx) return j < A.top ? __ldg(A.idx + b * A.idx_stride + j) : -1;
  return j < R.len ? j : -1;
}

// The record at a position, or null.
__device__ __forceinline__ const uint8_t* record_at(const csa_latent_attend_args& A, const RowView& R, int32_t pos,
                                                    int rec_bytes, int32_t* flags) {
  if (pos == -1) return nullptr;
  if (pos < 0 || pos >= R.len) {
    *flags |= CSA_DEV_LEN_OOB;
    return nullptr;
  }
  const int32_t page = __ldg(R.table + pos / kPageRecs);
  if (page < 0 || page >= A.cache.num_pages) {
    *flags |= CSA_DEV_PAGE_OOB;
    return nullptr;
  }
  return A.cache.pages + page * A.cache.page_stride_bytes + static_cast<int64_t>(pos % kPageRecs) * rec_bytes;
}

__host__ __device__ __forceinline__ int64_t run_start(int64_t total, int c, int grid) { return total * c / grid; }

// This CTA's run: the total of all units' tiles, and the unit and the tile in it where the run starts.
template <int kThreads, int kRope>
__device__ void make_plan(const Kernel& K, Smem<kRope>& S, int64_t* scan) {
  const csa_latent_attend_args& A = K.A;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (K.cluster) {
    if (tid == 0) {
      S.unit = blockIdx.x / K.cluster;
      const int n = tiles_of(A, row_of(K, S.unit)), rank = blockIdx.x % K.cluster;
      S.off = n * rank / K.cluster;
      S.total = n * (rank + 1) / K.cluster - S.off;  // this CTA's tiles, maybe none
    }
    __syncthreads();
    return;
  }
  if (A.idx) {
    if (tid == 0) {
      const int64_t per = tiles_of(A, 0);
      S.total = per * A.num_q * K.groups;
      const int64_t at = run_start(S.total, blockIdx.x, gridDim.x);
      S.unit = static_cast<int32_t>(at / per);
      S.off = static_cast<int32_t>(at % per);
    }
    __syncthreads();
    return;
  }
  const int per = (A.num_q + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, A.num_q), b1 = min(b0 + per, A.num_q);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += tiles_of(A, b);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  before *= K.groups;
  total *= K.groups;
  const int64_t at = run_start(total, blockIdx.x, gridDim.x);
  if (tid == 0) S.total = total;
  if (at >= before && at < before + mine * K.groups) {
    for (int b = b0; b < b1; ++b) {
      const int64_t n = tiles_of(A, b), all = n * K.groups;
      if (at < before + all) {
        S.unit = b * K.groups + static_cast<int32_t>((at - before) / n);
        S.off = static_cast<int32_t>((at - before) % n);
        break;
      }
      before += all;
    }
  }
  __syncthreads();
}

// Walks a run piece by piece: a piece is the run's part of one unit.
struct Pieces {
  int64_t left;
  int unit, off, tiles, n;  // tiles of the unit, tiles of the piece
  template <int kRope>
  __device__ __forceinline__ Pieces(const Kernel& K, const Smem<kRope>& S) {
    left = K.cluster ? S.total : run_start(S.total, blockIdx.x + 1, gridDim.x) - run_start(S.total, blockIdx.x, gridDim.x);
    unit = S.unit;
    off = S.off;
    size(K);
  }
  __device__ __forceinline__ void size(const Kernel& K) {
    if (left <= 0) return;
    tiles = tiles_of(K.A, row_of(K, unit));
    n = static_cast<int>(min(left, static_cast<int64_t>(tiles - off)));
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next(const Kernel& K) {
    left -= n;
    ++unit;
    off = 0;
    size(K);
  }
};

// The units that begin in this run.
template <int kRope>
__device__ void write_opens(const Kernel& K, const Smem<kRope>& S) {
  int64_t at = run_start(S.total, blockIdx.x, gridDim.x);
  if (!K.by_unit) K.opens[blockIdx.x].cut = 0;
  for (Pieces run(K, S); run.more(); run.next(K)) {
    const bool cut = run.n < run.tiles;
    if (run.off == 0 && (cut || K.by_unit))
      K.opens[K.by_unit ? run.unit : blockIdx.x] = {at, S.total, run.unit, static_cast<int32_t>(blockIdx.x), run.tiles, cut};
    at += run.n;
  }
}

// The bytes of one tile in a loader thread's registers, 128 values of its records at a time, and how
// they become the tile in shared memory: value v of record r at column v / 64, row r, 16-byte
// chunk (v % 64) / 8 ^ (r % 8). The rope values travel with the first 128.
template <bool kFp4, int kRope>
struct TileRegs;

// bf16: eight lanes a record (128 bytes of it at a time), records r and r + 32.
template <int kRope>
struct TileRegs<false, kRope> {
  static constexpr int kRecords = 2;  // records a thread has a share in
  uint4 w[kRecords][kDim / 64], rope[kRecords];
  static __device__ __forceinline__ int record(int t, int k) { return (t >> 3) + 32 * k; }
  static __device__ __forceinline__ bool leads(int t) { return (t & 7) == 0; }
  __device__ __forceinline__ void convert(int, int) {}
  static __device__ __forceinline__ void prefetch(const uint8_t* const (&rec)[kRecords], int t) {
#pragma unroll
    for (int k = 0; k < kRecords; ++k) {
      if (!rec[k]) continue;
      csa::prefetch_l2(rec[k] + 128 * (t & 7));
      if (kRope != 0 && (t & 7) == 0) csa::prefetch_l2(rec[k] + 2 * kDim);
    }
  }
  __device__ __forceinline__ void fetch(const uint8_t* const (&rec)[kRecords], int pair, int t) {
#pragma unroll
    for (int k = 0; k < kRecords; ++k) {
      const uint4* p = reinterpret_cast<const uint4*>(rec[k]) + (t & 7);
      const uint4 zero = make_uint4(0, 0, 0, 0);
      w[k][2 * pair] = rec[k] ? __ldg(p + 16 * pair) : zero;
      w[k][2 * pair + 1] = rec[k] ? __ldg(p + 16 * pair + 8) : zero;
      if (kRope != 0 && pair == 0) rope[k] = rec[k] ? __ldg(p + kDim / 8) : zero;
    }
  }
  __device__ __forceinline__ void store(uint32_t dst, int pair, int t) const {
#pragma unroll
    for (int k = 0; k < kRecords; ++k) {
      const int r = record(t, k);
      const uint32_t at = dst + r * 128 + (((t & 7) ^ (r & 7)) << 4);
#pragma unroll
      for (int c = 2 * pair; c < 2 * pair + 2; ++c)
        csa::st_shared_v4(at + c * kColBytes, w[k][c].x, w[k][c].y, w[k][c].z, w[k][c].w);
      if (kRope != 0 && pair == 0)
        csa::st_shared_v4(at + kDim / 64 * kColBytes, rope[k].x, rope[k].y, rope[k].z, rope[k].w);
    }
  }
};

// MXFP4: four lanes a record; of each 128 values (four blocks of 32: 16 code bytes and one scale
// byte) lane s takes block s, and a quarter of the rope values.
template <int kRope>
struct TileRegs<true, kRope> {
  static constexpr int kRecords = 1;
  uint4 code[kPairs], rope[2], rope_now[2];
  uint32_t scale[kPairs], value[2][16];
  static __device__ __forceinline__ int record(int t, int) { return t >> 2; }
  static __device__ __forceinline__ bool leads(int t) { return (t & 3) == 0; }
  __device__ __forceinline__ void fetch(const uint8_t* const (&rec)[kRecords], int pair, int t) {
    const uint4* p = reinterpret_cast<const uint4*>(rec[0]);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    code[pair] = p ? __ldg(p + 4 * pair + (t & 3)) : zero;
    scale[pair] = p ? __ldg(rec[0] + kCodeBytes + 4 * pair + (t & 3)) : 0u;
    if (pair == 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        rope[k] = kRope != 0 && p ? __ldg(p + (kCodeBytes + kScaleBytes) / 16 + 2 * (t & 3) + k) : zero;
    }
  }
  static __device__ __forceinline__ void prefetch(const uint8_t* const (&rec)[kRecords], int t) {
    if (rec[0]) csa::prefetch_l2(rec[0] + min(128 * (t & 3), record_bytes(true, kRope) - 1));
  }
  // The codes fetched become the values to store, ahead of the tile's turn.
  __device__ __forceinline__ void convert(int pair, int t) {
    const bool swap = (t & 3) >= 2;  // lanes 2, 3 store their words in another order: no two on one bank
    const uint32_t sb = scale[pair];
    const uint32_t bits = sb == 0 ? 0x0040u : (sb == 255 ? 0x7FC0u : sb << 7);
    const uint32_t two = bits | (bits << 16);
    const __nv_bfloat162 s2 = *reinterpret_cast<const __nv_bfloat162*>(&two);
    const uint4 c = code[pair];
    const uint32_t word[4] = {swap ? c.z : c.x, swap ? c.w : c.y, swap ? c.x : c.z, swap ? c.y : c.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t* v = value[pair & 1] + 4 * j;
      mxfp4_four(word[j], s2, &v[0], &v[1]);
      mxfp4_four(word[j] >> 16, s2, &v[2], &v[3]);
    }
    if (kRope != 0 && pair == 0) {
      rope_now[0] = rope[0];
      rope_now[1] = rope[1];
    }
  }
  __device__ __forceinline__ void store(uint32_t dst, int pair, int t) const {
    const int r = t >> 2, s = t & 3;
    const uint32_t row = dst + r * 128;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int chunk = 4 * (s & 1) + (s >= 2 ? j ^ 2 : j);
      const uint32_t* v = value[pair & 1] + 4 * j;
      csa::st_shared_v4(row + (2 * pair + (s >> 1)) * kColBytes + ((chunk ^ (r & 7)) << 4), v[0], v[1], v[2], v[3]);
    }
    if (kRope != 0 && pair == 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        csa::st_shared_v4(row + kDim / 64 * kColBytes + (((2 * s + k) ^ (r & 7)) << 4), rope_now[k].x, rope_now[k].y,
                          rope_now[k].z, rope_now[k].w);
    }
  }
};

// A whole warp's bounded wait. The answer is the same for all lanes: a lane that left a role alone
// would strand the others at their next warp barrier.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* stop) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, stop));
}

template <bool kFp4, int kRope>
__device__ void role_load_regs(const Kernel& K, Smem<kRope>& S, int32_t* flags) {
  constexpr int kCols = Smem<kRope>::kCols;
  using Regs = TileRegs<kFp4, kRope>;
  const csa_latent_attend_args& A = K.A;
  const int t = threadIdx.x - 32 * kSoftmaxWarps, lane = t & 31;
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars);
  csa::test_delay();
  Pieces run(K, S);
  if (!run.more()) return;
  // A tile's records are found in two steps, one tile apart, so that no load waits for another one just
  // issued: the entries' positions, then their pages.
  Pieces ahead = run;
  int tile = ahead.off, piece_end = ahead.off + ahead.n;
  RowView R = row_view(A, row_of(K, ahead.unit), flags), R_found = R;
  int32_t pos[Regs::kRecords];
  const uint8_t* rec[Regs::kRecords];
  auto find = [&]() {  // the positions of the next tile of the run, -1 past its end
    if (ahead.more() && tile == piece_end) {
      ahead.next(K);
      if (ahead.more()) {
        R = row_view(A, row_of(K, ahead.unit), flags);
        tile = ahead.off;
        piece_end = ahead.off + ahead.n;
      }
    }
#pragma unroll
    for (int k = 0; k < Regs::kRecords; ++k)
      pos[k] = ahead.more() ? position_of(A, R, row_of(K, ahead.unit), tile * kTile + Regs::record(t, k)) : -1;
    R_found = R;
    ++tile;
  };
  auto locate = [&]() {  // the records at the positions found
#pragma unroll
    for (int k = 0; k < Regs::kRecords; ++k) rec[k] = record_at(A, R_found, pos[k], record_bytes(kFp4, kRope), flags);
  };
  Regs x;
  bool live[Regs::kRecords];
  // `rec` are the records of the tile after the one in the registers
  find();
  locate();
  find();
#pragma unroll
  for (int pair = 0; pair < kPairs; ++pair) x.fetch(rec, pair, t);
#pragma unroll
  for (int k = 0; k < Regs::kRecords; ++k) live[k] = rec[k] != nullptr;
  locate();
  find();
  uint32_t g = 0, piece = 0;
  for (; run.more(); run.next(K), ++piece) {
    // Q of the piece: head h's 64-value columns at row h, swizzled as the records; zeros past the last head
    const int b = row_of(K, run.unit), h0 = group_of(K, run.unit) * kHeads;
    if (!warp_wait(bars + 8 * kBarQEmpty, (piece & 1) ^ 1, stop)) return;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int h = (t >> 3) + 32 * k;
      const bool on = h0 + h < A.num_heads;
      const uint8_t* q = static_cast<const uint8_t*>(A.q) +
                         2 * (b * A.q_row_stride + (on ? h0 + h : 0) * A.q_head_stride) + 16 * (t & 7);
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        csa::cp_async16(smem_u32(S.q) + c * kColBytes + h * 128 + (((t & 7) ^ (h & 7)) << 4), q + 128 * c, on);
    }
    if (run.left > run.n) {  // the next unit's Q on its way to L2: its own copy can only start when this one's last S is done
      const int nb = row_of(K, run.unit + 1), n0 = group_of(K, run.unit + 1) * kHeads;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int h = (t >> 3) + 32 * k;
        if (n0 + h < A.num_heads && (t & 7) == 0)
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            csa::prefetch_l2(static_cast<const uint8_t*>(A.q) + 2 * (nb * A.q_row_stride + (n0 + h) * A.q_head_stride) + 128 * c);
      }
    }
    csa::cp_async_wait_all();
    csa::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * kBarQFull);
    for (int i = 0; i < run.n; ++i, ++g) {
      const uint32_t stage = g & 1;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        x.convert(2 * half, t);  // before the tile's turn, where that is not yet come
        x.convert(2 * half + 1, t);
        if constexpr (kFp4) {  // the codes' registers are free: the next tile's have all of this one's time to arrive
          x.fetch(rec, 2 * half, t);
          x.fetch(rec, 2 * half + 1, t);
        }
        if (!warp_wait(bars + 8 * (kBarCEmpty + 2 * stage + half), ((g >> 1) & 1) ^ 1, stop)) return;
        x.store(smem_u32(S.c[stage]), 2 * half, t);
        x.store(smem_u32(S.c[stage]), 2 * half + 1, t);
        if (half == 0 && Regs::leads(t)) {
#pragma unroll
          for (int k = 0; k < Regs::kRecords; ++k) S.valid[stage][Regs::record(t, k)] = live[k];
        }
        csa::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + 8 * (kBarCFull + 2 * stage + half));
        if constexpr (!kFp4) {  // in flight until this half's turn comes again
          x.fetch(rec, 2 * half, t);
          x.fetch(rec, 2 * half + 1, t);
        }
      }
#pragma unroll
      for (int k = 0; k < Regs::kRecords; ++k) live[k] = rec[k] != nullptr;
      // While the tile's turn has not come: the records of the one after it, on their way to L2. Not where many
      // rows list positions: 1024 rows of one request, 512 positions, 128 heads take 289 us with it and 286
      // without, their records being in L2 already. Rows of 128 different requests, which take this branch too, would be
      // better off with it: 73 us, 79 without (bf16; 65 and 67 of 4-bit records).
      locate();
      find();
      if (!A.idx || K.cluster) x.prefetch(rec, t);
    }
  }
}

struct Maps {  // tensor maps of the TMA loader
  CUtensorMap q;      // [row][head][value], boxes of 64 values of 64 heads
  CUtensorMap pages;  // [page][record][column of 64 values][value], boxes of one column of a page: a tile
};

// The TMA loader: one warp, for whole histories, where a tile is a page and nine (or eight) copies fill it. Where a
// page's end is not visible, its rows become zeros before the tile is handed over (they may hold NaN, and 0 x NaN is
// not 0).
template <int kRope>
__device__ void role_load_tma(const Kernel& K, const Maps& M, Smem<kRope>& S, int32_t* flags) {
  constexpr int kCols = Smem<kRope>::kCols, kRec = record_bytes(false, kRope);
  const csa_latent_attend_args& A = K.A;
  const int lane = threadIdx.x & 31;
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars);
  csa::test_delay();
  Pieces run(K, S), ahead = run;
  if (!run.more()) return;
  struct Tile {
    int32_t page, rows;  // -1, 0: nothing of it is visible
  };
  int tile = ahead.off, piece_end = ahead.off + ahead.n;
  RowView R = row_view(A, row_of(K, ahead.unit), flags);
  auto next_tile = [&]() {  // of the run, its page on the way to L2
    if (ahead.more() && tile == piece_end) {
      ahead.next(K);
      if (ahead.more()) {
        R = row_view(A, row_of(K, ahead.unit), flags);
        tile = ahead.off;
        piece_end = ahead.off + ahead.n;
      }
    }
    Tile T = {-1, 0};
    if (ahead.more() && tile * kTile < R.len) {
      const int32_t page = __ldg(R.table + tile);
      if (page < 0 || page >= A.cache.num_pages) *flags |= CSA_DEV_PAGE_OOB;
      else T = {page, min(kTile, R.len - tile * kTile)};
    }
    if (lane == 0 && T.rows > 0) csa::bulk_prefetch_l2(A.cache.pages + T.page * A.cache.page_stride_bytes, T.rows * kRec);
    ++tile;
    return T;
  };
  static_assert(kTile == kPageRecs, "a tile is a page");
  Tile now = next_tile(), next = next_tile();
  uint32_t g = 0, piece = 0, landed = 0, filled[2] = {0, 0};  // tiles whose halves were begun (or handed over)
  bool ok = true, landing = false;                            // landing: copies to kBarLand are in flight
  for (; run.more(); run.next(K)) {
    ok = ok && warp_wait(bars + 8 * kBarQEmpty, (piece & 1) ^ 1, stop);
    if (!ok) break;
    ++piece;
    if (lane == 0) {
      const uint32_t bar = bars + 8 * kBarQFull;
      csa::mbar_arrive_expect_tx(bar, sizeof(S.q));
      for (int c = 0; c < kCols; ++c)
        csa::tma_tile_3d(smem_u32(S.q) + c * kColBytes, &M.q, 64 * c, group_of(K, run.unit) * kHeads, row_of(K, run.unit), bar);
    }
    for (int i = 0; i < run.n; ++i, ++g) {
      const uint32_t stage = g & 1, dst = smem_u32(S.c[stage]);
      const bool whole = now.rows == kTile;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        ok = ok && warp_wait(bars + 8 * (kBarCEmpty + 2 * stage + half), ((g >> 1) & 1) ^ 1, stop);
        if (!ok) break;
        const uint32_t full = bars + 8 * (kBarCFull + 2 * stage + half), bar = whole ? full : bars + 8 * kBarLand;
        if (half == 0) {
          S.valid[stage][lane] = lane < now.rows;
          S.valid[stage][lane + 32] = lane + 32 < now.rows;
          __syncwarp();
        }
        const int columns = kDim / 128 + (kRope != 0 && half == 0);  // of the half: 4 half .. 4 half + 3, and rope with the first
        auto column = [&](int c) { return c < kDim / 128 ? kDim / 128 * half + c : kDim / 64; };
        if (now.rows > 0 && lane == 0) {
          csa::mbar_arrive_expect_tx(bar, columns * kColBytes);
          for (int c = 0; c < columns; ++c) csa::tma_tile_4d(dst + column(c) * kColBytes, &M.pages, 0, column(c), 0, now.page, bar);
        }
        if (whole) filled[half] = g + 1;
        if (whole) continue;
        if (now.rows > 0) {
          landing = true;
          ok = warp_wait(bar, landed & 1, stop);
          if (!ok) break;
          landing = false;
          ++landed;
        }
        for (int c = 0; c < columns; ++c)
          for (int b = now.rows * 128 + 16 * lane; b < kColBytes; b += 512) csa::st_shared_v4(dst + column(c) * kColBytes + b, 0, 0, 0, 0);
        csa::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
        filled[half] = g + 1;
      }
      if (!ok) break;
      now = next;
      next = next_tile();
    }
  }
  // no copy of this CTA is in flight when it leaves
  if (lane == 0) {
    if (piece > 0) csa::mbar_wait_drain(bars + 8 * kBarQFull, (piece - 1) & 1);
    for (int half = 0; half < 2; ++half)
      for (uint32_t k = filled[half] > 2 ? filled[half] - 2 : 0; k < filled[half]; ++k)
        csa::mbar_wait_drain(bars + 8 * (kBarCFull + 2 * (k & 1) + half), (k >> 1) & 1);
    if (landing) csa::mbar_wait_drain(bars + 8 * kBarLand, landed & 1);
  }
  __syncwarp();
}

template <int kRope>
__device__ void role_mma_s(const Kernel& K, Smem<kRope>& S) {
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars), tmem = csa::uniform(S.tmem) + kTmemS, lead = csa::elect_lane();
  constexpr uint32_t idesc = csa::idesc_bf16_f32(64, kTile);
  const csa::Desc q_desc(csa::sdesc_kmajor_sw128(smem_u32(S.q))), c_descs(csa::sdesc_kmajor_sw128(smem_u32(S.c[0])));
  uint32_t g = 0, piece = 0;
  bool ok = true;
  for (Pieces run(K, S); ok && run.more(); run.next(K), ++piece) {
    ok = warp_wait(bars + 8 * kBarQFull, piece & 1, stop);
    const int n = csa::uniform(run.n);
    for (int i = 0; ok && i < n; ++i, ++g) {
      ok = warp_wait(bars + 8 * (kBarSEmpty + (g & 1)), ((g >> 1) & 1) ^ 1, stop);
      const csa::Desc c_desc = c_descs.at((g & 1) * sizeof(S.c[0]));
      const uint32_t d = tmem + (g & 1) * kTile;
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // as the tile is filled
        ok = ok && warp_wait(bars + 8 * (kBarCFull + 2 * (g & 1) + half), (g >> 1) & 1, stop);
        if (!ok) break;
        csa::tc_fence_after();
#pragma unroll
        for (int at = kDim / 2 * half; at < kDim / 2 * (half + 1); at += 16) {
          const uint32_t bytes = at / 64 * kColBytes + at % 64 * 2;
          csa::mma_f16_ss(lead, d, q_desc.at(bytes), c_desc.at(bytes), idesc, at > 0);
        }
        if (kRope != 0 && half == 0) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t bytes = kDim / 64 * kColBytes + 32 * k;
            csa::mma_f16_ss(lead, d, q_desc.at(bytes), c_desc.at(bytes), idesc, true);
          }
        }
      }
      if (!ok) break;
      csa::mma_commit_if(lead, bars + 8 * (kBarSFull + (g & 1)));
      if (i + 1 == n) csa::mma_commit_if(lead, bars + 8 * kBarQEmpty);
    }
  }
  csa::mma_commit_if(lead, bars + 8 * kBarDrainS);  // nothing of this warp's MMAs is in flight when it leaves
  csa::mbar_wait_drain(bars + 8 * kBarDrainS, 0);
  __syncwarp();
}

template <int kRope>
__device__ void role_mma_o(const Kernel& K, Smem<kRope>& S) {
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars), tmem = csa::uniform(S.tmem), lead = csa::elect_lane();
  const csa::Desc p_desc(csa::sdesc_kmajor_sw128(smem_u32(S.p))), c_descs(csa::sdesc_mn_sw128_b16(smem_u32(S.c[0]), kColBytes));
  uint32_t g = 0, piece = 0;
  bool ok = true;
  for (Pieces run(K, S); ok && run.more(); run.next(K), ++piece) {
    const int heads = min(K.A.num_heads - group_of(K, run.unit) * kHeads, kHeads);
    const uint32_t idesc = csa::uniform(csa::idesc_bf16_f32(128, (heads + 15) / 16 * 16) | csa::kIdescAMnMajor);
    ok = warp_wait(bars + 8 * kBarOEmpty, (piece & 1) ^ 1, stop);
    const int n = csa::uniform(run.n);
    for (int i = 0; ok && i < n; ++i, ++g) {
      ok = warp_wait(bars + 8 * kBarPFull, g & 1, stop);
      if (!ok) break;
      csa::tc_fence_after();
      // the tile's records are complete and read by S: the softmax waited for both
      const csa::Desc c_desc = c_descs.at((g & 1) * sizeof(S.c[0]));
#pragma unroll
      for (int d = 0; d < kDim / 128; ++d) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)  // the piece's first tile overwrites
          csa::mma_f16_ss(lead, tmem + d * kHeads, c_desc.at(2 * d * kColBytes + k * 2048), p_desc.at(32 * k), idesc, i > 0 || k > 0);
        if (d & 1) csa::mma_commit_if(lead, bars + 8 * (kBarCEmpty + 2 * (g & 1) + (d >> 1)));
      }
    }
  }
  csa::mma_commit_if(lead, bars + 8 * kBarDrainO);
  csa::mbar_wait_drain(bars + 8 * kBarDrainO, 0);
  __syncwarp();
}

// out from O^T: 32 heads x 128 values a step, a warp its 32 values (32 lanes of TMEM). They are read as 8 x 8
// matrices (values x heads), scaled and rounded, transposed on the way to shared memory (2 KB a warp of P's, which
// is not in use between a unit's last O and the next one's first P: head h at 64 h, its four 16-byte chunks
// exchanged by h / 2 so that neither side has two lanes on one bank), and written as 64 contiguous bytes a head.
// Lane exchanges and 4-byte stores took 7.5 k clocks a unit.
template <int kRope>
__device__ void write_out(const Kernel& K, Smem<kRope>& S, int unit, int heads, int warp, int lane) {
  const int b = row_of(K, unit), h0 = group_of(K, unit) * kHeads;
  const uint32_t stage = smem_u32(S.p) + 2048 * warp, lanes = static_cast<uint32_t>(32 * warp) << 16;
  uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(K.A.out) +
                                        (static_cast<int64_t>(b) * K.A.num_heads + h0) * kDim + 32 * warp + 8 * (lane & 3));
  const int row = lane & 7, chunk = lane >> 3;  // this lane's row of a matrix, and which of the four
#pragma unroll 1
  for (int hh = 0; hh < heads; hh += 32) {
    float2 alpha[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) alpha[i] = *reinterpret_cast<const float2*>(S.alpha + hh + 8 * i + 2 * (lane & 3));
#pragma unroll 1
    for (int d = 0; d < kDim / 128; ++d) {
      uint32_t v[2][16];  // values 0 .. 15 and 16 .. 31 of the warp's
      const uint32_t at = S.tmem + d * kHeads + hh + lanes;
      csa::tmem_ld_16x32(at, v[0]);
      csa::tmem_ld_16x32(at + (16u << 16), v[1]);
      csa::tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // heads hh + 8 i ..
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // values 8 k ..
          const uint32_t* x = v[k >> 1] + 4 * i + 2 * (k & 1);
          const __nv_bfloat162 two = __floats2bfloat162_rn(__uint_as_float(x[0]) * alpha[i].x, __uint_as_float(x[1]) * alpha[i].y);
          w[k] = *reinterpret_cast<const uint32_t*>(&two);
        }
        const int h = 8 * i + row;
        csa::stmatrix_x4_trans(stage + 64 * h + ((chunk ^ ((h >> 1) & 3)) << 4), w[0], w[1], w[2], w[3]);
      }
      __syncwarp();
      uint4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = 8 * i + (lane >> 2);
        x[i] = csa::ld_shared_v4(stage + 64 * h + (((lane & 3) ^ ((h >> 1) & 3)) << 4));
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = hh + 8 * i + (lane >> 2);
        if (h < heads) out[(h * kDim + 128 * d) / 8] = x[i];
      }
    }
  }
}

template <int kRope>
__device__ void write_part(const Kernel& K, Smem<kRope>& S, float* part, int heads, int warp, int lane) {
#pragma unroll 1
  for (int d = 0; d < kDim / 128; ++d) {
#pragma unroll 1
    for (int hh = 0; hh < heads; hh += 32) {
      uint32_t v[32];
      csa::tmem_ld32(S.tmem + d * kHeads + hh + (static_cast<uint32_t>(32 * warp) << 16), v);
      csa::tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; ++j) part[(hh + j) * kDim + 128 * d + 32 * warp + lane] = __uint_as_float(v[j]);
    }
  }
}

template <int kRope>
__device__ void role_softmax(const Kernel& K, Smem<kRope>& S) {
  const csa_latent_attend_args& A = K.A;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* stop = &S.abort;
  const uint32_t bars = smem_u32(S.bars);
  const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;  // this warp's TMEM lanes
  // S of 64 rows lies in lanes 0 .. 15 of each warp's 32: heads 16 warp .. 16 warp + 15. A thread holds
  // two heads' scores (head[0], head[0] + 8), a quarter of the tile's records each.
  const int head[2] = {16 * warp + (lane >> 2), 16 * warp + (lane >> 2) + 8};
  const int col = 2 * (lane & 3);  // its records: 8 i + col, 8 i + col + 1
  // where this lane's row of a group of four 8 x 8 matrices of P goes: matrices 0, 1 the heads' halves at
  // records 8 i, 2, 3 at records 8 (i + 1)
  const int p_head = 16 * warp + (lane & 15);
  const uint32_t p_row = smem_u32(S.p) + p_head * 128;
  const float c = A.scale * 1.4426950408889634f;
  const float grow = fminf(kGrow / c, FLT_MAX);  // finite also where the scale is almost nothing
  // O of the tile before tile g is complete: its second half is free (there is nothing before tile 0)
  auto o_done = [&](uint32_t tile) {
    return tile == 0 || warp_wait(bars + 8 * (kBarCEmpty + 2 * ((tile - 1) & 1) + 1), ((tile - 1) >> 1) & 1, stop);
  };
  uint32_t g = 0;
  bool ok = true;  // once a wait has run out, the rest runs through without waiting: all warps meet at every barrier
  for (Pieces run(K, S); run.more(); run.next(K)) {
    const int heads = min(A.num_heads - group_of(K, run.unit) * kHeads, kHeads);
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // l: this thread's share of the sum
    for (int i = 0; i < run.n; ++i, ++g) {
      ok = ok && warp_wait(bars + 8 * (kBarCFull + 2 * (g & 1)), (g >> 1) & 1, stop);
      const bool all = __all_sync(0xFFFFFFFFu, reinterpret_cast<const uint16_t*>(S.valid[g & 1])[lane] == 0x0101u);
      ok = ok && warp_wait(bars + 8 * (kBarSFull + (g & 1)), (g >> 1) & 1, stop);
      csa::tc_fence_after();
      uint32_t raw[32];
      csa::tmem_ld_16x64(S.tmem + kTmemS + (g & 1) * kTile + lanes, raw);
      csa::tmem_wait_ld();
      csa::tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (kBarSEmpty + (g & 1)));
      float s[2][16];
#pragma unroll
      for (int j = 0; j < 32; ++j) s[(j >> 1) & 1][2 * (j >> 2) + (j & 1)] = __uint_as_float(raw[j]);
      if (!all) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (!S.valid[g & 1][8 * (j >> 1) + col + (j & 1)]) s[0][j] = s[1][j] = -INFINITY;
      }
      float keep[2];
      bool up = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float top = s[r][0];
#pragma unroll
        for (int j = 1; j < 16; ++j) top = fmaxf(top, s[r][j]);
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        keep[r] = 1.f;
        if (top > m[r] + grow) {  // also when there was nothing (-infinity), not where there is still nothing
          up = true;
          keep[r] = csa::ex2((m[r] - top) * c);  // 0 when there was nothing
          m[r] = top;
          l[r] *= keep[r];
        }
      }
      if (i > 0 && csa::named_bar_any(kBarSoftmax, 32 * kSoftmaxWarps, up)) {
        if ((lane & 3) == 0) {
          S.alpha[head[0]] = keep[0];
          S.alpha[head[1]] = keep[1];
        }
        csa::named_bar_sync(kBarSoftmax, 32 * kSoftmaxWarps);
        ok = ok && o_done(g);  // O of the tile before is complete
        csa::tc_fence_after();
#pragma unroll 1
        for (int at = 0; at < kDim / 128 * kHeads; at += 32) {
          uint32_t v[32];
          csa::tmem_ld32(S.tmem + at + lanes, v);
          csa::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * S.alpha[(at & (kHeads - 1)) + j]);
          csa::tmem_st32(S.tmem + at + lanes, v);
        }
        csa::tmem_wait_st();
        csa::tc_fence_before();
        csa::named_bar_sync(kBarSoftmax, 32 * kSoftmaxWarps);  // alpha is free again
      }
      // p is rounded to bf16 here, the tensor cores' operand type; l sums it unrounded
      uint32_t w[2][8];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float ref = m[r] == -INFINITY ? 0.f : m[r], factor = exponent_factor(ref * c, c), mc = ref * factor;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float p0 = csa::ex2(fmaf(s[r][j], factor, -mc)), p1 = csa::ex2(fmaf(s[r][j + 1], factor, -mc));
          sum += p0 + p1;
          const __nv_bfloat162 two = __floats2bfloat162_rn(p0, p1);
          w[r][j >> 1] = *reinterpret_cast<const uint32_t*>(&two);
        }
        l[r] += sum;
      }
      ok = ok && o_done(g);
#pragma unroll
      for (int k = 0; k < 8; k += 2)
        csa::stmatrix_x4(p_row + (((k + (lane >> 4)) ^ (p_head & 7)) << 4), w[0][k], w[1][k], w[0][k + 1], w[1][k + 1]);
      csa::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * kBarPFull);
    }
    // the piece's output
    ok = ok && o_done(g);
    csa::tc_fence_after();
    float mc[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
      l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
      mc[r] = m[r] == -INFINITY ? -INFINITY : m[r] * c;
    }
    if (K.cluster) {  // joined by cluster_join, once all CTAs of the unit are here
      if ((lane & 3) == 0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          S.mc[head[r]] = mc[r];
          S.l[head[r]] = l[r];
        }
      }
      return;
    }
    if (run.n == run.tiles) {
      csa::named_bar_sync(kBarSoftmax, 32 * kSoftmaxWarps);
      if ((lane & 3) == 0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          S.alpha[head[r]] = l[r] > 0.f ? 1.f / l[r] : l[r];  // 0 for an empty row; a NaN stays one
          if (A.lse && head[r] < heads)
            A.lse[static_cast<int64_t>(row_of(K, run.unit)) * A.num_heads + group_of(K, run.unit) * kHeads + head[r]] =
                l[r] == 0.f ? -INFINITY : (mc[r] + log2f(l[r])) * 0.6931471805599453f;
        }
      }
      csa::named_bar_sync(kBarSoftmax, 32 * kSoftmaxWarps);
      write_out(K, S, run.unit, heads, warp, lane);
    } else {
      float* part = K.parts + (2 * blockIdx.x + (run.off == 0)) * kPartFloats;
      if ((lane & 3) == 0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          part[kHeads * kDim + head[r]] = mc[r];
          part[kHeads * (kDim + 1) + head[r]] = l[r];
        }
      }
      write_part(K, S, part, heads, warp, lane);
    }
    csa::tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * kBarOEmpty);
  }
}

// A part's weight 2^x, x <= 0: as a square, so that it becomes subnormal before it becomes 0 and how a
// row is split does not decide at which size its smallest terms vanish.
__device__ __forceinline__ float weight(float x) {
  const float h = csa::ex2(0.5f * x);
  return h * h;
}

// Joins a unit among its cluster's CTAs, each of which has seen a part of the tiles: CTA r finishes values
// 512 r / size .. of all heads (of 32 heads where size is 8). Everyone scales its O by its share of the
// softmax, 2^(m c - M c) / L, and writes the others' slices into their record tiles, which are free by
// now; sums go in the order of the ranks. Needs no workspace and no second launch.
template <int kMmaWarp, int kRope>
__device__ void cluster_join(const Kernel& K, Smem<kRope>& S) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t size = K.cluster, rank = blockIdx.x % size;
  const int heads = min(K.A.num_heads - group_of(K, S.unit) * kHeads, kHeads);
  const int64_t row = static_cast<int64_t>(row_of(K, S.unit)) * K.A.num_heads + group_of(K, S.unit) * kHeads;
  const int64_t tiles = S.total;
  csa::cluster_arrive();
  csa::cluster_wait();  // every CTA's m, l are there and its MMAs are done
  if (threadIdx.x < kHeads) {
    const int h = threadIdx.x;
    float top = -INFINITY, sum = 0.f;
    for (uint32_t r = 0; r < size; ++r) top = fmaxf(top, csa::ld_peer_f32(csa::peer_smem(smem_u32(&S.mc[h]), r)));
    const float ref = top == -INFINITY ? 0.f : top;
    for (uint32_t r = 0; r < size; ++r)
      sum = fmaf(csa::ld_peer_f32(csa::peer_smem(smem_u32(&S.l[h]), r)),
                 weight(csa::ld_peer_f32(csa::peer_smem(smem_u32(&S.mc[h]), r)) - ref), sum);
    S.alpha[h] = (sum > 0.f ? 1.f / sum : sum) * weight(S.mc[h] - ref);
    if (rank == 0 && K.A.lse && h < heads) K.A.lse[row + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
  }
  __syncthreads();
  // A step is 16 heads of a block of 128 values (as four by four heads in a CTA's inbox, a float4 a lane); step s of the
  // unit belongs to CTA s / per
  constexpr int kSteps = kDim / 128 * (kHeads / 16), kStepBytes = 16 * 128 * 4;
  const int per = kSteps / size;
  auto inbox = [&](uint32_t from, int s) {  // where CTA `from` puts its part of step s at the step's owner
    return smem_u32(S.c[0]) + static_cast<uint32_t>(from * per + s % per) * kStepBytes + 16 * (32 * (warp & 3) + lane);
  };
  const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  auto mine = [&](int s, float (&v)[16]) {
    const int d = s / (kHeads / 16), h = s % (kHeads / 16) * 16;
    uint32_t raw[16];
    csa::tmem_ld16(S.tmem + d * kHeads + h + lanes, raw);
    csa::tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = tiles > 0 ? __uint_as_float(raw[j]) * S.alpha[h + j] : 0.f;
  };
  if (warp < kMmaWarp) {  // two or three warps a lane quarter
    for (int s = warp >> 2; s < kSteps; s += kMmaWarp / 4) {
      const uint32_t owner = s / per;
      if (owner == rank || s % (kHeads / 16) * 16 >= heads) continue;
      float v[16];
      mine(s, v);
      const uint32_t at = csa::peer_smem(inbox(rank, s), owner);
#pragma unroll
      for (int j = 0; j < 4; ++j) csa::st_peer_v4(at + 2048 * j, v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
  }
  csa::cluster_arrive();
  csa::cluster_wait();
  if (warp < kMmaWarp) {
    const int odd = lane & 1;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(K.A.out) + (row + odd) * kDim + 32 * (warp & 3) + (lane & ~1);
    for (int s = static_cast<int>(rank) * per + (warp >> 2); s < static_cast<int>(rank + 1) * per; s += kMmaWarp / 4) {
      const int d = s / (kHeads / 16), h = s % (kHeads / 16) * 16;
      if (h >= heads) continue;
      float own[16], v[16] = {};
      mine(s, own);
      for (uint32_t r = 0; r < size; ++r) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float4 x = make_float4(own[4 * j], own[4 * j + 1], own[4 * j + 2], own[4 * j + 3]);
          if (r != rank) {
            const uint4 y = csa::ld_shared_v4(inbox(r, s) + 2048 * j);
            x = make_float4(__uint_as_float(y.x), __uint_as_float(y.y), __uint_as_float(y.z), __uint_as_float(y.w));
          }
          v[4 * j] += x.x;
          v[4 * j + 1] += x.y;
          v[4 * j + 2] += x.z;
          v[4 * j + 3] += x.w;
        }
      }
      // two heads at a time: even lanes end with values (lane, lane + 1) of the first, odd lanes with values
      // (lane - 1, lane) of the second
      uint32_t two[8];
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[j] : v[j + 1], 1);
        const __nv_bfloat162 pair = __floats2bfloat162_rn(odd ? got : v[j], odd ? v[j + 1] : got);
        two[j / 2] = *reinterpret_cast<const uint32_t*>(&pair);
      }
#pragma unroll
      for (int j = 0; j < 16; j += 2)
        if (h + j + odd < heads) *reinterpret_cast<uint32_t*>(out + static_cast<int64_t>(h + j) * kDim + 128 * d) = two[j / 2];
    }
  }
}

template <int kLoad>
struct MapsFor {
  using type = int;  // none
};
template <>
struct MapsFor<kLoadTma> {
  using type = Maps;
};
template <int kLoad>
using MapsOf = typename MapsFor<kLoad>::type;

template <int kLoad, int kRope>
__global__ void __launch_bounds__(Warps<kLoad>::kThreads, 1)
    attend_kernel(const __grid_constant__ Kernel K, const __grid_constant__ MapsOf<kLoad> M) {
  constexpr int kMmaWarp = Warps<kLoad>::kMma, kFills = Warps<kLoad>::kFills, kThreads = Warps<kLoad>::kThreads;
  extern __shared__ uint8_t smem_raw[];
  Smem<kRope>& S = *reinterpret_cast<Smem<kRope>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ int64_t scan[kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = smem_u32(S.bars);
  if (threadIdx.x == 0) {
    for (int k = 0; k < 4; ++k) {
      csa::mbar_init(bars + 8 * (kBarCFull + k), kFills);
      csa::mbar_init(bars + 8 * (kBarCEmpty + k), 1);
    }
    for (int k = 0; k < 2; ++k) {
      csa::mbar_init(bars + 8 * (kBarSFull + k), 1);
      csa::mbar_init(bars + 8 * (kBarSEmpty + k), kSoftmaxWarps);
    }
    csa::mbar_init(bars + 8 * kBarQFull, kFills);
    csa::mbar_init(bars + 8 * kBarLand, 1);
    csa::mbar_init(bars + 8 * kBarQEmpty, 1);
    csa::mbar_init(bars + 8 * kBarPFull, kSoftmaxWarps);
    csa::mbar_init(bars + 8 * kBarOEmpty, kSoftmaxWarps);
    csa::mbar_init(bars + 8 * kBarDrainS, 1);
    csa::mbar_init(bars + 8 * kBarDrainO, 1);
    csa::mbar_init_fence();
    S.abort = 0;
  }
  if (threadIdx.x < kHeads) {  // of a CTA without tiles
    S.mc[threadIdx.x] = -INFINITY;
    S.l[threadIdx.x] = 0.f;
  }
  if (warp == kMmaWarp) {
    csa::tmem_alloc(smem_u32(&S.tmem), kTmemCols);
    csa::tmem_relinquish();
  }
  csa::tc_fence_before();
  make_plan<kThreads>(K, S, scan);  // ends with a block barrier
  csa::tc_fence_after();
  int32_t flags = 0;
  if (warp < kSoftmaxWarps) {
    role_softmax(K, S);
  } else if (warp < kMmaWarp) {
    if constexpr (kLoad != kLoadTma) role_load_regs<kLoad == kLoadFp4, kRope>(K, S, &flags);
    else if (warp == kSoftmaxWarps) role_load_tma(K, M, S, &flags);
  } else {
    if (warp == kMmaWarp) {
      role_mma_s(K, S);
    } else {
      if (lane == 0 && !K.cluster) write_opens(K, S);
      __syncwarp();
      role_mma_o(K, S);
    }
  }
  csa::tc_fence_before();
  __syncthreads();
  if (K.cluster) {
    csa::tc_fence_after();
    cluster_join<kMmaWarp>(K, S);
    csa::tc_fence_before();
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    csa::tc_fence_after();
    csa::tmem_dealloc(S.tmem, kTmemCols);
  }
  if (threadIdx.x == 0 && S.abort) flags |= CSA_DEV_TIMEOUT;
  flags = static_cast<int32_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(flags)));
  if (flags && K.A.dev_status && lane == 0) atomicOr(K.A.dev_status, flags);
}

// Joins a cut unit. Its parts are those of run `o.run` (which ends inside the unit) and of the runs after it up to the
// unit's end, added in that order (by eight warps: each every eighth, then the warps' sums in their order), so the
// result does not depend on timing. Launched as a programmatic dependent of the attention kernel: its blocks are in
// place when that one ends. kJoinWarps a head where a unit has many parts; one a head where it has a few (2048
// units of 8 tiles: 39 us with eight, most of them idle).
constexpr int kJoinWarps = 8;
template <bool kMany>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const Kernel K, int grid) {
  const csa_latent_attend_args& A = K.A;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int head = kMany ? blockIdx.y : blockIdx.y * kJoinWarps + warp;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Open o = K.opens[blockIdx.x];
  const int h = group_of(K, o.unit) * kHeads + head;
  if (!o.cut || (kMany && h >= A.num_heads)) return;
  // runs o.run .. last; a run without tiles has no part
  const int64_t end = o.begin + o.tiles;
  int last = static_cast<int>(min((end * grid - 1) / o.total, static_cast<int64_t>(grid) - 1)) + 1;
  while (last >= grid || run_start(o.total, last, grid) >= end) --last;
  if (h >= A.num_heads) return;
  auto part_of = [&](int r) { return K.parts + (2 * static_cast<int64_t>(r) + (r == o.run)) * kPartFloats; };
  auto there = [&](int r) { return r <= last && run_start(o.total, r, grid) < run_start(o.total, r + 1, grid); };
  float top = -INFINITY;
  for (int r = o.run + lane; r <= last; r += 32)
    if (there(r)) top = fmaxf(top, part_of(r)[kHeads * kDim + head]);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, k));
  float l = 0.f;
  float4 v[4] = {};
  const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll 2
  for (int r = o.run + (kMany ? warp : 0); r <= last; r += kMany ? kJoinWarps : 1) {
    if (!there(r)) continue;
    const float* part = part_of(r);
    const float4* x = reinterpret_cast<const float4*>(part + head * kDim);
    const float w = weight(part[kHeads * kDim + head] - ref);
    l = fmaf(part[kHeads * (kDim + 1) + head], w, l);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 y = x[lane + 32 * k];
      v[k] = make_float4(fmaf(y.x, w, v[k].x), fmaf(y.y, w, v[k].y), fmaf(y.z, w, v[k].z), fmaf(y.w, w, v[k].w));
    }
  }
  const int64_t row = static_cast<int64_t>(row_of(K, o.unit)) * A.num_heads + h;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(A.out) + row * kDim;
  if constexpr (kMany) {
    __shared__ float s_o[kJoinWarps][kDim], s_l[kJoinWarps];
#pragma unroll
    for (int k = 0; k < 4; ++k) reinterpret_cast<float4*>(s_o[warp])[lane + 32 * k] = v[k];
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    l = 0.f;
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float2 y = reinterpret_cast<const float2*>(s_o[w])[threadIdx.x];
      sum.x += y.x;
      sum.y += y.y;
      l += s_l[w];
    }
    const float inv = l > 0.f ? 1.f / l : l;
    reinterpret_cast<__nv_bfloat162*>(out)[threadIdx.x] = __floats2bfloat162_rn(sum.x * inv, sum.y * inv);
  } else {
    const float inv = l > 0.f ? 1.f / l : l;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v[k].x * inv, v[k].y * inv), b = __floats2bfloat162_rn(v[k].z * inv, v[k].w * inv);
      reinterpret_cast<uint2*>(out)[lane + 32 * k] = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
  }
  if (A.lse && (kMany ? threadIdx.x : lane) == 0) A.lse[row] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
}

// CTAs of the call: one an SM, fewer when there cannot be as many tiles.
int grid_cap(const csa_latent_attend_args* a) {
  const int64_t groups = (a->num_heads + kHeads - 1) / kHeads;
  const int64_t per = a->idx ? (a->top + kTile - 1) / kTile : (a->pt_stride > 0 ? a->pt_stride : 1);
  const int64_t units = a->num_q * groups;
  return static_cast<int>(units > kMaxGrid || per > kMaxGrid || units * per > kMaxGrid ? kMaxGrid : units * per);
}

constexpr size_t kOpenBytes = (kMaxGrid * sizeof(Open) + 255) / 256 * 256;

// CTAs that share a unit: where every unit is short (8 tiles a CTA at most) and there are fewer units than
// SMs, the largest power of two up to 8 that still fits the SMs; else 0, the runs. How long a unit can be is all that the
// host knows: the table's width, or the number of positions. In a graph, L2 cold: 64 rows of 8 tiles take 31.8 us in
// clusters of two, 38.0 us cut into 152 runs (whose parts are 28 MB, against 38 MB of records), in two launches; one row
// of 16 tiles is the other way round, 23.7 us in a cluster of eight and 19.6 us in 16 runs.
int cluster_of(const csa_latent_attend_args* a, int sms) {
  const int64_t units = static_cast<int64_t>(a->num_q) * ((a->num_heads + kHeads - 1) / kHeads);
  const int64_t per = a->idx ? (a->top + kTile - 1) / kTile : a->pt_stride;
  if (units > sms) return 0;
  int size = 1;
  while (size < 8 && 2 * size * units <= sms && size < per) size *= 2;
  return per <= 8 * size ? size : 0;
}

template <int kLoad, int kRope>
csa_status launch(const Kernel& K, const MapsOf<kLoad>& M, int grid, int dev, cudaStream_t stream) {
  static Kept ready;  // the kernel's shared memory size is set on each device once
  constexpr size_t smem = sizeof(Smem<kRope>) + 1024;
  static_assert(smem + 256 <= 232448, "shared memory of one CTA");
  if (!ready.get(dev)) {
    if (cudaFuncSetAttribute(attend_kernel<kLoad, kRope>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess)
      return CSA_ERR_CUDA;
    ready.set(dev, 1);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Warps<kLoad>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {static_cast<unsigned>(K.cluster ? K.cluster : 1), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_kernel<kLoad, kRope>, K, M) == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

// Whole histories of bf16 records go through TMA where the cache's pages are a tensor of 128-byte columns (pages that
// are not padded, or by such columns): long rows 112 us with L2 cold, 118 through registers. Listed positions do not (gathered
// four rows a copy, 64 rows of 512 positions took 47 us where registers took 28), nor do short units in a cluster, whose few
// tiles do not pay for the maps (one row of 1000 records: 20.8 us where registers took 17.4).
template <int kRope>
csa_status launch_bf16(const Kernel& K, int grid, int dev, cudaStream_t stream) {
  const csa_latent_attend_args& a = K.A;
  constexpr int64_t kRec = record_bytes(false, kRope);
  const int64_t stride = a.cache.page_stride_bytes;
  if (a.idx || K.cluster || stride % 128 != 0) return launch<kLoadBf16, kRope>(K, 0, grid, dev, stream);
  Maps M;
  const cuuint64_t page_dims[4] = {64, static_cast<cuuint64_t>(kRec / 128), kPageRecs, static_cast<cuuint64_t>(a.cache.num_pages)};
  const cuuint64_t page_strides[3] = {128, static_cast<cuuint64_t>(kRec), static_cast<cuuint64_t>(stride)};
  const cuuint32_t page_boxes[4] = {64, 1, kPageRecs, 1};
  if (!encode_bf16(&M.q, a.q, kDim + kRope, a.num_heads, a.num_q, a.q_head_stride, a.q_row_stride, kHeads, 1) ||
      !encode_map(&M.pages, a.cache.pages, 4, page_dims, page_strides, page_boxes))
    return CSA_ERR_INVALID_ARG;
  return launch<kLoadTma, kRope>(K, M, grid, dev, stream);
}

csa_status check_args(const csa_latent_attend_args* a) {
  if (!a || a->num_q < 0 || a->num_req < 0 || a->pt_stride < 0 || a->top < 0) return CSA_ERR_INVALID_ARG;
  if (a->num_heads < 1 || a->num_heads > CSA_LATENT_MAX_HEADS) return CSA_ERR_UNSUPPORTED;
  if (!good_scale(a->scale)) return CSA_ERR_INVALID_ARG;
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
  if (!a || a->num_q < 0 || a->num_heads < 1 || a->num_heads > CSA_LATENT_MAX_HEADS || a->pt_stride < 0 || a->top < 0) return 0;
  if (a->num_q > 0 && (a->pt_stride < 1 || (a->idx != nullptr) != (a->top > 0))) return 0;
  return kOpenBytes + 2 * static_cast<size_t>(grid_cap(a)) * kPartFloats * sizeof(float);
}

extern "C" csa_status csa_latent_attend(const csa_latent_attend_args* a, void* ws, size_t ws_bytes, void* stream) {
  const csa_status st = check_args(a);
  if (st != CSA_OK) return st;
  if (a->num_q == 0) return CSA_OK;
  if (!ws || ws_bytes < csa_latent_attend_workspace_bytes(a)) return CSA_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return CSA_ERR_ALIGNMENT;
  const int groups = (a->num_heads + kHeads - 1) / kHeads;
  const int64_t units = static_cast<int64_t>(a->num_q) * groups;
  if (units > INT32_MAX) return CSA_ERR_INVALID_ARG;
  int sms = 0, dev = 0;
  if (sm_count(&sms, &dev) != CSA_OK) return CSA_ERR_CUDA;
  Kernel K;
  K.A = *a;
  K.cluster = cluster_of(a, sms);
  const int cap = K.cluster ? static_cast<int>(units) * K.cluster : grid_cap(a);
  const int grid = cap < sms ? cap : sms;
  K.groups = groups;
  K.by_unit = units <= grid;
  K.opens = static_cast<Open*>(ws);
  K.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kOpenBytes);
  const auto s = static_cast<cudaStream_t>(stream);
  const bool fp4 = a->cache.record_format == CSA_LATENT_MXFP4, rope = a->cache.rope_dim != 0;
  const csa_status ls = fp4 ? (rope ? launch<kLoadFp4, 64>(K, 0, grid, dev, s) : launch<kLoadFp4, 0>(K, 0, grid, dev, s))
                            : (rope ? launch_bf16<64>(K, grid, dev, s) : launch_bf16<0>(K, grid, dev, s));
  if (ls != CSA_OK || grid == 1 || K.cluster) return ls;
  cudaLaunchConfig_t cfg = {};
  const bool many = units * kJoinWarps < grid;  // parts a unit, on average
  const int heads = a->num_heads < kHeads ? a->num_heads : kHeads;
  cfg.gridDim = dim3(K.by_unit ? static_cast<unsigned>(units) : grid, many ? heads : (heads + kJoinWarps - 1) / kJoinWarps);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, many ? join_kernel<true> : join_kernel<false>, K, grid) == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}
