// csa_latent_cache.cu — block tables and slot maps, the latent cache's writer and
// its reader (include/csa_latent.h). All three only move and re-encode data.
#include "csa_latent_rows.cuh"

namespace csa_latent {
namespace {

// ------------------------------------------------------------- block tables
//
// One launch: every block takes the running sums over all requests for itself
// (num_req is at most CSA_TABLES_MAX_REQ, three words a request in shared memory),
// so no block waits for another, then does its share of the new pages and of the
// rows, each found by bisection in the running sums. A row's page is looked up in
// the old entries of the table or in the free list, never in an entry that this
// launch writes. 509 requests and a million rows: 11.2 us in a graph, of which 3.2 us are the bytes; the call costs the host more.

constexpr int kTabThreads = 512;
constexpr int kTabRowsPerBlock = 2048;  // rows a block is launched for

struct Scan3 {
  int64_t rows, kv, fresh;
};

__device__ __forceinline__ Scan3 operator+(Scan3 a, Scan3 b) { return {a.rows + b.rows, a.kv + b.kv, a.fresh + b.fresh}; }

__device__ __forceinline__ Scan3 shfl_up(Scan3 v, int o) {
  return {__shfl_up_sync(0xFFFFFFFFu, v.rows, o), __shfl_up_sync(0xFFFFFFFFu, v.kv, o),
          __shfl_up_sync(0xFFFFFFFFu, v.fresh, o)};
}

// Lengths of request r cut to the table; *bad is set when they had to be.
__device__ __forceinline__ void request_lengths(const csa_tables_args& A, int r, int64_t* old_len, int64_t* new_len,
                                                bool* bad) {
  const int64_t cap = static_cast<int64_t>(kPageRecs) * A.pt_stride;
  const int64_t o = A.old_len[r], n = A.new_len[r];
  const int64_t oc = min(max(o, int64_t(0)), cap), nc = min(max(n, int64_t(0)), cap - oc);
  *bad |= oc != o || nc != n;
  *old_len = oc;
  *new_len = nc;
}

__device__ __forceinline__ int64_t pages_of(int64_t n) { return (n + kPageRecs - 1) / kPageRecs; }

__device__ __forceinline__ int32_t held(int64_t v, bool* bad) {  // a running sum as int32
  if (v <= INT32_MAX) return static_cast<int32_t>(v);
  *bad = true;
  return INT32_MAX;
}

// The last index k in [0, n) with a[k] <= v (a ascending, a[0] = 0 <= v).
__device__ __forceinline__ int last_not_above(const int32_t* a, int n, int32_t v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTabThreads) build_tables_kernel(const csa_tables_args A) {
  extern __shared__ int32_t tab_smem[];
  int32_t* s_row = tab_smem;                   // [num_req + 1] running sum of new records
  int32_t* s_fresh = tab_smem + A.num_req + 1;  // [num_req + 1] running sum of new pages
  int32_t* s_old = tab_smem + 2 * (A.num_req + 1);  // [num_req] old lengths
  __shared__ Scan3 s_warp[kTabThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (A.num_req + kTabThreads - 1) / kTabThreads;
  const int r0 = min(tid * per, A.num_req), r1 = min(r0 + per, A.num_req);
  bool bad_len = false;
  Scan3 mine = {0, 0, 0};
  for (int r = r0; r < r1; ++r) {
    int64_t o, n;
    request_lengths(A, r, &o, &n, &bad_len);
    mine = mine + Scan3{n, o + n, pages_of(o + n) - pages_of(o)};
  }
  Scan3 incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Scan3 up = shfl_up(incl, o);
    if (lane >= o) incl = incl + up;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  Scan3 at = {incl.rows - mine.rows, incl.kv - mine.kv, incl.fresh - mine.fresh};
  for (int w = 0; w < warp; ++w) at = at + s_warp[w];
  const bool first = blockIdx.x == 0;
  for (int r = r0; r < r1; ++r) {
    int64_t o, n;
    bool ignore = false;
    request_lengths(A, r, &o, &n, &ignore);
    s_row[r] = held(at.rows, &bad_len);
    s_fresh[r] = held(at.fresh, &bad_len);
    s_old[r] = static_cast<int32_t>(o);
    if (first) {
      A.row_start[r] = s_row[r];
      A.kv_start[r] = held(at.kv, &bad_len);
    }
    at = at + Scan3{n, o + n, pages_of(o + n) - pages_of(o)};
  }
  if (tid == kTabThreads - 1) {
    s_row[A.num_req] = held(at.rows, &bad_len);
    s_fresh[A.num_req] = held(at.fresh, &bad_len);
    if (first) {
      A.row_start[A.num_req] = s_row[A.num_req];
      A.kv_start[A.num_req] = held(at.kv, &bad_len);
      A.taken[0] = static_cast<int32_t>(min(at.fresh, A.n_free));
    }
  }
  __syncthreads();
  int32_t flags = bad_len ? CSA_DEV_LEN_OOB : 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kTabThreads;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kTabThreads + tid;
  const int32_t total_fresh = s_fresh[A.num_req], total_rows = s_row[A.num_req];
  if (total_fresh > A.n_free) flags |= CSA_DEV_POOL;
  if (total_rows > A.n_rows) flags |= CSA_DEV_ROWS;
  for (int64_t j = i0; j < total_fresh; j += step) {
    const int r = last_not_above(s_fresh, A.num_req, static_cast<int32_t>(j));
    A.page_table[static_cast<int64_t>(r) * A.pt_stride + pages_of(s_old[r]) + (j - s_fresh[r])] =
        j < A.n_free ? A.free_pages[j] : -1;
  }
  for (int64_t i = i0; i < A.n_rows; i += step) {
    int32_t req = 0, pos = -1;
    int64_t slot = -1;
    if (i < total_rows) {
      req = last_not_above(s_row, A.num_req, static_cast<int32_t>(i));
      const int64_t o = s_old[req];
      pos = static_cast<int32_t>(o + (i - s_row[req]));
      const int64_t p = pos / kPageRecs, a = pages_of(o), j = s_fresh[req] + (p - a);
      int32_t page = -1;
      if (p < a) {
        page = A.page_table[static_cast<int64_t>(req) * A.pt_stride + p];
        if (page < 0) flags |= CSA_DEV_PAGE_OOB;
      } else if (j < A.n_free) {
        page = A.free_pages[j];
        if (page < 0) flags |= CSA_DEV_PAGE_OOB;
      }
      if (page >= 0) slot = static_cast<int64_t>(page) * kPageRecs + pos % kPageRecs;
    }
    A.row_req[i] = req;
    A.row_pos[i] = pos;
    A.row_len[i] = pos + 1;
    A.row_slot[i] = slot;
  }
  flags = static_cast<int32_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(flags)));
  if (flags && A.dev_status && lane == 0) atomicOr(A.dev_status, flags);
}

// ------------------------------------------------------------- writer
//
// A warp stores kRowsInFlight rows at a time, their loads all issued first: lane l holds the 16 latent
// values 16 l .. 16 l + 15 (half a 32-value block, so a block's amax takes one exchange with the
// neighbour lane) and the rope values 2 l, 2 l + 1. Rows are read once, coalesced. Bound by HBM:
// 65537 fp32 rows stored in 4 bits and read back (two launches, 279 MB) take 53 us, 5.3 TB/s.

template <bool kBf16In, bool kFp4>
__device__ __forceinline__ int32_t store_row(const csa_latent_write_args& A, const RowIn<kBf16In>& x, int64_t slot, int lane) {
  if (slot == -1) return 0;
  if (slot < 0 || slot >= A.cache.num_pages * kPageRecs) return CSA_DEV_PAGE_OOB;
  const uint32_t rope_word = pack_bf16(x.r[0], x.r[1]);
  const Coded<kFp4> c = encode<kFp4>(x.v);
  if (__any_sync(0xFFFFFFFFu, c.bad || nonfinite_bf16x2(rope_word))) return CSA_DEV_RANGE;
  put_record<kFp4>(A.cache, slot, c, rope_word, lane);
  return 0;
}

template <bool kBf16In, bool kFp4>
__global__ void __launch_bounds__(kCopyThreads) latent_write_kernel(const csa_latent_write_args A) {
  constexpr int kRowsInFlight = kBf16In ? 4 : 2;
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kCopyThreads / 32);
  int32_t flags = 0;
  // rows warp, warp + warps, ...: a small call spreads over the SMs
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x) >> 5; i < A.n; i += kRowsInFlight * warps) {
    int64_t slot[kRowsInFlight];
    RowIn<kBf16In> x[kRowsInFlight];
#pragma unroll
    for (int k = 0; k < kRowsInFlight; ++k) {
      const int64_t r = i + k * warps, at = r < A.n ? r : i;
      slot[k] = r < A.n ? A.slots[r] : -1;
      x[k].load(static_cast<const uint8_t*>(A.x) + at * A.x_stride * (kBf16In ? 2 : 4), lane, A.cache.rope_dim);
    }
#pragma unroll
    for (int k = 0; k < kRowsInFlight; ++k) flags |= store_row<kBf16In, kFp4>(A, x[k], slot[k], lane);
  }
  if (flags && A.dev_status && lane == 0) atomicOr(A.dev_status, flags);
}

// ------------------------------------------------------------- reader
//
// A warp reads kReadRows neighbouring rows at a time: lane r < kReadRows finds row r's record (its request by
// bisection, its page), then all lanes copy, many 16-byte pieces in flight. Bound by HBM: 3 histories
// of up to 16384 bf16 records (79 MB) take 16.5 us, 4.8 TB/s, of which 3 us are launch and ramp.

constexpr int kReadRows = 4;  // with 8, a 16384-row history is 1.2 waves of blocks

// Row i's record: 0 where no request covers the row, 1 where the row becomes zeros.
__device__ __forceinline__ uintptr_t record_of_row(const csa_latent_read_args& A, int64_t i, int rec_bytes, int32_t* flags) {
  if (i >= A.n_rows) return 0;
  int lo = 0, hi = A.num_req;  // the last request that starts at or before row i
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (A.kv_start[mid] <= i) lo = mid;
    else hi = mid;
  }
  const int64_t begin = A.kv_start[lo], end = A.kv_start[lo + 1], pos = i - begin;
  if (begin < 0 || i < begin || i >= end) return 0;
  if (pos >= static_cast<int64_t>(kPageRecs) * A.pt_stride) {
    *flags |= CSA_DEV_LEN_OOB;
    return 1;
  }
  const int32_t page = A.page_table[static_cast<int64_t>(lo) * A.pt_stride + pos / kPageRecs];
  if (page < 0 || page >= A.cache.num_pages) {
    *flags |= CSA_DEV_PAGE_OOB;
    return 1;
  }
  return reinterpret_cast<uintptr_t>(A.cache.pages + page * A.cache.page_stride_bytes + (pos % kPageRecs) * rec_bytes);
}

// bf16 records: 16 bytes to 16 bytes.
template <int kRope>
__device__ __forceinline__ void copy_rows(uintptr_t mine, uint8_t* out, int lane) {
  constexpr int kChunks = 2 * (kDim + kRope) / 16, kAll = kReadRows * kChunks / 32;
  uint4 w[kAll];
  uintptr_t rec[kAll];
#pragma unroll
  for (int k = 0; k < kAll; ++k) {
    const int at = 32 * k + lane;
    rec[k] = __shfl_sync(0xFFFFFFFFu, mine, at / kChunks);
    w[k] = rec[k] > 1 ? __ldg(reinterpret_cast<const uint4*>(rec[k]) + at % kChunks) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int k = 0; k < kAll; ++k)
    if (rec[k]) reinterpret_cast<uint4*>(out)[32 * k + lane] = w[k];
}

// MXFP4 records: lane l decodes values 8 l .. 8 l + 7 and the same of the second half (4 code bytes to 16 each), and
// copies rope values 2 l, 2 l + 1, so that every load and store of the warp is one contiguous piece.
template <int kRope>
__device__ __forceinline__ void decode_rows(uintptr_t mine, uint8_t* out, int lane) {
  uintptr_t rec[kReadRows];
  uint32_t code[kReadRows][2], scale[kReadRows][2], rope[kReadRows];
#pragma unroll
  for (int k = 0; k < kReadRows; ++k) {
    rec[k] = __shfl_sync(0xFFFFFFFFu, mine, k);
    const uint8_t* p = reinterpret_cast<const uint8_t*>(rec[k]);
    const bool live = rec[k] > 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      code[k][h] = live ? __ldg(reinterpret_cast<const uint32_t*>(p) + 32 * h + lane) : 0u;
      scale[k][h] = live ? __ldg(p + kCodeBytes + 8 * h + (lane >> 2)) : 0u;
    }
    rope[k] = live && kRope != 0 ? __ldg(reinterpret_cast<const uint32_t*>(p + kCodeBytes + kScaleBytes) + lane) : 0u;
  }
#pragma unroll
  for (int k = 0; k < kReadRows; ++k) {
    if (!rec[k]) continue;
    uint8_t* row = out + k * (2 * (kDim + kRope));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float s = ue8m0(scale[k][h]);
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2_raw r = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>((code[k][h] >> (8 * j)) & 0xFFu), __NV_E2M1);
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&r));
        w[j] = pack_bf16(v.x * s, v.y * s);  // exact: two significant bits times a power of two
      }
      reinterpret_cast<uint4*>(row)[32 * h + lane] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (kRope != 0) reinterpret_cast<uint32_t*>(row)[kDim / 2 + lane] = rope[k];
  }
}

template <bool kFp4, int kRope>
__global__ void __launch_bounds__(kCopyThreads) latent_read_kernel(const csa_latent_read_args A) {
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kCopyThreads / 32) * kReadRows;
  int32_t flags = 0;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; r < A.num_req;
       r += static_cast<int64_t>(gridDim.x) * kCopyThreads)
    if (A.kv_start[r] < 0 || A.kv_start[r + 1] < A.kv_start[r]) flags |= CSA_DEV_LEN_OOB;
  for (int64_t i = ((static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x) >> 5) * kReadRows; i < A.n_rows; i += step) {
    const uintptr_t mine = lane < kReadRows ? record_of_row(A, i + lane, record_bytes(kFp4, kRope), &flags) : 0;
    uint8_t* out = static_cast<uint8_t*>(A.out) + i * (2 * (kDim + kRope));
    if constexpr (kFp4) decode_rows<kRope>(mine, out, lane);
    else copy_rows<kRope>(mine, out, lane);
  }
  flags = static_cast<int32_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(flags)));
  if (flags && A.dev_status && lane == 0) atomicOr(A.dev_status, flags);
}

template <bool kBf16In, bool kFp4>
csa_status launch_write(const csa_latent_write_args& a, cudaStream_t stream) {
  static Kept kept;
  unsigned grid = 1;
  const csa_status st = wave_grid(latent_write_kernel<kBf16In, kFp4>, kCopyThreads, 0, &kept, a.n, kCopyThreads / 32, &grid);
  if (st != CSA_OK) return st;
  latent_write_kernel<kBf16In, kFp4><<<grid, kCopyThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

template <bool kFp4, int kRope>
csa_status launch_read(const csa_latent_read_args& a, cudaStream_t stream) {
  static Kept kept;
  unsigned grid = 1;
  const csa_status st =
      wave_grid(latent_read_kernel<kFp4, kRope>, kCopyThreads, 0, &kept, a.n_rows, kCopyThreads / 32 * kReadRows, &grid);
  if (st != CSA_OK) return st;
  latent_read_kernel<kFp4, kRope><<<grid, kCopyThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

}  // namespace
}  // namespace csa_latent

using namespace csa_latent;

extern "C" int32_t csa_latent_abi_version(void) { return CSA_LATENT_ABI_VERSION; }

extern "C" int64_t csa_latent_record_bytes(int32_t record_format, int32_t rope_dim) {
  if ((record_format != CSA_LATENT_BF16 && record_format != CSA_LATENT_MXFP4) || (rope_dim != 0 && rope_dim != 64))
    return 0;
  return record_bytes(record_format == CSA_LATENT_MXFP4, rope_dim);
}

extern "C" csa_status csa_build_tables(const csa_tables_args* a, void* stream) {
  if (!a || a->num_req < 0 || a->pt_stride < 0 || a->n_free < 0 || a->n_rows < 0) return CSA_ERR_INVALID_ARG;
  if (a->num_req > CSA_TABLES_MAX_REQ) return CSA_ERR_UNSUPPORTED;
  if (!a->row_start || !a->kv_start || !a->taken) return CSA_ERR_INVALID_ARG;
  if (a->num_req > 0 && (!a->old_len || !a->new_len || !a->page_table || a->pt_stride < 1)) return CSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(kPageRecs) * a->pt_stride > INT32_MAX) return CSA_ERR_INVALID_ARG;
  if ((a->n_free > 0 && !a->free_pages) ||
      (a->n_rows > 0 && (!a->row_req || !a->row_pos || !a->row_len || !a->row_slot)))
    return CSA_ERR_INVALID_ARG;
  if (!aligned(a->old_len, 4) || !aligned(a->new_len, 4) || !aligned(a->page_table, 4) || !aligned(a->free_pages, 4) ||
      !aligned(a->row_req, 4) || !aligned(a->row_pos, 4) || !aligned(a->row_len, 4) || !aligned(a->row_slot, 8) ||
      !aligned(a->row_start, 4) || !aligned(a->kv_start, 4) || !aligned(a->taken, 4) || !aligned(a->dev_status, 4))
    return CSA_ERR_ALIGNMENT;
  const size_t smem = 3 * sizeof(int32_t) * (static_cast<size_t>(a->num_req) + 1);
  static Kept ready;
  if (smem > 48 * 1024) {  // the limit is the kernel's, not the call's: set to what the most requests need, never lowered
    int sms = 0, dev = 0;
    if (sm_count(&sms, &dev) != CSA_OK) return CSA_ERR_CUDA;
    constexpr int most = 3 * sizeof(int32_t) * (CSA_TABLES_MAX_REQ + 1);
    if (!ready.get(dev)) {
      if (cudaFuncSetAttribute(build_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) return CSA_ERR_CUDA;
      ready.set(dev, 1);
    }
  }
  static Kept kept;  // of calls of up to about 1000 requests
  unsigned grid = 1;
  const csa_status st = wave_grid(build_tables_kernel, kTabThreads, smem < 12288 ? 12288 : smem, smem <= 12288 ? &kept : nullptr,
                                  a->n_rows + a->num_req, kTabRowsPerBlock, &grid);
  if (st != CSA_OK) return st;
  build_tables_kernel<<<grid, kTabThreads, smem, static_cast<cudaStream_t>(stream)>>>(*a);
  return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

extern "C" csa_status csa_latent_write(const csa_latent_write_args* a, void* stream) {
  if (!a || a->n < 0 || a->reserved0 != 0 || (a->dtype != CSA_KEYS_F32 && a->dtype != CSA_KEYS_BF16))
    return CSA_ERR_INVALID_ARG;
  if (a->n == 0) return CSA_OK;
  const csa_status st = check_cache(a->cache);
  if (st != CSA_OK) return st;
  const bool bf16 = a->dtype == CSA_KEYS_BF16;
  if (!a->x || !a->slots || a->x_stride < kDim + a->cache.rope_dim) return CSA_ERR_INVALID_ARG;
  if (!aligned(a->x, 16) || a->x_stride % (bf16 ? 8 : 4) != 0 || !aligned(a->slots, 8) || !aligned(a->dev_status, 4))
    return CSA_ERR_ALIGNMENT;
  const bool fp4 = a->cache.record_format == CSA_LATENT_MXFP4;
  const auto s = static_cast<cudaStream_t>(stream);
  if (bf16) return fp4 ? launch_write<true, true>(*a, s) : launch_write<true, false>(*a, s);
  return fp4 ? launch_write<false, true>(*a, s) : launch_write<false, false>(*a, s);
}

extern "C" csa_status csa_latent_read(const csa_latent_read_args* a, void* stream) {
  if (!a || a->n_rows < 0 || a->num_req < 0 || a->pt_stride < 0) return CSA_ERR_INVALID_ARG;
  if (a->n_rows == 0 || a->num_req == 0) return CSA_OK;
  const csa_status st = check_cache(a->cache);
  if (st != CSA_OK) return st;
  if (!a->page_table || !a->kv_start || !a->out || a->pt_stride < 1 ||
      static_cast<int64_t>(kPageRecs) * a->pt_stride > INT32_MAX)
    return CSA_ERR_INVALID_ARG;
  if (!aligned(a->page_table, 4) || !aligned(a->kv_start, 4) || !aligned(a->out, 16) || !aligned(a->dev_status, 4))
    return CSA_ERR_ALIGNMENT;
  const auto s = static_cast<cudaStream_t>(stream);
  if (a->cache.record_format == CSA_LATENT_MXFP4)
    return a->cache.rope_dim ? launch_read<true, 64>(*a, s) : launch_read<true, 0>(*a, s);
  return a->cache.rope_dim ? launch_read<false, 64>(*a, s) : launch_read<false, 0>(*a, s);
}
