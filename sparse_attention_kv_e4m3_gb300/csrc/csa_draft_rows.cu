// csa_draft_rows.cu — norms and rotation of queries and keys, the writer that norms and rotates on the way,
// and the move of accepted drafts' records (include/csa_draft.h). All three are one pass over their data.
#include "csa_latent_rows.cuh"
#include "csa_rotation.cuh"

namespace csa_latent {
namespace {

// ------------------------------------------------------------- norm and rotation of heads
//
// A group of 8, 16 or 32 lanes takes a head, a lane up to 4 pieces of 8 values of it (16 or 32 bytes a load): the fewest lanes with which
// most of them have work. A head's values stay in registers between the sum of squares and the store, so every value is
// read and written once; a rotated pair of halves comes from another lane's values, which are loaded again (from L1)
// rather than exchanged, because where the rotated part begins is free. A block takes up to 32 rows at a time, whose cosines and
// sines are made once, in shared memory, for all heads, as are the weights. 16384 rows of 17 heads of 192 (214 MB): 44 us, 4.9 TB/s; what
// it takes beyond the bytes are instructions (72% of the issue slots when it took 49 us).

constexpr int kRotThreads = 256;

template <bool kF32>
struct Eight {  // eight values as they lie in memory
  uint4 w[kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p) {
#pragma unroll
    for (int k = 0; k < (kF32 ? 2 : 1); ++k) w[k] = reinterpret_cast<const uint4*>(p)[k];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (kF32) {
      const uint32_t x[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(x[k]);
    } else {
      const uint32_t x[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = bf16_lo(x[k]);
        v[2 * k + 1] = bf16_hi(x[k]);
      }
    }
  }
  __device__ __forceinline__ void put(const float (&v)[8]) {
    if constexpr (kF32) {
      w[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      w[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    } else {
      w[0] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    }
  }
  __device__ __forceinline__ void times(float f) {
    float v[8];
    get(v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= f;
    put(v);
  }
  __device__ __forceinline__ void store(void* p) const {
#pragma unroll
    for (int k = 0; k < (kF32 ? 2 : 1); ++k) reinterpret_cast<uint4*>(p)[k] = w[k];
  }
};

struct RotateKernel {
  csa_rotate_args A;
  int32_t rows;              // a block's at a time
  int32_t q_lanes, k_lanes;  // of a head
};

constexpr int kMostRows = 32;

// Pieces of 8 values that a lane has of a head whose `lanes` share it.
__host__ __device__ constexpr int pieces_of(int dim, int lanes) { return (dim / 8 + lanes - 1) / lanes; }

// y r w of eight values; the weights lie as the first and the last four of each chunk of eight, apart.
__device__ __forceinline__ void weighted(float (&y)[8], float r, const float4* w, int chunk, int chunks) {
  const float4 a = w[chunk], b = w[chunks + chunk];
  y[0] = y[0] * r * a.x, y[1] = y[1] * r * a.y, y[2] = y[2] * r * a.z, y[3] = y[3] * r * a.w;
  y[4] = y[4] * r * b.x, y[5] = y[5] * r * b.y, y[6] = y[6] * r * b.z, y[7] = y[7] * r * b.w;
}

// Heads head0 .. head0 + heads of one tensor, of rows row0 .. row0 + rows. `weights` are the tensor's, in shared memory. Lanes
// past a head's end, and groups past the last head, load what others load, and neither add nor store it.
template <bool kF32In, int kPieces, bool kHalves>
__device__ __forceinline__ void rotate_heads(const csa_rotate_args& A, const csa_heads& T, int G, int64_t row0, int rows, int head0, int heads,
                                             const float4* turns, const int32_t* pos, const float4* weights) {
  constexpr int kIn = kF32In ? 4 : 2;
  const int lane = threadIdx.x & (G - 1), chunks = T.dim / 8, half = A.rotation.rope_dim / 2, groups = kRotThreads / G;
  const float per_value = 1.f / static_cast<float>(T.dim);
  // of the head's chunks of 8 values, those that rotate, and how far apart halves lie
  const int turn0 = A.rope_first ? 0 : chunks - half / 4, turn1 = turn0 + half / 4, apart = half / 8;
  // heads g, g + groups, ... of the rows' heads, row by row
  const int step_rows = groups / heads, step_heads = groups - step_rows * heads;
  int row = static_cast<int>(threadIdx.x) / G / heads, head = static_cast<int>(threadIdx.x) / G - row * heads;
  const int most = (rows * heads + groups - 1) / groups;  // the same for all groups, whose lanes share warps
  for (int i = 0; i < most; ++i) {
    const int at_row = min(row, rows - 1), at_head = head0 + head;
    const bool live = row < rows && pos[at_row] >= 0;
    const uint8_t* src = static_cast<const uint8_t*>(T.x) + kIn * ((row0 + at_row) * T.x_row_stride + at_head * T.x_head_stride);
    Eight<kF32In> x[kPieces], other[kHalves ? kPieces : 1];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int c = min(lane + G * k, chunks - 1);
      x[k].load(src + 8 * kIn * c);
      if (kHalves) other[k].load(src + 8 * kIn * (c >= turn0 && c < turn1 ? (c < turn0 + apart ? c + apart : c - apart) : c));
    }
    float r = 1.f;
    if (T.norm) {
      float part[2] = {0.f, 0.f};
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        float v[8];
        x[k].get(v);
        if (lane + G * k < chunks)
#pragma unroll
          for (int j = 0; j < 8; ++j) part[j & 1] = fmaf(v[j], v[j], part[j & 1]);
      }
      float sum = part[0] + part[1];
      for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      const float mean = fmaf(sum, per_value, A.eps);
      r = rsqrtf(mean);
      if (__any_sync(0xFFFFFFFFu, !plain_mean(mean))) {
        double wide = 0.0;
#pragma unroll 1
        for (int c = lane; c < chunks; c += G) {
          Eight<kF32In> again;
          again.load(src + 8 * kIn * c);
          float v[8];
          again.get(v);
#pragma unroll
          for (int j = 0; j < 8; ++j) wide += static_cast<double>(v[j]) * v[j];
        }
        for (int o = G / 2; o > 0; o >>= 1) wide += __shfl_xor_sync(0xFFFFFFFFu, wide, o);
        if (!plain_mean(mean)) {
          const Factor f = factor_of(1.0 / sqrt(wide / T.dim + A.eps));
          r = f.rest;
#pragma unroll
          for (int k = 0; k < kPieces; ++k) {
            x[k].times(f.first);
            if (kHalves) other[k].times(f.first);
          }
        }
      }
    }
    __syncwarp();  // in place: all of a head is read before any of it is written
    if (live) {
      const int64_t to = (row0 + at_row) * T.out_row_stride + at_head * T.out_head_stride;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int c = lane + G * k;
        if (c >= chunks) break;
        float v[8];
        x[k].get(v);
        if (T.norm) weighted(v, r, weights, c, chunks);
        if (c >= turn0 && c < turn1) {
          const float4* t = turns + at_row * (half / 2);
          if constexpr (kHalves) {
            const bool low = c < turn0 + apart;
            float u[8];
            other[k].get(u);
            if (T.norm) weighted(u, r, weights, low ? c + apart : c - apart, chunks);
            t += 4 * (low ? c - turn0 : c - turn0 - apart);
            const float sign = low ? -1.f : 1.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4 w = t[j];
              v[2 * j] = v[2 * j] * w.x + sign * u[2 * j] * w.y;
              v[2 * j + 1] = v[2 * j + 1] * w.z + sign * u[2 * j + 1] * w.w;
            }
          } else {
            t += 2 * (c - turn0);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float4 w = t[j];
              float* y = v + 4 * j;
              const float a0 = y[0], b0 = y[1], a1 = y[2], b1 = y[3];
              y[0] = a0 * w.x - b0 * w.y, y[1] = b0 * w.x + a0 * w.y;
              y[2] = a1 * w.z - b1 * w.w, y[3] = b1 * w.z + a1 * w.w;
            }
          }
        }
        if (A.out_dtype == CSA_KEYS_F32) {
          Eight<true> y;
          y.put(v);
          y.store(static_cast<float*>(T.out) + to + 8 * c);
        } else {
          Eight<false> y;
          y.put(v);
          y.store(static_cast<__nv_bfloat16*>(T.out) + to + 8 * c);
        }
      }
    }
    row += step_rows;
    head += step_heads;
    if (head >= heads) {
      head -= heads;
      ++row;
    }
  }
}

template <bool kF32In, int kPieces, bool kHalves>
__global__ void __launch_bounds__(kRotThreads, kF32In || kPieces > 3 ? 3 : 4) rotate_kernel(const RotateKernel K) {
  extern __shared__ float4 rotate_smem[];  // the weights of q and of k, then [rows of the block][rope_dim / 2] cos, sin
  __shared__ uint64_t per_token[CSA_ROTATE_MAX_ROPE / 2];
  __shared__ int32_t pos[kMostRows];
  const csa_rotate_args& A = K.A;
  const int half = A.rotation.rope_dim / 2, tid = threadIdx.x;
  const int q_dim = A.q.heads > 0 ? A.q.dim : 0, k_dim = A.k.heads > 0 ? A.k.dim : 0;
  float* weights = reinterpret_cast<float*>(rotate_smem);
  float2* turns = reinterpret_cast<float2*>(weights + q_dim + k_dim);
  const float4 *q_weights = rotate_smem, *k_weights = rotate_smem + q_dim / 4, *row_turns = reinterpret_cast<const float4*>(turns);
  int32_t flags = 0;
  // this block's heads of each tensor: all of them, unless there are few rows
  const int y = blockIdx.y, ys = gridDim.y;
  const int q0 = A.q.heads * y / ys, q1 = A.q.heads * (y + 1) / ys, k0 = A.k.heads * y / ys, k1 = A.k.heads * (y + 1) / ys;
  auto rows_at = [&](int64_t row0) { return static_cast<int>(min(static_cast<int64_t>(K.rows), A.n - row0)); };
  const int64_t step = static_cast<int64_t>(gridDim.x) * K.rows;
  for (int j = tid; j < half; j += kRotThreads) per_token[j] = turns_per_token(A.rotation.freq[j]);
  for (int i = tid; i < q_dim + k_dim; i += kRotThreads) {
    const float* w = i < q_dim ? A.q.weight : A.k.weight;
    const int first = i < q_dim ? 0 : q_dim, n = i - first, dim = i < q_dim ? q_dim : k_dim;
    weights[first + (n & 4) / 4 * (dim / 2) + n / 8 * 4 + (n & 3)] = w ? w[n] : 1.f;
  }
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * K.rows; row0 < A.n; row0 += step) {
    const int rows = rows_at(row0);
    if (tid < rows) {  // every thread has taken what it needs of the last rows' positions: it has read their turns
      const int32_t p = A.pos ? A.pos[row0 + tid] : 0;
      if (p < -1) flags |= CSA_DEV_LEN_OOB;
      pos[tid] = p;
    }
    __syncthreads();
    for (int i = tid; i < rows * half; i += kRotThreads) turns[i] = cos_sin(per_token[i % half], pos[i / half], A.rotation.scale);
    __syncthreads();
    if (q1 > q0) rotate_heads<kF32In, kPieces, kHalves>(A, A.q, K.q_lanes, row0, rows, q0, q1 - q0, row_turns, pos, q_weights);
    if (k1 > k0) rotate_heads<kF32In, kPieces, kHalves>(A, A.k, K.k_lanes, row0, rows, k0, k1 - k0, row_turns, pos, k_weights);
    if (row0 + step < A.n) __syncthreads();
  }
  flags = static_cast<int32_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(flags)));
  if (flags && A.dev_status && (tid & 31) == 0) atomicOr(A.dev_status, flags);
}

template <bool kF32In, int kPieces, bool kHalves>
csa_status launch_rotate(RotateKernel& K, int sms, int dev, cudaStream_t stream) {
  const csa_rotate_args& a = K.A;
  auto smem = [&](int rows) {
    return sizeof(float) * ((a.q.heads > 0 ? a.q.dim : 0) + (a.k.heads > 0 ? a.k.dim : 0)) + sizeof(float2) * rows * (a.rotation.rope_dim / 2);
  };
  static Kept kept;  // resident blocks an SM, with the most shared memory
  int per_sm = kept.get(dev);
  if (per_sm == 0) {
    constexpr size_t most = sizeof(float) * 2 * CSA_ROTATE_MAX_DIM + sizeof(float2) * kMostRows * (CSA_ROTATE_MAX_ROPE / 2);
    static_assert(most <= 40 * 1024, "shared memory of a block");
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, rotate_kernel<kF32In, kPieces, kHalves>, kRotThreads, most) != cudaSuccess || per_sm < 1)
      return CSA_ERR_CUDA;
    kept.set(dev, per_sm);
  }
  // At most one wave; fewer rows a block where there are few, so that all SMs have some, and where there are fewer rows than SMs
  // several blocks a row (64 rows of 65 heads: 8.6 us, with a block a row 10.5).
  const int64_t cap = static_cast<int64_t>(sms) * per_sm, rounds = (a.n + cap * kMostRows - 1) / (cap * kMostRows);
  K.rows = static_cast<int32_t>((a.n + cap * rounds - 1) / (cap * rounds));
  const int64_t blocks = (a.n + K.rows - 1) / K.rows, heads = a.q.heads > a.k.heads ? a.q.heads : a.k.heads, share = 2 * sms / blocks;
  const dim3 grid(static_cast<unsigned>(blocks < cap ? blocks : cap), static_cast<unsigned>(share < 1 ? 1 : (share < heads ? share : heads) < 16 ? (share < heads ? share : heads) : 16));
  rotate_kernel<kF32In, kPieces, kHalves><<<grid, kRotThreads, smem(K.rows), stream>>>(K);
  return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

template <bool kF32In, bool kHalves>
csa_status launch_rotate_dim(RotateKernel& K, cudaStream_t stream) {
  int sms = 0, dev = 0;
  if (sm_count(&sms, &dev) != CSA_OK) return CSA_ERR_CUDA;
  // lanes of a head: 8, 16 or 32, with the fewest idle, the fewest lanes first, and at most 3 pieces a lane where 32 are enough for that
  auto lanes = [](const csa_heads& t) {
    int best = 32;
    for (int g = 16; g >= 8; g /= 2)
      if (pieces_of(t.dim, g) <= 3 && g * pieces_of(t.dim, g) <= best * pieces_of(t.dim, best)) best = g;
    return best;
  };
  int pieces = 1;
  K.q_lanes = K.k_lanes = 32;
  if (K.A.q.heads > 0) pieces = pieces_of(K.A.q.dim, K.q_lanes = lanes(K.A.q));
  if (K.A.k.heads > 0) {
    K.k_lanes = lanes(K.A.k);
    const int k = pieces_of(K.A.k.dim, K.k_lanes);
    pieces = k > pieces ? k : pieces;
  }
  if (pieces == 1) return launch_rotate<kF32In, 1, kHalves>(K, sms, dev, stream);
  if (pieces == 2) return launch_rotate<kF32In, 2, kHalves>(K, sms, dev, stream);
  if (pieces == 3) return launch_rotate<kF32In, 3, kHalves>(K, sms, dev, stream);
  return launch_rotate<kF32In, 4, kHalves>(K, sms, dev, stream);
}

csa_status check_heads(const csa_heads& t, int64_t n, int rope, bool f32_in, bool f32_out) {
  if (t.heads < 0) return CSA_ERR_INVALID_ARG;
  if (t.heads == 0) return CSA_OK;
  if (t.reserved0 != 0 || (t.norm != 0 && t.norm != 1)) return CSA_ERR_INVALID_ARG;
  if (t.dim < 8 || t.dim > CSA_ROTATE_MAX_DIM || t.dim % 8 != 0 || t.heads > CSA_ROTATE_MAX_HEADS) return CSA_ERR_UNSUPPORTED;
  if (rope > t.dim || !t.x || !t.out) return CSA_ERR_INVALID_ARG;
  if ((t.heads > 1 && (t.x_head_stride < t.dim || t.out_head_stride < t.dim)) || (n > 1 && (t.x_row_stride < t.dim || t.out_row_stride < t.dim)))
    return CSA_ERR_INVALID_ARG;
  const int in = f32_in ? 4 : 8, out = f32_out ? 4 : 8;
  if (!aligned(t.x, 16) || !aligned(t.out, 16) || !aligned(t.weight, 16) || t.x_row_stride % in != 0 || t.x_head_stride % in != 0 ||
      t.out_row_stride % out != 0 || t.out_head_stride % out != 0)
    return CSA_ERR_ALIGNMENT;
  if (t.x == t.out && (f32_in != f32_out || (n > 1 && t.x_row_stride != t.out_row_stride) || (t.heads > 1 && t.x_head_stride != t.out_head_stride)))
    return CSA_ERR_INVALID_ARG;
  return CSA_OK;
}

// ------------------------------------------------------------- norm, rotation and store of latents
//
// The cache's writer (a warp a row, its loads ahead of it) with the norm and the rotation between load and store. The codes of
// a 4-bit record depend on which side of a border a value lies, so the fast result, whose error is known, is encoded
// twice, a little larger and a little smaller; where the two differ (a value or two of one row in 100) the row's factor
// and those values are computed again in fp64. (All of the row in fp64 cost 65537 rows 5 us of 82.) 65537 fp32 rows to 4 bits: 50 us where the
// bytes are 26, 380 instructions a row and 61% of the issue slots: with 16 warps an SM neither is full; 16381 bf16 rows: 13.6 us, of which the bytes
// are 5.6, 44% of the issue slots.

// The relative error of x r w in fp32: the sum of 16 squares a lane and 5 steps over the lanes, (16 + 5) 2^-24, the mean and eps
// 2 x 2^-24, halved by the root; rsqrtf (two units in the last place) 4 x 2^-24 and two products 2 x 2^-24 more: 18 x 2^-24.
// 2^-19 is nearly twice that. Where x r is subnormal it is off by 2^-150 instead: with weights up to 2^24 that is 2^-126 of a value, in a
// block whose smallest border is 2^-104 or more (its largest value is above 2^-100), 2^-22 of it and still within 2^-19. Rows with
// larger weights are computed in fp64 whole.
constexpr float kNear = 0x1p-19f, kMostWeight = 0x1p24f;

// The norm's factor in fp64. Rows are read again where they are wanted exactly, so that their values need not have an
// address where they are not.
template <bool kBf16In>
__device__ __noinline__ double exact_factor(const void* row, float eps) {
  RowIn<kBf16In> x;
  x.load(row, threadIdx.x & 31, 0);
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < 16; ++k) sum += static_cast<double>(x.v[k]) * x.v[k];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  return 1.0 / sqrt(sum / kDim + eps);
}

// Value k of the lane's, normed by the factor r.
template <bool kBf16In>
__device__ __forceinline__ double exact_value(const void* row, const float* weight, double r, int k) {
  const int at = 16 * (threadIdx.x & 31) + k;
  const float x = kBf16In ? __bfloat162float(static_cast<const __nv_bfloat16*>(row)[at]) : static_cast<const float*>(row)[at];
  return x * r * (weight ? __ldg(weight + at) : 1.f);
}

// The e2m1 code of y 2^-e: nearest, ties to the even code, saturating at 6.
__device__ __forceinline__ uint32_t exact_code(double y, int e) {
  const double t = fabs(y) * __hiloint2double((1023 - e) << 20, 0);
  const uint32_t m = (t > 0.25) + (t >= 0.75) + (t > 1.25) + (t >= 1.75) + (t > 2.5) + (t >= 3.5) + (t > 5.0);
  return m | (signbit(y) ? 8u : 0u);
}

// Codes and exponent of a lane's values, all of them in fp64.
template <bool kBf16In>
__device__ __noinline__ Coded<true> encode_exact(const void* row, const float* weight, float eps) {
  const double r = exact_factor<kBf16In>(row, eps);
  Coded<true> c;
  double amax = 0.0;
  c.bad = false;
#pragma unroll 1
  for (int k = 0; k < 16; ++k) {
    const double y = fabs(exact_value<kBf16In>(row, weight, r, k));
    c.bad |= !(y < 0x1.ffffffp127);  // what rounds to a finite fp32, and no NaN
    amax = fmax(amax, y);
  }
  amax = fmax(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  // floor(log2 amax) - 2, held at -127 (a double that is subnormal lies far below)
  c.e = max(static_cast<int>(__double2hiint(amax) >> 20) - 1023 - 2, -127);
  c.w[0] = c.w[1] = 0;
#pragma unroll 1
  for (int k = 0; k < 16; ++k) {
    const uint32_t code = exact_code(exact_value<kBf16In>(row, weight, r, k), c.e) << (4 * (k & 7));
    if (k < 8) c.w[0] |= code;
    else c.w[1] |= code;
  }
  return c;
}

template <bool kBf16In, bool kFp4>
__device__ __forceinline__ int32_t append_row(const csa_append_args& A, const RowIn<kBf16In>& x, const void* row, const float (&w)[16],
                                              bool large, const uint64_t (&per_token)[2], int64_t slot, int32_t pos, int lane) {
  if (slot == -1) return 0;
  if (slot < 0 || slot >= A.cache.num_pages * kPageRecs) return CSA_DEV_PAGE_OOB;
  const bool rope = A.cache.rope_dim != 0;
  uint32_t rope_word = 0;
  if (rope) {
    if (pos < 0) return CSA_DEV_LEN_OOB;
    const float2 t = cos_sin(per_token[0], pos, A.rotation.scale);
    const float a = x.r[0], b = x.r[1];
    if (A.rotation.pairing == CSA_PAIRS_ADJACENT) {
      rope_word = pack_bf16(a * t.x - b * t.y, b * t.x + a * t.y);
    } else {  // values 2 l, 2 l + 1 of one half, the same of the other one 16 lanes away
      const float2 t1 = cos_sin(per_token[1], pos, A.rotation.scale);
      const float c = __shfl_xor_sync(0xFFFFFFFFu, a, 16), d = __shfl_xor_sync(0xFFFFFFFFu, b, 16), sign = lane < 16 ? -1.f : 1.f;
      rope_word = pack_bf16(a * t.x + sign * c * t.y, b * t1.x + sign * d * t1.y);
    }
  }
  Coded<kFp4> c;
  if (!A.norm) {
    c = encode<kFp4>(x.v);
  } else {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) sum = fmaf(x.v[k], x.v[k], sum);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    const float mean = sum * (1.f / kDim) + A.eps;
    float r = rsqrtf(mean);
    const bool plain = plain_mean(mean);
    float y[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) y[k] = x.v[k];
    if (!kFp4 && !plain) {
      double wide = 0.0;
#pragma unroll
      for (int k = 0; k < 16; ++k) wide += static_cast<double>(x.v[k]) * x.v[k];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) wide += __shfl_xor_sync(0xFFFFFFFFu, wide, o);
      const Factor f = factor_of(1.0 / sqrt(wide / kDim + A.eps));
      r = f.rest;
#pragma unroll
      for (int k = 0; k < 16; ++k) y[k] *= f.first;
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) y[k] = y[k] * r * w[k];
    if constexpr (!kFp4) {
      c = encode<false>(y);
    } else {  // the codes and the exponent a little further out, and a little further in
      uint32_t amax = 0;
#pragma unroll
      for (int k = 0; k < 16; ++k) amax = max(amax, __float_as_uint(y[k]) & 0x7FFFFFFFu);
      amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      const float top = __uint_as_float(amax), far = 1.f + kNear, close = 1.f - kNear;
      c.e = block_exponent(__float_as_uint(top * far));
      c.bad = false;  // what is not finite is not plain, or near
      const float up = block_up(c.e), up_far = up * far, up_close = up * close;
      uint32_t differ[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t b = 0;
        c.w[h] = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          c.w[h] |= e2m1_pair(y[8 * h + 2 * k] * up_far, y[8 * h + 2 * k + 1] * up_far) << (8 * k);
          b |= e2m1_pair(y[8 * h + 2 * k] * up_close, y[8 * h + 2 * k + 1] * up_close) << (8 * k);
        }
        differ[h] = c.w[h] ^ b;
      }
      // outside of 2^-100 .. 2^100 products and borders may leave fp32's normal range; next to a power of two the exponent is open
      if (__any_sync(0xFFFFFFFFu, large || !plain || !(top > 0x1p-100f && top < 0x1p100f) || block_exponent(__float_as_uint(top * close)) != c.e)) {
        c = encode_exact<kBf16In>(row, A.weight, A.eps);
      } else if (__any_sync(0xFFFFFFFFu, differ[0] | differ[1])) {
        const double exact_r = exact_factor<kBf16In>(row, A.eps);
        while (differ[0] | differ[1]) {  // the values whose code is open
          const bool second = differ[0] == 0;
          const int n = (__ffs(second ? differ[1] : differ[0]) - 1) / 4;
          const uint32_t clear = ~(15u << (4 * n)), code = exact_code(exact_value<kBf16In>(row, A.weight, exact_r, 8 * second + n), c.e) << (4 * n);
          if (second) c.w[1] = (c.w[1] & clear) | code, differ[1] &= clear;
          else c.w[0] = (c.w[0] & clear) | code, differ[0] &= clear;
        }
        __syncwarp();
      }
    }
  }
  if (__any_sync(0xFFFFFFFFu, c.bad || nonfinite_bf16x2(rope_word))) return CSA_DEV_RANGE;
  put_record<kFp4>(A.cache, slot, c, rope_word, lane);
  return 0;
}

template <bool kBf16In, bool kFp4>
__global__ void __launch_bounds__(kCopyThreads, 2) append_kernel(const csa_append_args A) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kCopyThreads / 32);
  int32_t flags = 0;
  float w[16];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 v = A.norm && A.weight ? __ldg(reinterpret_cast<const float4*>(A.weight) + 4 * lane + k) : make_float4(1.f, 1.f, 1.f, 1.f);
    w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
  }
  bool large = false;  // a weight of the lane's, or NaN
  if (kFp4)
#pragma unroll
    for (int k = 0; k < 16; ++k) large |= !(fabsf(w[k]) <= kMostWeight);
  uint64_t per_token[2] = {0, 0};
  if (A.cache.rope_dim != 0) {
    const bool adjacent = A.rotation.pairing == CSA_PAIRS_ADJACENT;
    per_token[0] = turns_per_token(A.rotation.freq[adjacent ? lane : 2 * lane & 31]);
    if (!adjacent) per_token[1] = turns_per_token(A.rotation.freq[(2 * lane & 31) + 1]);
  }
  auto row_of = [&](int64_t i) { return static_cast<const uint8_t*>(A.x) + i * A.x_stride * (kBf16In ? 2 : 4); };
  struct Row {
    RowIn<kBf16In> x;
    int64_t slot;
    int32_t pos;
  };
  auto fetch = [&](Row& r, int64_t i) {
    r.slot = i < A.n ? A.slots[i] : -1;
    const int64_t at = i < A.n ? i : 0;
    r.pos = A.cache.rope_dim != 0 ? A.pos[at] : 0;
    r.x.load(row_of(at), lane, A.cache.rope_dim);
  };
  Row now, next;
  int64_t i = (static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x) >> 5;
  if (i < A.n) fetch(now, i);
  for (; i < A.n; i += warps, now = next) {
    fetch(next, i + warps);  // on its way while this one is normed and stored
    flags |= append_row<kBf16In, kFp4>(A, now.x, row_of(i), w, large, per_token, now.slot, now.pos, lane);
  }
  if (flags && A.dev_status && lane == 0) atomicOr(A.dev_status, flags);
}

template <bool kBf16In, bool kFp4>
csa_status launch_append(const csa_append_args& a, cudaStream_t stream) {
  static Kept kept;
  unsigned grid = 1;
  const csa_status st = wave_grid(append_kernel<kBf16In, kFp4>, kCopyThreads, 0, &kept, a.n, kCopyThreads / 32, &grid);
  if (st != CSA_OK) return st;
  append_kernel<kBf16In, kFp4><<<grid, kCopyThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

// ------------------------------------------------------------- accepted drafts
//
// One launch. Block 0 makes the lengths and the list of pages; each of the others moves a request's records in as many
// layers as it has teams of threads, one a 16-byte column of a record. A column belongs to one thread, which takes the path
// in order, kMoves loads and then their stores: as path[k] >= k and both ascend, no store falls on a record that a later load
// wants, and none of the batch's loads is behind its stores. Every block checks the whole path of its request before it
// moves anything. 48 requests, 24 layers (7 MB): 8.7 us, four loads each waiting on the one before.

constexpr int kCommitThreads = 288, kMoves = 8;  // 4 layers of 72 columns, 11 of 25, 16 of 17
constexpr int kPathBatch = 128;

struct Commit {
  int32_t base, drafts, n;  // n: accepted
};

__device__ __forceinline__ int64_t slot_at(const csa_commit_args& A, const int32_t* table, int32_t pos) {  // -1: the page is out of range
  const int32_t page = __ldg(table + pos / kPageRecs);
  return page < 0 || page >= A.cache.num_pages ? -1 : static_cast<int64_t>(page) * kPageRecs + pos % kPageRecs;
}

// Request r's numbers; whether they are in range.
__device__ __forceinline__ bool commit_of(const csa_commit_args& A, int r, Commit* C) {
  const int64_t cap = static_cast<int64_t>(kPageRecs) * A.pt_stride, base = A.base_len[r], drafts = A.draft_len[r], n = A.path_len[r];
  *C = {static_cast<int32_t>(base), static_cast<int32_t>(drafts), static_cast<int32_t>(n)};
  return base >= 0 && drafts >= 0 && base + drafts <= cap && n >= 0 && n <= drafts && n <= A.path_stride;
}

// What is wrong with entries first, first + step, ... of request r's path and of the pages that it gives back.
__device__ __forceinline__ int32_t path_faults(const csa_commit_args& A, int r, const Commit& C, int first, int step) {
  const int32_t* path = A.path + static_cast<int64_t>(r) * A.path_stride;
  const int32_t* table = A.page_table + static_cast<int64_t>(r) * A.pt_stride;
  int32_t bad = 0;
  for (int k = first; k < C.n; k += step) {
    const int32_t d = path[k];
    if (d < k || d >= C.drafts || (k > 0 && path[k - 1] >= d)) bad |= CSA_DEV_LEN_OOB;
    else if (d != k && (slot_at(A, table, C.base + d) < 0 || slot_at(A, table, C.base + k) < 0)) bad |= CSA_DEV_PAGE_OOB;
  }
  const int64_t end = (static_cast<int64_t>(C.base) + C.drafts + kPageRecs - 1) / kPageRecs;
  for (int64_t p = (static_cast<int64_t>(C.base) + C.n + kPageRecs - 1) / kPageRecs + first; p < end; p += step)
    if (table[p] < 0 || table[p] >= A.cache.num_pages) bad |= CSA_DEV_PAGE_OOB;
  return bad;
}

__device__ void move_records(const csa_commit_args& A, int r, int layer0, int columns, int64_t* from, int64_t* to) {
  Commit C;
  if (!commit_of(A, r, &C) || C.n == 0) return;
  const int32_t* path = A.path + static_cast<int64_t>(r) * A.path_stride;
  const int32_t* table = A.page_table + static_cast<int64_t>(r) * A.pt_stride;
  const int tid = threadIdx.x;
  if (__syncthreads_or(path_faults(A, r, C, tid, kCommitThreads))) return;
  auto byte_of = [&](int32_t pos) {
    const int64_t slot = slot_at(A, table, pos);
    return slot / kPageRecs * A.cache.page_stride_bytes + slot % kPageRecs * (16 * columns);
  };
  const int layer = layer0 + tid / columns;
  const bool mover = tid / columns < kCommitThreads / columns && layer < A.num_layers;
  uint8_t* column = A.cache.pages + layer * A.layer_stride_bytes + 16 * (tid % columns);
  for (int k0 = 0; k0 < C.n; k0 += kPathBatch) {
    const int n = min(kPathBatch, C.n - k0);
    __syncthreads();
    if (tid < n) {
      const int k = k0 + tid, d = path[k];
      from[tid] = d == k ? -1 : byte_of(C.base + d);
      to[tid] = d == k ? -1 : byte_of(C.base + k);
    }
    __syncthreads();
    for (int k = 0; mover && k < n; k += kMoves) {
      uint4 v[kMoves];
#pragma unroll
      for (int i = 0; i < kMoves; ++i)
        if (k + i < n && from[k + i] >= 0) v[i] = *reinterpret_cast<const uint4*>(column + from[k + i]);
#pragma unroll
      for (int i = 0; i < kMoves; ++i)
        if (k + i < n && from[k + i] >= 0) *reinterpret_cast<uint4*>(column + to[k + i]) = v[i];
    }
  }
}

// Lengths after the step, and the pages given back: a warp checks a request, a block's threads of requests at a time, then a
// thread lists a request's pages behind those of the requests before.
__device__ void list_pages(const csa_commit_args& A, int32_t* count, int32_t* sums, int32_t* flags) {
  constexpr int batch = kCommitThreads, warps = kCommitThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t before = 0;
  for (int r0 = 0; r0 < A.num_req; r0 += batch) {
    for (int i = warp; i < batch && r0 + i < A.num_req; i += warps) {
      const int r = r0 + i;
      Commit C;
      const bool ok = commit_of(A, r, &C);
      const int32_t bad = ok ? static_cast<int32_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(path_faults(A, r, C, lane, 32)))) : CSA_DEV_LEN_OOB;
      *flags |= bad;
      if (lane == 0) {
        A.new_len[r] = bad ? C.base : C.base + C.n;
        count[i] = bad ? 0 : (C.base + C.drafts + kPageRecs - 1) / kPageRecs - (C.base + C.n + kPageRecs - 1) / kPageRecs;
      }
    }
    __syncthreads();
    const int mine = r0 + tid < A.num_req ? count[tid] : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int64_t at = before + incl - mine;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) at += sums[w];
      before += sums[w];
    }
    if (mine > 0) {
      const int r = r0 + tid;
      const int32_t* pages = A.page_table + static_cast<int64_t>(r) * A.pt_stride + (A.new_len[r] + kPageRecs - 1) / kPageRecs;
      for (int p = 0; p < mine && at + p < A.room; ++p) A.freed[at + p] = pages[p];
    }
    __syncthreads();
  }
  for (int64_t i = before + tid; i < A.room; i += kCommitThreads) A.freed[i] = -1;
  if (before > A.room) *flags |= CSA_DEV_ROWS;
  if (tid == 0) A.n_freed[0] = static_cast<int32_t>(min(before, static_cast<int64_t>(INT32_MAX)));
}

__global__ void __launch_bounds__(kCommitThreads) commit_kernel(const csa_commit_args A, int columns) {
  __shared__ int64_t from[kPathBatch], to[kPathBatch];
  __shared__ int32_t count[kCommitThreads], sums[kCommitThreads / 32];
  int32_t flags = 0;
  const int at = static_cast<int>(blockIdx.x) - 1;
  if (at < 0) list_pages(A, count, sums, &flags);
  else move_records(A, at % A.num_req, at / A.num_req * (kCommitThreads / columns), columns, from, to);
  flags = static_cast<int32_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(flags)));
  if (flags && A.dev_status && (threadIdx.x & 31) == 0) atomicOr(A.dev_status, flags);
}

}  // namespace
}  // namespace csa_latent

using namespace csa_latent;

extern "C" int32_t csa_draft_abi_version(void) { return CSA_DRAFT_ABI_VERSION; }

extern "C" csa_status csa_head_norm_rotate(const csa_rotate_args* a, void* stream) {
  if (!a || a->n < 0 || (a->dtype != CSA_KEYS_F32 && a->dtype != CSA_KEYS_BF16) || (a->out_dtype != CSA_KEYS_F32 && a->out_dtype != CSA_KEYS_BF16) ||
      (a->rope_first != 0 && a->rope_first != 1) || !good_eps(a->eps))
    return CSA_ERR_INVALID_ARG;
  csa_status st = check_rotation(a->rotation);
  if (st != CSA_OK) return st;
  const int rope = a->rotation.rope_dim;
  if (rope > CSA_ROTATE_MAX_ROPE || rope % 16 != 0) return CSA_ERR_UNSUPPORTED;
  if (a->q.heads < 0 || a->k.heads < 0) return CSA_ERR_INVALID_ARG;
  if (a->n == 0 || (a->q.heads == 0 && a->k.heads == 0)) return CSA_OK;
  if (rope > 0 && !a->pos) return CSA_ERR_INVALID_ARG;
  if (a->n > INT64_C(1) << 40) return CSA_ERR_INVALID_ARG;
  const bool f32_in = a->dtype == CSA_KEYS_F32, f32_out = a->out_dtype == CSA_KEYS_F32;
  for (const csa_heads* t : {&a->q, &a->k})
    if ((st = check_heads(*t, a->n, rope, f32_in, f32_out)) != CSA_OK) return st;
  if (!aligned(a->pos, 4) || !aligned(a->dev_status, 4)) return CSA_ERR_ALIGNMENT;
  RotateKernel K = {*a, 1, 32, 32};
  const auto s = static_cast<cudaStream_t>(stream);
  const bool halves = rope > 0 && a->rotation.pairing == CSA_PAIRS_HALVES;
  if (f32_in) return halves ? launch_rotate_dim<true, true>(K, s) : launch_rotate_dim<true, false>(K, s);
  return halves ? launch_rotate_dim<false, true>(K, s) : launch_rotate_dim<false, false>(K, s);
}

extern "C" csa_status csa_latent_append(const csa_append_args* a, void* stream) {
  if (!a || a->n < 0 || a->reserved0 != 0 || (a->dtype != CSA_KEYS_F32 && a->dtype != CSA_KEYS_BF16) || (a->norm != 0 && a->norm != 1) || !good_eps(a->eps))
    return CSA_ERR_INVALID_ARG;
  csa_status st = check_rotation(a->rotation);
  if (st != CSA_OK || a->n == 0) return st;
  if ((st = check_cache(a->cache)) != CSA_OK) return st;
  const int rope = a->cache.rope_dim;
  const bool bf16 = a->dtype == CSA_KEYS_BF16;
  if (a->rotation.rope_dim != rope || (rope > 0 && !a->pos)) return CSA_ERR_INVALID_ARG;
  if (!a->x || !a->slots || a->x_stride < kDim + rope) return CSA_ERR_INVALID_ARG;
  if (!aligned(a->x, 16) || a->x_stride % (bf16 ? 8 : 4) != 0 || !aligned(a->slots, 8) || !aligned(a->pos, 4) || !aligned(a->weight, 16) ||
      !aligned(a->dev_status, 4))
    return CSA_ERR_ALIGNMENT;
  const bool fp4 = a->cache.record_format == CSA_LATENT_MXFP4;
  const auto s = static_cast<cudaStream_t>(stream);
  if (bf16) return fp4 ? launch_append<true, true>(*a, s) : launch_append<true, false>(*a, s);
  return fp4 ? launch_append<false, true>(*a, s) : launch_append<false, false>(*a, s);
}

extern "C" csa_status csa_draft_commit(const csa_commit_args* a, void* stream) {
  if (!a || a->num_req < 0 || a->pt_stride < 0 || a->path_stride < 0 || a->num_layers < 1 || a->room < 0 || !a->n_freed || (a->room > 0 && !a->freed))
    return CSA_ERR_INVALID_ARG;
  if (a->num_req > CSA_COMMIT_MAX_REQ) return CSA_ERR_UNSUPPORTED;
  int columns = 1, groups = 0;  // 16-byte columns of a record; blocks a request
  if (a->num_req > 0) {
    const csa_status st = check_cache(a->cache);
    if (st != CSA_OK) return st;
    const int64_t rec = csa_latent_record_bytes(a->cache.record_format, a->cache.rope_dim);
    if (!a->page_table || a->pt_stride < 1 || static_cast<int64_t>(kPageRecs) * a->pt_stride > INT32_MAX || !a->base_len || !a->draft_len ||
        !a->path_len || !a->new_len || (a->path_stride > 0 && !a->path))
      return CSA_ERR_INVALID_ARG;
    if (a->new_len == a->base_len || a->new_len == a->draft_len || a->new_len == a->path_len) return CSA_ERR_INVALID_ARG;  // read by other blocks
    if (a->num_layers > 1 && a->layer_stride_bytes < kPageRecs * rec) return CSA_ERR_INVALID_ARG;
    columns = static_cast<int>(rec / 16);
    groups = (a->num_layers - 1) / (kCommitThreads / columns) + 1;
    if (static_cast<int64_t>(groups) * a->num_req >= INT32_MAX) return CSA_ERR_INVALID_ARG;
  }
  if (a->layer_stride_bytes % 16 != 0 || !aligned(a->page_table, 4) || !aligned(a->base_len, 4) || !aligned(a->draft_len, 4) || !aligned(a->path, 4) ||
      !aligned(a->path_len, 4) || !aligned(a->new_len, 4) || !aligned(a->freed, 4) || !aligned(a->n_freed, 4) || !aligned(a->dev_status, 4))
    return CSA_ERR_ALIGNMENT;
  commit_kernel<<<1 + groups * a->num_req, kCommitThreads, 0, static_cast<cudaStream_t>(stream)>>>(*a, columns);
  return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}
