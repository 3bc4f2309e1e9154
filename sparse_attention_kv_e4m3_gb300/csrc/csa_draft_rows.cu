// csa_draft_rows.cu — norms and rotation of queries and keys, the writer that norms and rotates on the way,
// and the move of accepted drafts' records (include/csa_draft.h). All three are one pass over their data.
#include "csa_latent_rows.cuh"
#include "csa_rotation.cuh"

namespace csa_latent {
namespace {

// ------------------------------------------------------------- norm and rotation of heads
//
// A group of 8, 16 or 32 lanes takes a head, a lane 8 values of each 256 (16 or 32 bytes a load). A head's values stay
// in registers between the sum of squares and the store, so every value is read and written once; a rotated pair of halves
// comes from another lane's values, which are loaded again (from L1) rather than exchanged, because where the rotated
// part begins is free. The rows' cosines and sines are made once a block, in shared memory, for all heads of the row.

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
  __device__ __forceinline__ void store(void* p) const {
#pragma unroll
    for (int k = 0; k < (kF32 ? 2 : 1); ++k) reinterpret_cast<uint4*>(p)[k] = w[k];
  }
};

struct RotateKernel {
  csa_rotate_args A;
  int32_t q_blocks, q_items, k_items;  // blocks of the queries; heads a block, of each tensor
};

// Lanes of a head, and heads that a block takes at a time.
__host__ __device__ constexpr int lanes_of(int dim) { return dim <= 64 ? 8 : (dim <= 128 ? 16 : 32); }

template <bool kF32In, bool kF32Out, int kChunks, int kHeadsInFlight>
__global__ void __launch_bounds__(kRotThreads) rotate_kernel(const RotateKernel K) {
  extern __shared__ float2 turns[];  // [rows of the block][rope_dim / 2] cos, sin
  __shared__ uint64_t per_token[CSA_ROTATE_MAX_ROPE / 2];
  const csa_rotate_args& A = K.A;
  const bool is_q = static_cast<int>(blockIdx.x) < K.q_blocks;
  const csa_heads& T = is_q ? A.q : A.k;
  const int64_t per = is_q ? K.q_items : K.k_items;
  const int64_t first = per * (is_q ? blockIdx.x : blockIdx.x - K.q_blocks);
  const int64_t last = min(first + per, A.n * T.heads);  // heads first .. last of all rows' heads
  const int64_t row0 = first / T.heads;
  const int half = A.rotation.rope_dim / 2;
  int32_t flags = 0;
  if (half > 0) {
    for (int j = threadIdx.x; j < half; j += kRotThreads) per_token[j] = turns_per_token(A.rotation.freq[j]);
    __syncthreads();
    const int rows = static_cast<int>((last - 1) / T.heads - row0 + 1);
    for (int i = threadIdx.x; i < rows * half; i += kRotThreads) turns[i] = cos_sin(per_token[i % half], A.pos[row0 + i / half], A.rotation.scale);
    __syncthreads();
  }
  const int G = lanes_of(T.dim), lane = threadIdx.x & (G - 1), chunks = T.dim / 8;
  const uint32_t mates = (G == 32 ? 0xFFFFFFFFu : (1u << G) - 1u) << (threadIdx.x & 31 & ~(G - 1));
  // of the head's chunks of 8 values, those that rotate, and how far apart halves lie
  const int turn0 = A.rope_first ? 0 : chunks - half / 4, turn1 = turn0 + half / 4, apart = half / 8;
  const bool halves = A.rotation.pairing == CSA_PAIRS_HALVES;
  constexpr int kIn = kF32In ? 4 : 2, kOut = kF32Out ? 4 : 2;
  const int64_t step = kRotThreads / G;
  for (int64_t at = first + threadIdx.x / G; at - threadIdx.x / G < last; at += kHeadsInFlight * step) {
    Eight<kF32In> x[kHeadsInFlight][kChunks], other[kHeadsInFlight][kChunks];
    int64_t row[kHeadsInFlight], head[kHeadsInFlight];
    bool live[kHeadsInFlight];
#pragma unroll
    for (int i = 0; i < kHeadsInFlight; ++i) {
      const int64_t item = at + i * step;
      live[i] = item < last;
      row[i] = live[i] ? item / T.heads : row0;
      head[i] = live[i] ? item % T.heads : 0;
      if (A.pos) {
        const int32_t p = A.pos[row[i]];
        if (live[i] && p < -1) flags |= CSA_DEV_LEN_OOB;
        live[i] = live[i] && p >= 0;
      }
      const uint8_t* src = static_cast<const uint8_t*>(T.x) + kIn * (row[i] * T.x_row_stride + head[i] * T.x_head_stride);
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const int c = lane + G * k;
        if (!live[i] || c >= chunks) continue;
        x[i][k].load(src + 8 * kIn * c);
        if (halves && c >= turn0 && c < turn1) other[i][k].load(src + 8 * kIn * (c < turn0 + apart ? c + apart : c - apart));
      }
    }
    __syncwarp();  // in place: all of a head is read before any of it is written
#pragma unroll
    for (int i = 0; i < kHeadsInFlight; ++i) {
      float r = 1.f;
      if (T.norm) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
          if (!live[i] || lane + G * k >= chunks) continue;
          float v[8];
          x[i][k].get(v);
#pragma unroll
          for (int j = 0; j < 8; ++j) sum = fmaf(v[j], v[j], sum);
        }
        for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float mean = sum / static_cast<float>(T.dim) + A.eps;
        r = 1.f / sqrtf(mean);
        if (!plain_mean(mean)) {  // the same for all lanes of the head
          double wide = 0.0;
#pragma unroll
          for (int k = 0; k < kChunks; ++k) {
            if (!live[i] || lane + G * k >= chunks) continue;
            float v[8];
            x[i][k].get(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) wide += static_cast<double>(v[j]) * v[j];
          }
          for (int o = G / 2; o > 0; o >>= 1) wide += __shfl_xor_sync(mates, wide, o);
          r = static_cast<float>(1.0 / sqrt(wide / T.dim + A.eps));
        }
      }
      if (!live[i]) continue;
      uint8_t* dst = static_cast<uint8_t*>(T.out) + kOut * (row[i] * T.out_row_stride + head[i] * T.out_head_stride);
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const int c = lane + G * k;
        if (c >= chunks) continue;
        float v[8];
        x[i][k].get(v);
        auto scale = [&](float (&y)[8], int chunk) {
          if (!T.norm) return;
          float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
          if (T.weight) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(T.weight) + 2 * chunk), b = __ldg(reinterpret_cast<const float4*>(T.weight) + 2 * chunk + 1);
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = y[j] * r * w[j];
        };
        scale(v, c);
        if (c >= turn0 && c < turn1) {
          const float2* t = turns + (row[i] - row0) * half;
          if (halves) {
            const bool low = c < turn0 + apart;
            float u[8];
            other[i][k].get(u);
            scale(u, low ? c + apart : c - apart);
            t += 8 * (low ? c - turn0 : c - turn0 - apart);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = low ? v[j] * t[j].x - u[j] * t[j].y : v[j] * t[j].x + u[j] * t[j].y;
          } else {
            t += 4 * (c - turn0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float a = v[2 * j], b = v[2 * j + 1];
              v[2 * j] = a * t[j].x - b * t[j].y;
              v[2 * j + 1] = b * t[j].x + a * t[j].y;
            }
          }
        }
        Eight<kF32Out> y;
        y.put(v);
        y.store(dst + 8 * kOut * c);
      }
    }
  }
  flags = static_cast<int32_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(flags)));
  if (flags && A.dev_status && (threadIdx.x & 31) == 0) atomicOr(A.dev_status, flags);
}

template <bool kF32In, bool kF32Out, int kChunks, int kHeadsInFlight>
csa_status launch_rotate(RotateKernel& K, cudaStream_t stream) {
  const csa_rotate_args& a = K.A;
  auto items = [](const csa_heads& t) { return kHeadsInFlight * kRotThreads / lanes_of(t.dim); };
  auto blocks = [&](const csa_heads& t) { return t.heads > 0 ? (a.n * t.heads + items(t) - 1) / items(t) : 0; };
  auto rows = [&](const csa_heads& t) { return t.heads > 0 ? (items(t) - 1) / t.heads + 2 : 0; };  // that a block's heads can be of
  K.q_items = a.q.heads > 0 ? items(a.q) : 0;
  K.k_items = a.k.heads > 0 ? items(a.k) : 0;
  const int64_t grid = blocks(a.q) + blocks(a.k);
  if (grid > INT32_MAX) return CSA_ERR_INVALID_ARG;
  K.q_blocks = static_cast<int32_t>(blocks(a.q));
  const int most = rows(a.q) > rows(a.k) ? rows(a.q) : rows(a.k);
  const size_t smem = sizeof(float2) * most * (a.rotation.rope_dim / 2);
  rotate_kernel<kF32In, kF32Out, kChunks, kHeadsInFlight><<<static_cast<unsigned>(grid), kRotThreads, smem, stream>>>(K);
  return cudaGetLastError() == cudaSuccess ? CSA_OK : CSA_ERR_CUDA;
}

template <bool kF32In, bool kF32Out>
csa_status launch_rotate_dim(RotateKernel& K, cudaStream_t stream) {
  const int q = K.A.q.heads > 0 ? K.A.q.dim : 0, k = K.A.k.heads > 0 ? K.A.k.dim : 0, dim = q > k ? q : k;
  if (dim <= 256) return launch_rotate<kF32In, kF32Out, 1, 2>(K, stream);
  return dim <= 512 ? launch_rotate<kF32In, kF32Out, 2, 1>(K, stream) : launch_rotate<kF32In, kF32Out, 4, 1>(K, stream);
}

csa_status check_heads(const csa_heads& t, int64_t n, int rope, bool f32_in, bool f32_out) {
  if (t.heads < 0) return CSA_ERR_INVALID_ARG;
  if (t.heads == 0) return CSA_OK;
  if (t.reserved0 != 0 || (t.norm != 0 && t.norm != 1)) return CSA_ERR_INVALID_ARG;
  if (t.dim < 8 || t.dim > CSA_ROTATE_MAX_DIM || t.dim % 8 != 0) return CSA_ERR_UNSUPPORTED;
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
// twice, a little larger and a little smaller; where the two differ anywhere in the row (about one row in 100) the row is
// computed again in fp64.

// The relative error of x r w in fp32: the sum of 16 squares a lane and 5 steps over the lanes, (16 + 5) 2^-24, the division
// and eps 2 x 2^-24, halved by the root; root, reciprocal and two products 4 x 2^-24 more. 2^-19 is more than twice that.
constexpr float kNear = 0x1p-19f;

// Codes and exponent of a lane's values in fp64: the exact norm's, next to a border too.
__device__ __noinline__ void encode_exact(const float (&x)[16], const float (&w)[16], float eps, Coded<true>& c) {
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < 16; ++k) sum += static_cast<double>(x[k]) * x[k];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  const double r = 1.0 / sqrt(sum / kDim + eps);
  double amax = 0.0;
  bool bad = false;
#pragma unroll 1
  for (int k = 0; k < 16; ++k) {
    const double y = fabs(x[k] * r * w[k]);
    bad |= !(y < 0x1.ffffffp127);  // what rounds to a finite fp32, and no NaN
    amax = fmax(amax, y);
  }
  amax = fmax(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  c.bad = bad;
  // floor(log2 amax) - 2, held at -127 (a double that is subnormal lies far below)
  c.e = max(static_cast<int>(__double2hiint(amax) >> 20) - 1023 - 2, -127);
  const double up = __hiloint2double((1023 - c.e) << 20, 0);
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    c.w[h] = 0;
#pragma unroll 1
    for (int k = 0; k < 8; ++k) {
      const double y = x[8 * h + k] * r * w[8 * h + k], t = fabs(y) * up;
      const uint32_t m = (t > 0.25) + (t >= 0.75) + (t > 1.25) + (t >= 1.75) + (t > 2.5) + (t >= 3.5) + (t > 5.0);
      c.w[h] |= (m | (signbit(y) ? 8u : 0u)) << (4 * k);
    }
  }
}

template <bool kBf16In, bool kFp4>
__device__ __forceinline__ int32_t append_row(const csa_append_args& A, RowIn<kBf16In>& x, const float (&w)[16], const uint64_t (&per_token)[2],
                                              int64_t slot, int32_t pos, int lane) {
  if (slot == -1) return 0;
  if (slot < 0 || slot >= A.cache.num_pages * kPageRecs) return CSA_DEV_PAGE_OOB;
  const bool rope = A.cache.rope_dim != 0;
  uint32_t rope_word = 0;
  if (rope) {
    if (pos < 0) return CSA_DEV_LEN_OOB;
    const float2 t = cos_sin(per_token[0], pos, A.rotation.scale);
    float a = x.r[0], b = x.r[1];
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
    const float mean = sum / kDim + A.eps;
    float r = 1.f / sqrtf(mean);
    const bool plain = plain_mean(mean);
    if (!kFp4 && !plain) {
      double wide = 0.0;
#pragma unroll
      for (int k = 0; k < 16; ++k) wide += static_cast<double>(x.v[k]) * x.v[k];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) wide += __shfl_xor_sync(0xFFFFFFFFu, wide, o);
      r = static_cast<float>(1.0 / sqrt(wide / kDim + A.eps));
    }
    float y[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) y[k] = x.v[k] * r * w[k];
    c = encode<kFp4>(y);
    if constexpr (kFp4) {
      // the same codes and exponent a little further out and in
      uint32_t amax = 0;
#pragma unroll
      for (int k = 0; k < 16; ++k) amax = max(amax, __float_as_uint(y[k]) & 0x7FFFFFFFu);
      amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      const float top = __uint_as_float(amax), out = 1.f + kNear, in = 1.f - kNear, up = block_up(c.e);
      // below 2^-100 products and borders leave fp32's normal range
      bool near = !plain || !(top > 0x1p-100f && top < 0x1p100f) || block_exponent(__float_as_uint(top * out)) != c.e || block_exponent(__float_as_uint(top * in)) != c.e;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a = 0, b = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a |= e2m1_pair(y[8 * h + 2 * k] * (up * out), y[8 * h + 2 * k + 1] * (up * out)) << (8 * k);
          b |= e2m1_pair(y[8 * h + 2 * k] * (up * in), y[8 * h + 2 * k + 1] * (up * in)) << (8 * k);
        }
        near |= a != b;
      }
      if (__any_sync(0xFFFFFFFFu, near)) encode_exact(x.v, w, A.eps, c);
    }
  }
  if (__any_sync(0xFFFFFFFFu, c.bad || nonfinite_bf16x2(rope_word))) return CSA_DEV_RANGE;
  put_record<kFp4>(A.cache, slot, c, rope_word, lane);
  return 0;
}

template <bool kBf16In, bool kFp4>
__global__ void __launch_bounds__(kCopyThreads) append_kernel(const csa_append_args A) {
  constexpr int kRowsInFlight = kBf16In ? 4 : 2;
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kCopyThreads / 32);
  int32_t flags = 0;
  float w[16];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 v = A.norm && A.weight ? __ldg(reinterpret_cast<const float4*>(A.weight) + 4 * lane + k) : make_float4(1.f, 1.f, 1.f, 1.f);
    w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
  }
  uint64_t per_token[2] = {0, 0};
  if (A.cache.rope_dim != 0) {
    const bool adjacent = A.rotation.pairing == CSA_PAIRS_ADJACENT;
    per_token[0] = turns_per_token(A.rotation.freq[adjacent ? lane : 2 * lane & 31]);
    if (!adjacent) per_token[1] = turns_per_token(A.rotation.freq[(2 * lane & 31) + 1]);
  }
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x) >> 5; i < A.n; i += kRowsInFlight * warps) {
    int64_t slot[kRowsInFlight];
    int32_t pos[kRowsInFlight];
    RowIn<kBf16In> x[kRowsInFlight];
#pragma unroll
    for (int k = 0; k < kRowsInFlight; ++k) {
      const int64_t r = i + k * warps, at = r < A.n ? r : i;
      slot[k] = r < A.n ? A.slots[r] : -1;
      pos[k] = A.cache.rope_dim != 0 ? A.pos[at] : 0;
      x[k].load(static_cast<const uint8_t*>(A.x) + at * A.x_stride * (kBf16In ? 2 : 4), lane, A.cache.rope_dim);
    }
#pragma unroll
    for (int k = 0; k < kRowsInFlight; ++k) flags |= append_row<kBf16In, kFp4>(A, x[k], w, per_token, slot[k], pos[k], lane);
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
// moves anything.

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
  RotateKernel K = {*a, 0, 0, 0};
  const auto s = static_cast<cudaStream_t>(stream);
  if (f32_in) return f32_out ? launch_rotate_dim<true, true>(K, s) : launch_rotate_dim<true, false>(K, s);
  return f32_out ? launch_rotate_dim<false, true>(K, s) : launch_rotate_dim<false, false>(K, s);
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
