// csa_latent_ptx.cuh — the tensor-core building blocks of the latent attention
// kernels beyond csa_ptx.cuh: bf16 MMAs and their operand descriptors.
#pragma once

#include <cstdint>

// Internal linkage: the out-of-line waits of csa_ptx.cuh are not inline, and more
// than one translation unit of the library includes them.
namespace {

#include "csa_ptx.cuh"

namespace csa {

// Instruction descriptor of a dense kind::f16 MMA with bf16 A and B and an fp32
// accumulator, shape M x N: accumulator format in bits 4-5 (1 = f32), A / B formats
// in bits 7-9 / 10-12 (1 = bf16), A / B transposed (MN-major) in bits 15 / 16,
// N >> 3 in bits 17-22, M >> 4 in bits 24-28.
constexpr uint32_t kIdescAMnMajor = 1u << 15;
__host__ __device__ constexpr uint32_t idesc_bf16_f32(uint32_t M, uint32_t N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// MN-major operand of 16-bit elements in the 128-byte swizzle layout: a row holds 64
// consecutive M (or N) elements at one K index, 8 consecutive K rows form a 1024-byte
// atom, atoms follow each other along K (stride-dimension offset 1024 B), and the next
// 64 elements along M lie `group_bytes` further (leading-dimension offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128_b16(uint32_t saddr, uint32_t group_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(group_bytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// D[tmem] (+)= A[smem] * B[smem]^T, one CTA, kind::f16 (K = 16 per call).
__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 2^x: 2^-22 relative error, subnormal results become 0, 2^-infinity is 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Whether `p` holds for any of the `nthreads` threads that meet at barrier `id`.
__device__ __forceinline__ bool named_bar_any(int id, int nthreads, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p)), "r"(id), "r"(nthreads)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 16 bytes global -> shared without a register, or zeros when !live (src is not read then).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

}  // namespace csa

}  // namespace
