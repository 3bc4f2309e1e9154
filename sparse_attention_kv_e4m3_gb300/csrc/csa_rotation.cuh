// csa_rotation.cuh — the position rotation's angles and the norm of a row, as the kernels that rotate share them
// (include/csa_draft.h).
#pragma once

#include "csa_draft.h"
#include "csa_latent_common.cuh"

namespace csa_latent {
namespace {

// Turns a token of a frequency, freq / 2 pi modulo 1, in units of 2^-64 (the last bit is 0). A position times this, modulo 2^64,
// is the angle: an exact integer product, so a far position loses nothing, where a product in fp32 is off by a radian at
// position 2^24. 1 / 2 pi is two doubles; the first product's rounding error comes back through an fma, so the result is
// right to 2^-63, and an angle at position 2^31 to 2^-32 turns.
__device__ __forceinline__ uint64_t turns_per_token(float freq) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;  // 1 / 2 pi = kHi + kLo to 2^-109
  const double f = freq, p = f * kHi, rest = fma(f, kHi, -p) + f * kLo;
  const double part = p - rint(p);  // exact, -1/2 .. 1/2
  const int64_t units = __double2ll_rn(part * 0x1p63) + __double2ll_rn(rest * 0x1p63);
  return static_cast<uint64_t>(units) << 1;
}

// cos and sin of the angle, times the rotation's scale: 2^-32 turns are taken to fp32 (2^-25 relative) and through sincospif.
__device__ __forceinline__ float2 cos_sin(uint64_t per_token, int32_t pos, float scale) {
  const uint64_t turns = per_token * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const float half_turns = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * scale, s * scale);
}

// Whether a mean of squares (plus eps) computed in fp32 can be relied on: no square that matters has overflowed or vanished. Where
// not, the sum is taken again in fp64, which holds the square of any fp32 value.
__device__ __forceinline__ bool plain_mean(float mean_eps) { return mean_eps > 1e-30f && mean_eps < 1e36f; }

// A norm's factor in two steps. It may leave fp32's normal numbers where the normed values do not: these take a power of two of it first, which
// is exact (upwards always; downwards but for values that the factor makes 0).
struct Factor {
  float first, rest;
};

__device__ __forceinline__ Factor factor_of(double all) {
  const float first = all > 0x1p100 ? 0x1p64f : (all < 0x1p-126 ? 0x1p-8f : 1.f);
  return {first, static_cast<float>(all / first)};
}

inline bool good_eps(float eps) { return eps >= 0.f && eps < INFINITY; }

inline csa_status check_rotation(const csa_rotation& r) {
  if (r.reserved0 != 0 || (r.pairing != CSA_PAIRS_ADJACENT && r.pairing != CSA_PAIRS_HALVES)) return CSA_ERR_INVALID_ARG;
  if (!(r.scale > -INFINITY && r.scale < INFINITY)) return CSA_ERR_INVALID_ARG;
  if (r.rope_dim < 0 || (r.rope_dim > 0 && !r.freq)) return CSA_ERR_INVALID_ARG;
  return aligned(r.freq, 4) ? CSA_OK : CSA_ERR_ALIGNMENT;
}

}  // namespace
}  // namespace csa_latent
