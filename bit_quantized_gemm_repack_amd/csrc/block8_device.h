// Device helpers of the fp8 x fp8 kernels with 128-block scales.
#pragma once

#include "device_common.h"

namespace hq {

// P[r] = sum_k w[n = 4 (l / 16) + r, k] a[token l % 16, k] over 128 k, exact
// products in fp32 accumulation: the weight is the first operand, so a lane
// holds four consecutive columns of one token, and the token's scale is one
// value per lane.  Scale arguments 0 select the form without block scales.
__device__ inline f4_t b8_mfma(i8_t w, i8_t a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, f4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// Four fp32 values over their block's scale -> e4m3 codes, little-endian:
// the correctly rounded quotient, rounded to nearest even and saturated at
// 448 (-0 gives code 0, as in the per-token quantiser); NaN gives NaN.
__device__ inline uint32_t b8_codes(float v0, float v1, float v2, float v3, float s) {
  auto q = [&](float v) {
    const float x = v / s;
    return x != x ? x : __builtin_amdgcn_fmed3f(x, 448.f, -448.f);
  };
  int t = __builtin_amdgcn_cvt_pk_fp8_f32(q(v0), q(v1), 0, false);
  t = __builtin_amdgcn_cvt_pk_fp8_f32(q(v2), q(v3), t, true);
  const uint32_t u = (uint32_t)t;
  const uint32_t nz = ((u & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) & 0x80808080u;
  return u & (0x7F7F7F7Fu | nz);
}

// The scale of a block from its largest magnitude: max / 448, 1 where that is
// zero (a block of zeros, or of values under 448 * 2^-150), NaN where the block holds a value that is not finite (`top` is
// NaN or infinite then).
__device__ inline float b8_scale(uint32_t top_bits) {
  const float top = __uint_as_float(top_bits);
  if (!(top < __builtin_inff())) return __builtin_nanf("");
  const float s = top / 448.f;
  return s > 0.f ? s : 1.f;
}

// Magnitudes are compared as the bits of their absolute values: an infinity
// is above every number and a NaN above both, so neither is lost.
__device__ inline uint32_t b8_mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ inline float b8_silu_mul(float g, float u) { return g / (1.f + expf(-g)) * u; }

}  // namespace hq
