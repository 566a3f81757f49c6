// Device helpers of MXFP4 values: E2M1 elements with one power of two per 32.
#pragma once

#include "device_common.h"

namespace hq {

// Round-to-nearest-even fp32 -> E2M1 code, saturating at 6; -0 gives code 0.
// Below 1 the spacing is 0.5 (code = rint(2|x|)); above, the 23-bit mantissa
// is rounded to 1 bit (a carry moves into the exponent field).
__device__ inline uint32_t e2m1_code_rne(float x) {
  const uint32_t sign = (__float_as_uint(x) >> 28) & 0x8u;
  const float a = fminf(fabsf(x), 6.f);
  uint32_t code;
  if (a < 1.f) {
    code = (uint32_t)__builtin_rintf(a * 2.f);
  } else {
    const uint32_t bits = __float_as_uint(a);
    const uint32_t e = (bits >> 23) - 127u + 1u;  // exponent field, bias 1
    const uint32_t mant = bits & 0x7FFFFFu;
    const uint32_t r = (mant + 0x1FFFFFu + ((mant >> 22) & 1u)) >> 22;  // 0..2
    code = (e << 1) + r;
  }
  return code == 0 ? 0u : (sign | code);
}

// The E8M0 byte of a block from the bits of its largest magnitude: X + 127 with
// X = floor(log2 max) - 2 (2 = the largest E2M1 exponent), clamped to [-127, 127];
// X = 0 for a block of zeros, and the format's NaN (255) where the block holds a
// value that is not finite.
__device__ inline uint32_t mx4_scale(uint32_t top_bits) {
  if (top_bits >= 0x7F800000u) return 255u;
  if (top_bits == 0u) return 127u;
  return (uint32_t)max((int)(top_bits >> 23) - 2, 0);  // (a subnormal maximum clamps to -127)
}

// v / 2^X (exact but for results below fp32's range, which round to zero as
// elements either way).
__device__ inline float mx4_scaled(float v, uint32_t scale) { return __builtin_amdgcn_ldexpf(v, 127 - (int)scale); }

// Eight values of a block -> a word of codes, the first in the lowest bits: the
// hardware conversion, which agrees with e2m1_code_rne(mx4_scaled()) for every value
// that a block's scale leaves below 8 (checked exhaustively) but for the codes of -0,
// and a quarter of its instructions.  Blocks at the exponents' end go the long way.
__device__ inline uint32_t mx4_word(const float (&v)[8], uint32_t scale) {
  uint32_t w = 0u;
  if (scale == 0u) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w |= e2m1_code_rne(mx4_scaled(v[j], 0u)) << (4 * j);
    return w;
  }
#if defined(__HIP_DEVICE_COMPILE__)
  const float s = __uint_as_float(scale << 23);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
#endif
  return w & (0x77777777u | (((w & 0x77777777u) + 0x77777777u) & 0x88888888u));
}

// Maximum over the four lanes that share lane / 4, in each of them.
__device__ inline uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));  // quad_perm 1 0 3 2
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));  // quad_perm 2 3 0 1
}

// The scale bytes of the four blocks that 16 neighbouring lanes hold (four lanes each), as
// a word in each of them.
__device__ inline uint32_t mx4_scale_word(uint32_t s) {
  uint32_t all = 0u;
#pragma unroll
  for (int b = 0; b < 4; ++b) all |= (uint32_t)__shfl((int)s, ((int)threadIdx.x & 48) + 4 * b, 64) << (8 * b);
  return all;
}

}  // namespace hq
