// Device helpers of the MXFP4 products: the matrix instruction, a step's powers of two, and
// a block of the intermediate from the operand layout to its codes.
#pragma once

#include "block8_device.h"
#include "mx4.h"
#include "mx4_device.h"

namespace hq {

// acc += W . A^T over 128 k: the weight is the first operand, so a lane (token l % 16)
// holds four consecutive columns.  Byte J of sw and byte 0 of sa: the powers of two of this
// lane's 32 k of its weight column and of its activation row.
template <int J>
__device__ __forceinline__ f4_t mx4_mfma(u4_t w, u4_t a, f4_t acc, uint32_t sw, uint32_t sa) {
#if defined(__HIP_DEVICE_COMPILE__)
  const i8_t wv = i8_t{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  const i8_t av = i8_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, acc, 4, 4, J, (int)sw, 0, (int)sa);
#else
  return acc;
#endif
}
// The four fragments of a strip.
__device__ __forceinline__ void mx4_strip(const u4_t (&w)[4], u4_t a, f4_t (&acc)[4], uint32_t sw, uint32_t sa) {
  acc[0] = mx4_mfma<0>(w[0], a, acc[0], sw, sa);
  acc[1] = mx4_mfma<1>(w[1], a, acc[1], sw, sa);
  acc[2] = mx4_mfma<2>(w[2], a, acc[2], sw, sa);
  acc[3] = mx4_mfma<3>(w[3], a, acc[3], sw, sa);
}

// The powers of two of the step at byte `at`: a word a group.
template <int Q>
struct Mx4Scales {
  uint32_t v[Q];
  template <int AUX>
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int lane, int at) {
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (Q == 2) {
      const auto x = __builtin_amdgcn_raw_buffer_load_b64(r, lane * 8, at + 8192, AUX);
      v[0] = x[0];
      v[1] = x[1];
    } else {
      v[0] = __builtin_amdgcn_raw_buffer_load_b32(r, lane * 4, at + 4096, AUX);
    }
#endif
  }
};

// A block of 32 outputs of one row (lane l % 16) from the operand layout: v[0 .. 3] are its
// columns 4 kq .. + 3, v[4 .. 7] those 16 further (kq = l / 16).  s: the block's scale byte.
// Returns four bytes of codes, those at 8 (kq & 1) + 4 (kq >> 1) of the block's 16: lanes of
// odd kq give the first half to their neighbour and take its second.
__device__ inline uint32_t mx4_block_codes(const float (&v)[8], int kq, uint32_t& s) {
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, b8_mag(v[i]));
  top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
  top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
  s = mx4_scale(top);
  const uint32_t word = mx4_word(v, s);
  const uint32_t give = kq & 1 ? word & 0xFFFFu : word >> 16;
  const uint32_t got = (uint32_t)__shfl_xor((int)give, 16, 64);
  return kq & 1 ? got | (word & 0xFFFF0000u) : (word & 0xFFFFu) | (got << 16);
}

}  // namespace hq
