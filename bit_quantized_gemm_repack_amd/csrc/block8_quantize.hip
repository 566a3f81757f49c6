// The block quantiser of fp8 activations, and the repack of fp8 weights with
// 128 x 128 scales.
//
// Quantiser: a block is 128 consecutive values of a row,
//   s = max|v| / 448 (fp32; 1 where that is zero), code = RNE_e4m3(v / s),
// v being x or SiLU(x[:, :k]) * x[:, k:] formed in fp32.  Memory-bound: x is
// read once and held in registers between the maximum and the codes.  Sixteen
// lanes hold a block (8 values, one 16-byte load each), so the maximum is
// four rotations within the lanes' row.  Workgroups of 4 rows by 4 block columns
// run along the rows, so that memory sees runs of 1 KiB (16 rows of one column:
// 5 % more).  Ordinary loads: what the kernel before has left in the last-level
// cache is found there (4096 x 7168 15.9 us against 19.6 with loads that pass it
// by).  One token of 7168: 2.6 us in a graph, a launch; SiLU of 8191 x 2048, 84 MB:
// 18.9 .. 20.8 us a call, 4.0 .. 4.4 TB/s (a large copy reaches 4.9); 4096 x 7168, 88
// MB: 15.9 us with x in the last-level cache, 18.5 in a layer of that many tokens.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "block8.h"
#include "block8_device.h"
#include "launch.h"

namespace hq {

namespace {

template <bool BF16, bool SILU>
__global__ void __launch_bounds__(256) quantize_blocks_kernel(const u4_t* __restrict__ x, uint32_t m, uint32_t k8,
                                                              uint2* __restrict__ codes, float* __restrict__ scales) {
  // a workgroup takes 4 rows by 4 block columns, a wave 4 rows of one column
  const uint32_t G = k8 / 16, quads = (G + 3) / 4, block = grid_block(), rq = block / quads;
  const uint32_t g = (block - rq * quads) * 4 + (threadIdx.x >> 6), row = rq * 4 + ((threadIdx.x >> 4) & 3);
  if (g >= G || row >= m) return;
  const uint32_t c = g * 16 + (threadIdx.x & 15);
  float v[8];
  if constexpr (SILU) {
    const u4_t* r = x + (int64_t)row * 2 * k8 + c;
    const u4_t xg = r[0], xu = r[k8];
    float u[8];
    b8_unpack<BF16>(xg, v);
    b8_unpack<BF16>(xu, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = b8_silu_mul(v[j], u[j]);
  } else {
    b8_unpack<BF16>(x[(int64_t)row * k8 + c], v);
  }
  uint32_t top = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, b8_mag(v[j]));
  const float s = b8_scale(b8_row_max(top));
  const B8Div d(s);
  codes[(int64_t)row * k8 + c] = uint2{b8_codes(v[0], v[1], v[2], v[3], d), b8_codes(v[4], v[5], v[6], v[7], d)};
  if ((threadIdx.x & 15) == 0) scales[(int64_t)g * m + row] = s;
}

__global__ void repack_b8_kernel(const uint8_t* __restrict__ codes, uint32_t* __restrict__ out, int64_t K,
                                 int64_t words_per_expert, int64_t total) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t e = i / words_per_expert;
    out[i] = repack_word_b8(codes + e * words_per_expert * 4, K, i - e * words_per_expert);
  }
}

__global__ void copy_words_kernel(const uint32_t* __restrict__ src, uint32_t* __restrict__ dst, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    dst[i] = src[i];
}

dim3 grid_for(int64_t n) { return dim3((unsigned)std::min<int64_t>(std::max<int64_t>((n + 255) / 256, 1), 65536)); }

}  // namespace

int launch_quantize_blocks(int64_t m, int64_t k, int in_bf16, int silu, const void* x, void* codes, float* scales,
                           void* stream) {
  const int64_t blocks = m * (k / 128);
  if (blocks < 1 || blocks > INT32_MAX - 16) return (int)hipErrorInvalidValue;
  const dim3 grid = grid_of((k / 128 + 3) / 4 * ((m + 3) / 4)), block(256);
  const auto xs = static_cast<const u4_t*>(x);
  const auto cs = static_cast<uint2*>(codes);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const uint32_t mu = (uint32_t)m, k8 = (uint32_t)(k / 8);
  if (in_bf16)
    return silu ? (int)launch_timed(quantize_blocks_kernel<true, true>, grid, block, 0, s, xs, mu, k8, cs, scales)
                : (int)launch_timed(quantize_blocks_kernel<true, false>, grid, block, 0, s, xs, mu, k8, cs, scales);
  return silu ? (int)launch_timed(quantize_blocks_kernel<false, true>, grid, block, 0, s, xs, mu, k8, cs, scales)
              : (int)launch_timed(quantize_blocks_kernel<false, false>, grid, block, 0, s, xs, mu, k8, cs, scales);
}

int launch_b8_repack(int64_t N, int64_t K, int64_t E, const void* codes, const void* scales, void* w_out,
                     void* meta_out, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t words = N * K / 4, nsc = (N + 127) / 128 * (K / 128) * E;
  hipLaunchKernelGGL(repack_b8_kernel, grid_for(words * E), dim3(256), 0, s, static_cast<const uint8_t*>(codes),
                     static_cast<uint32_t*>(w_out), K, words, words * E);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return (int)err;
  hipLaunchKernelGGL(copy_words_kernel, grid_for(nsc), dim3(256), 0, s, static_cast<const uint32_t*>(scales),
                     static_cast<uint32_t*>(meta_out), nsc);
  return (int)hipGetLastError();
}

}  // namespace hq
