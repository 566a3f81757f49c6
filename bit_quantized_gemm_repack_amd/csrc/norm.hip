// Root-mean-square norm with the residual's addition, its output in 16 bits or
// quantised for the product that reads it.
//
//   h = RN16(x + r)                   (h = x without a residual)
//   y = (h w) / sqrt(mean(h^2) + eps)
//
// out: y in x's type; or y quantised by row (e4m3, int8), by row and 128 columns
// (e4m3), or by 32 columns (MXFP4), by the rules of quantize.hip and
// block8_quantize.hip applied to the fp32 y.
//
// The factor 1 / sqrt(..) comes last, so that the largest |y| of a row or block is
// the largest |h w| times it (rounding keeps order): the sum of squares and the
// maxima need one pass over registers and one meeting of the row's threads.  h w
// is exact for 16-bit weights, so y rounds once more than the factor.
//
// Bound by memory: x, r and h are moved once.  With residual, start to end of the kernel:
// 8191 x 4096 fp16 to e4m3 by row 38.2 us, 6.1 TB/s (a streaming read reaches 6.4, a copy of
// 1 GiB 5.2); 8191 x 7168 bf16 in 16 bits 81 us, 5.8 TB/s, to e4m3 by 128 76, to int8 by row
// 75, to MXFP4 70, 5.5 TB/s.  Few rows are a chain of loads, sums and codes: one of 7168 to
// e4m3 by 128 3.5 us; 509 to MXFP4 8.5, 2.8 TB/s, the waves waiting half of their time.
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <algorithm>

#include "block8_device.h"
#include "launch.h"
#include "mx4_device.h"
#include "norm.h"

namespace hq {

namespace {

// Sum over the 16 lanes of a row, in every lane.
__device__ inline float lanes16_sum(float v) {
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// T threads a row (16, 64: several rows a workgroup of 256), each C chunks of 8
// values, chunk c of a row in thread c % T: a wave's loads are runs of 1 KiB, 4
// neighbouring lanes hold an MXFP4 block, 16 a block of 128.
template <bool BF16, int OUT, int T, int C>
__global__ void __launch_bounds__(T < 256 ? 256 : T) rms_norm_kernel(NormArgs p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int ROWS = T < 256 ? 256 / T : 1;
  __shared__ float2 red[T > 64 ? T / 64 : 1];
  const int tid = threadIdx.x, lane = tid % T;
  const int64_t row = (int64_t)blockIdx.x * ROWS + tid / T;
  if (T < 256 && row >= p.m) return;
  const u4_t* xr = static_cast<const u4_t*>(p.x) + row * p.x_stride;
  const u4_t* rr = static_cast<const u4_t*>(p.residual) + row * p.r_stride;
  const int k8 = p.k8;

  u4_t xv[C], rv[C], wv[C][2];
#pragma unroll
  for (int i = 0; i < C; ++i) xv[i] = xr[min(lane + T * i, k8 - 1)];
  if (p.residual) {
#pragma unroll
    for (int i = 0; i < C; ++i) rv[i] = rr[min(lane + T * i, k8 - 1)];
  }
  if (p.w_f32) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const u4_t* w = static_cast<const u4_t*>(p.weight) + 2 * min(lane + T * i, k8 - 1);
      wv[i][0] = w[0];
      wv[i][1] = w[1];
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) wv[i][0] = static_cast<const u4_t*>(p.weight)[min(lane + T * i, k8 - 1)];
  }

  float t[C][8], sum = 0.f;
  uint32_t top[C], row_top = 0u;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = lane + T * i;
    float v[8], w[8];
    b8_unpack<BF16>(xv[i], v);
    if (p.residual) {
      b8_unpack<BF16>(rv[i], w);
      u4_t h;
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // (the fp32 sum rounds to 16 bits as the exact one does)
        const float a = v[2 * j] + w[2 * j], b = v[2 * j + 1] + w[2 * j + 1];
        h[j] = BF16 ? (uint32_t)float_to_bf16_bits(a) | ((uint32_t)float_to_bf16_bits(b) << 16)
                    : (uint32_t)float_to_f16_bits(a) | ((uint32_t)float_to_f16_bits(b) << 16);
      }
      if (c < k8) static_cast<u4_t*>(p.h)[row * p.h_stride + c] = h;
      b8_unpack<BF16>(h, v);
    }
    if (p.w_f32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __uint_as_float(wv[i][j >> 2][j & 3]);
    } else {
      b8_unpack<BF16>(wv[i][0], w);
    }
    top[i] = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum = c < k8 ? fmaf(v[j], v[j], sum) : sum;
      t[i][j] = v[j] * w[j];
      top[i] = max(top[i], b8_mag(t[i][j]));
    }
    if (c < k8) row_top = max(row_top, top[i]);
  }

  // the row's sum, and its largest |h w| where the scale is the row's
  constexpr bool BY_ROW = OUT == NORM_FP8 || OUT == NORM_INT8;
  sum = lanes16_sum(sum);
  if constexpr (BY_ROW) row_top = b8_row_max(row_top);
  if constexpr (T >= 64) {
#pragma unroll
    for (int d = 32; d >= 16; d >>= 1) {
      sum += __shfl_xor(sum, d, 64);
      if constexpr (BY_ROW) row_top = max(row_top, (uint32_t)__shfl_xor((int)row_top, d, 64));
    }
  }
  if constexpr (T > 64) {
    if ((tid & 63) == 0) red[tid >> 6] = float2{sum, __uint_as_float(row_top)};
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int u = 0; u < T / 64; ++u) {
      const float2 o = red[u];
      sum += o.x;
      row_top = max(row_top, __float_as_uint(o.y));
    }
  }
  const float f = 1.f / sqrtf(sum / (float)(8 * k8) + p.eps);

  if constexpr (OUT == NORM_16) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = lane + T * i;
      u4_t o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = t[i][2 * j] * f, b = t[i][2 * j + 1] * f;
        o[j] = BF16 ? (uint32_t)float_to_bf16_bits(a) | ((uint32_t)float_to_bf16_bits(b) << 16)
                    : (uint32_t)float_to_f16_bits(a) | ((uint32_t)float_to_f16_bits(b) << 16);
      }
      if (c < k8) static_cast<u4_t*>(p.out)[row * k8 + c] = o;
    }
  } else if constexpr (BY_ROW) {
    const float most = __uint_as_float(row_top) * f;
    constexpr float Q = OUT == NORM_FP8 ? 448.f : 127.f;
    float s = most / Q;
    if (!(most < __builtin_inff())) s = __builtin_nanf("");
    else if (!(s > 0.f)) s = 1.f;
    const B8Div d(s);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = lane + T * i;
      uint2 o;
      if constexpr (OUT == NORM_FP8) {
        o = uint2{b8_codes(t[i][0] * f, t[i][1] * f, t[i][2] * f, t[i][3] * f, d),
                  b8_codes(t[i][4] * f, t[i][5] * f, t[i][6] * f, t[i][7] * f, d)};
      } else {
        uint32_t q[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          q[j >> 2] |= ((uint32_t)(int)__builtin_amdgcn_fmed3f(__builtin_rintf(d(t[i][j] * f)), 127.f, -127.f) & 0xFFu) << (8 * (j & 3));
        o = uint2{q[0], q[1]};
      }
      if (c < k8) static_cast<uint2*>(p.out)[row * k8 + c] = o;
    }
    if (lane == 0) static_cast<float*>(p.scale)[row] = s;
  } else if constexpr (OUT == NORM_FP8_BLOCK) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = lane + T * i;
      const float s = b8_scale(__float_as_uint(__uint_as_float(b8_row_max(top[i])) * f));
      const B8Div d(s);
      if (c < k8) {
        static_cast<uint2*>(p.out)[row * k8 + c] = uint2{b8_codes(t[i][0] * f, t[i][1] * f, t[i][2] * f, t[i][3] * f, d),
                                                         b8_codes(t[i][4] * f, t[i][5] * f, t[i][6] * f, t[i][7] * f, d)};
        if ((lane & 15) == 0) static_cast<float*>(p.scale)[(int64_t)(c >> 4) * p.m + row] = s;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = lane + T * i;
      const uint32_t s = mx4_scale(b8_mag(__uint_as_float(quad_max(top[i])) * f));
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = t[i][j] * f;
      const uint32_t word = mx4_word(y, s);
      const uint32_t all = mx4_scale_word(s);
      if (c < k8) {
        static_cast<uint32_t*>(p.out)[row * k8 + c] = word;
        if ((lane & 15) == 0) static_cast<uint32_t*>(p.scale)[(int64_t)(c >> 4) * p.m + row] = all;
      }
    }
  }
#endif
}

// The rows from `first` on; m stays the whole's, as the scales' layout goes by it.
template <int OUT>
NormArgs rows_from(NormArgs a, int64_t first) {
  constexpr int64_t CHUNK = OUT == NORM_16 ? 16 : (OUT == NORM_MXFP4 ? 4 : 8);  // bytes of 8 outputs
  a.x = static_cast<const u4_t*>(a.x) + first * a.x_stride;
  if (a.residual) {
    a.residual = static_cast<const u4_t*>(a.residual) + first * a.r_stride;
    a.h = static_cast<u4_t*>(a.h) + first * a.h_stride;
  }
  a.out = static_cast<char*>(a.out) + first * a.k8 * CHUNK;
  if (OUT != NORM_16) a.scale = static_cast<float*>(a.scale) + first;
  return a;
}

template <bool BF16, int OUT>
int launch_out(const NormArgs& a, hipStream_t s) {
  auto go = [&]<int T, int C>() -> int {
    constexpr int ROWS = T < 256 ? 256 / T : 1;
    if constexpr (ROWS > 1)  // (at most 2^30 work-items)
      return (int)launch_timed(rms_norm_kernel<BF16, OUT, T, C>, dim3((unsigned)((a.m + ROWS - 1) / ROWS)), dim3(256), 0, s, a);
    else
      return (int)launch_rows(a.m, T, [&](int64_t first, int64_t rows) {
        return launch_timed(rms_norm_kernel<BF16, OUT, T, C>, dim3((unsigned)rows), dim3(T), 0, s, rows_from<OUT>(a, first));
      });
  };
  // The shape that leaves the fewest threads idle, with the more threads the fewer
  // rows there are (us a call in a graph, bf16 with residual, to 16 bits / e4m3 by row / MXFP4):
  //   k = 7168, 1 row: 512 threads of two chunks 3.0 / 3.5 / 3.1, 256 of four 3.4 /
  //   4.3 / 3.7, 64 of fourteen 5.8 / 9.1 / 7.4; 8191 rows: 82 / 74 / 70, 82 / 74 / 70,
  //   91 / 121 / 80
  //   k = 4096, 1 row: 512 of one 2.5 / 3.0 / 2.6, 256 of two 2.8 / 3.3 / 2.9; 8191
  //   rows: 46 / 48 / 40, 47 / 45 / 41
  //   k = 256, 33 rows: 64 of one 2.4 / 2.8 / 2.5, 16 of two 2.6 / 3.2 / 2.9; 100000
  //   rows: 40 / 59 / 40, 39 / 35 / 33
  const int k8 = a.k8;
  if (k8 <= 16) return go.template operator()<16, 1>();
  if (k8 <= 32 && a.m >= 2048) return go.template operator()<16, 2>();
  if (k8 <= 64) return go.template operator()<64, 1>();
  if (k8 <= 128) return go.template operator()<64, 2>();
  if (k8 <= 256) return go.template operator()<256, 1>();
  if (k8 <= 512) return a.m <= 256 ? go.template operator()<512, 1>() : go.template operator()<256, 2>();
  if (k8 <= 1024) return go.template operator()<512, 2>();
  if (k8 <= 2048) return go.template operator()<1024, 2>();
  if (k8 <= 4096) return go.template operator()<1024, 4>();
  if (k8 <= 8192) return go.template operator()<1024, 8>();
  return (int)hipErrorInvalidValue;
}

}  // namespace

int launch_rms_norm(int bf16, int out, const NormArgs& a, void* stream) {
  if (a.m < 1 || a.k8 < 1 || ((out == NORM_FP8_BLOCK || out == NORM_MXFP4) && a.k8 % 16)) return (int)hipErrorInvalidValue;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  switch (out) {
    case NORM_16: return bf16 ? launch_out<true, NORM_16>(a, s) : launch_out<false, NORM_16>(a, s);
    case NORM_FP8: return bf16 ? launch_out<true, NORM_FP8>(a, s) : launch_out<false, NORM_FP8>(a, s);
    case NORM_INT8: return bf16 ? launch_out<true, NORM_INT8>(a, s) : launch_out<false, NORM_INT8>(a, s);
    case NORM_FP8_BLOCK: return bf16 ? launch_out<true, NORM_FP8_BLOCK>(a, s) : launch_out<false, NORM_FP8_BLOCK>(a, s);
    case NORM_MXFP4: return bf16 ? launch_out<true, NORM_MXFP4>(a, s) : launch_out<false, NORM_MXFP4>(a, s);
  }
  return (int)hipErrorInvalidValue;
}

}  // namespace hq
