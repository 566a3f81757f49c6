// Internal interface of the root-mean-square norm (norm.hip).
#pragma once

#include "hq_internal.h"

namespace hq {

enum NormOut : int { NORM_16 = 0, NORM_FP8 = 1, NORM_INT8 = 2, NORM_FP8_BLOCK = 3, NORM_MXFP4 = 4 };

struct NormArgs {
  const void* x;         // [m][k] 16-bit, rows x_stride apart
  const void* residual;  // the same type, or null
  const void* weight;    // [k], x's type or fp32
  void* h;               // x + residual, with a residual
  void* out;             // 16-bit [m][k], 8-bit [m][k], or MXFP4 [m][k/2]
  void* scale;           // fp32 [m] or [k/128][m], or E8M0 words [k/128][m]
  int64_t x_stride, r_stride, h_stride;  // in 16-byte chunks
  int m, k8;             // rows, chunks of 8 values
  float eps;
  int w_f32;
};

int launch_rms_norm(int bf16, int out, const NormArgs& a, void* stream);

}  // namespace hq
