// Device helpers of the routing kernels: logits and scores as ordered keys, and the
// row of them that a wave chooses from.
#pragma once

#include "block8_device.h"

namespace hq {

// A logit as an unsigned key: larger for larger logits, 0 for -inf and NaN,
// which are never chosen.
__device__ inline uint32_t logit_key(float v) {
  if (!(v > -__builtin_inff())) return 0u;
  const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);  // -0 and 0 are equal
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ inline float key_logit(uint32_t k) {
  if (k == 0u) return -__builtin_inff();
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// e^d of a logit's difference d <= 0 from the largest: 2^(t + r), t the rounded
// product d log2(e) and r what the rounding left, by the hardware's power (1 ulp)
// and one multiply-add.  1.5 ulp whatever d, where 2^t alone is off by |d| 2^-24
// (16383 x 160 bf16 in a graph 7.1 us, 6.8 that way, 7.8 with expf).  Below 2^-126
// it is zero.
__device__ inline float routing_exp(float d) {
  constexpr float hi = 1.44269504f, lo = 1.92596299e-8f;  // log2(e)
  d = fmaxf(d, -200.f);  // zero from here on
  const float t = d * hi, r = fmaf(d, lo, fmaf(d, hi, -t)), p = __builtin_amdgcn_exp2f(t);
  return fmaf(p, r * 0.693147181f, p);
}

// LT: 0 fp32, 1 bf16, 2 fp16
template <int LT>
__device__ inline float load_logit(const void* p, int64_t i) {
  if constexpr (LT == 0) return static_cast<const float*>(p)[i];
  const uint32_t b = static_cast<const uint16_t*>(p)[i];
  return LT == 1 ? bf16_bits_to_float(b) : f16_bits_to_float(b);
}

// Wave-wide maximum and sum, uniform.
__device__ inline uint32_t wave_max(uint32_t v) {
  v = b8_row_max(v);
  const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
  const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
  return max(max(a, b), max(c, d));
}
__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// The row of logits a wave holds: lane l keeps experts l, l + 64, ... and the
// largest of their keys.
template <int NPL>
struct Logits {
  uint32_t key[NPL], head;
  template <int LT>
  __device__ inline void load_as(const void* p, int64_t row, int E, int lane) {
    float v[NPL];  // all in flight at once: a type looked up per load would wait for each in turn
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = load_logit<LT>(p, row * E + min(lane + 64 * i, E - 1));
#pragma unroll
    for (int i = 0; i < NPL; ++i) key[i] = lane + 64 * i < E ? logit_key(v[i]) : 0u;
  }
  __device__ inline void load(const void* p, int64_t row, int E, int lt, int lane) {
    if (lt == 0)
      load_as<0>(p, row, E, lane);
    else if (lt == 1)
      load_as<1>(p, row, E, lane);
    else
      load_as<2>(p, row, E, lane);
    refresh();
  }
  __device__ inline void refresh() {
    head = key[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) head = max(head, key[i]);
  }
  // The best expert left (largest key, then lowest index), struck out; -1 if
  // none is left.  Uniform.
  __device__ inline int take(int lane, uint32_t* best) {
    const uint32_t m = wave_max(head);
    *best = m;
    if (m == 0u) return -1;
    int mine = NPL - 1;  // the lowest of this lane's that has the key
#pragma unroll
    for (int i = NPL - 2; i >= 0; --i) mine = key[i] == m ? i : mine;
    const uint64_t has = __ballot(head == m);
    int l = __builtin_ctzll(has);
    if (NPL > 1 && (has & (has - 1))) {  // in several lanes
      uint64_t b = 0;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (!b) b = __ballot(key[i] == m);
      l = __builtin_ctzll(b);
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) key[i] = lane == l && mine == i ? 0u : key[i];
    refresh();
    return 64 * __builtin_amdgcn_readlane(mine, l) + l;
  }
  __device__ inline float exp_sum(float top) const {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (key[i]) s += routing_exp(key_logit(key[i]) - top);
    return wave_sum(s);
  }
};

}  // namespace hq
