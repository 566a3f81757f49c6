// Routing by scores, with a bias for balance and a choice of groups first.
//
//   s   = sigmoid(l), or softmax(l) over the row, as the nearest fp32 number
//   key = s + bias (fp32); experts of logit -inf or NaN have none
//   the group_topk groups of largest score stay, a group's score being the sum of its
//   group_best largest keys (fp32); of their experts the topk of largest key are
//   chosen; ties go to the lowest index
//   w   = s, over the chosen ones' sum if renormalised, times a factor
//
// The scores are formed in 64 bits and rounded once: a choice must not depend on how
// an exponential was rounded, and scores one last bit apart occur (saturated sigmoids,
// 16-bit logits, a few pairs among 16383 rows of 160 random ones).  The vector units
// run 64-bit multiply-adds at the rate of 32-bit ones.  Start to end of the kernel, one token by
// 256 experts takes 4.4 us, 4096 8.6, 16383 by 160 13.4 (in a graph the library's exp() and
// quotients took 9.0 for 8.2 at 4096).
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include "launch.h"
#include "route.h"
#include "route_device.h"

namespace hq {

namespace {

// e^x to 2^-51, x in [-745, 700]: 2^n e^r, |r| <= ln 2 / 2, by the Taylor sum of degree 12
// (what it leaves out is below 2^-52).  No cases: a third of the instructions of exp().
__device__ inline double exp64(double x) {
  const double n = __builtin_rint(x * 1.4426950408889634);
  double r = fma(n, -0x1.62e42fefa39efp-1, x);  // ln 2 in two parts
  r = fma(n, -0x1.abc9e3b39803fp-56, r);
  double e = 1. / 479001600.;
  constexpr double c[] = {1. / 39916800., 1. / 3628800., 1. / 362880., 1. / 40320., 1. / 5040., 1. / 720.,
                          1. / 120.,      1. / 24.,      1. / 6.,      0.5,         1.,         1.};
#pragma unroll
  for (int i = 0; i < 12; ++i) e = fma(e, r, c[i]);
  return __builtin_amdgcn_ldexp(e, (int)n);
}
// 1 / d to 2^-52, d in [1, 2^1011]
__device__ inline double inverse64(double d) {
  double y = __builtin_amdgcn_rcp(d);
#pragma unroll
  for (int i = 0; i < 2; ++i) y = fma(fma(-d, y, 1.), y, y);
  return y;
}
__device__ inline float sigmoid(float v) { return (float)inverse64(1. + exp64(fmin(fmax(-(double)v, -745.), 700.))); }

// v of the lane that DPP control `C` names, in rows of 16 lanes
template <int C, typename T>
__device__ inline T dpp(T v) {
  if constexpr (sizeof(T) == 8) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, C, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), C, 0xF, 0xF, false);
    return __builtin_bit_cast(T, (uint64_t)hi << 32 | lo);
  } else {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), C, 0xF, 0xF, false));
  }
}
// f over a row of 16 lanes, in all of them: neighbours, pairs, and then halves and the row
// by their mirrors
template <typename T, typename F>
__device__ inline T row_all(T v, F f) {
  v = f(v, dpp<0xB1>(v));
  v = f(v, dpp<0x4E>(v));
  v = f(v, dpp<0x141>(v));
  return f(v, dpp<0x140>(v));
}
template <typename T>
__device__ inline T row_sum(T v) {
  return row_all(v, [](T a, T b) { return a + b; });
}
// The sum over a wave: lanes l, l + 16, l + 32, l + 48 first.  Both kernels add in this order,
// so that a token's result does not depend on how many there are.
template <typename T>
__device__ inline T wave_sum_quarters(T v) {
  v += __shfl_xor(v, 16, 64);
  return row_sum(v + __shfl_xor(v, 32, 64));
}

// What a wave's lanes wrote to LDS is read by others of the same wave: no barrier,
// but nothing may move across.
__device__ inline void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// One wave per token; lane l holds experts l, l + 64, ...
template <int NPL>
__global__ void __launch_bounds__(256) route_experts_kernel(RouteArgs p) {
  __shared__ uint32_t keys[4][64 * NPL];  // of all experts, for the groups
  __shared__ float scores[4][64 * NPL];
  __shared__ uint32_t group_keys[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * 4 + wave;
  if (row >= p.t) return;
  const int E = p.E;

  float v[NPL], b[NPL];
  auto load = [&](auto lt) {  // all in flight at once
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = load_logit<decltype(lt)::value>(p.logits, row * E + min(lane + 64 * i, E - 1));
  };
  if (p.logit_type == 0) load(std::integral_constant<int, 0>{});
  else if (p.logit_type == 1) load(std::integral_constant<int, 1>{});
  else load(std::integral_constant<int, 2>{});
#pragma unroll
  for (int i = 0; i < NPL; ++i) b[i] = p.bias ? p.bias[min(lane + 64 * i, E - 1)] : 0.f;

  float s[NPL];
  bool live[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) live[i] = lane + 64 * i < E && v[i] > -__builtin_inff();
  if (p.softmax) {
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < NPL; ++i) most = max(most, live[i] ? logit_key(v[i]) : 0u);
    const double top = (double)key_logit(wave_max(most));
    double e[NPL], sum = 0.;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      e[i] = live[i] ? exp64(fmax((double)v[i] - top, -745.)) : 0.;
      sum += e[i];
    }
    const double per = inverse64(wave_sum_quarters(sum));  // (without a live expert of no use)
#pragma unroll
    for (int i = 0; i < NPL; ++i) s[i] = (float)(e[i] * per);
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) s[i] = sigmoid(v[i]);
  }
  Logits<NPL> x;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    x.key[i] = live[i] ? logit_key(s[i] + b[i]) : 0u;
    scores[wave][lane + 64 * i] = s[i];
  }

  if (p.group_topk < p.groups) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) keys[wave][lane + 64 * i] = x.key[i];
    wave_lds_fence();
    // per lanes a group, as many as a power of two allows
    const int size = E / p.groups;
    const int per = 1 << (31 - __builtin_clz(64 / p.groups));
    const int g = lane / per;
    uint32_t first = 0u, second = 0u;
    if (g < p.groups)
      for (int c = lane % per; c < size; c += per) {
        const uint32_t k = keys[wave][g * size + c];
        second = max(second, min(first, k));
        first = max(first, k);
      }
    for (int d = 1; d < per; d <<= 1) {
      const uint32_t f = (uint32_t)__shfl_xor((int)first, d, 64), o = (uint32_t)__shfl_xor((int)second, d, 64);
      second = max(max(second, o), min(first, f));
      first = max(first, f);
    }
    uint32_t mine = first;  // an expert's key orders as the key of its score
    if (p.group_best == 2 && second) mine = logit_key(key_logit(first) + key_logit(second));
    if (g < p.groups && lane % per == 0) group_keys[wave][g] = mine;
    wave_lds_fence();
    // lane u's group stays if fewer than group_topk come before it
    const uint32_t own = group_keys[wave][min(lane, p.groups - 1)];
    int before = 0;
    for (int u = 0; u < p.groups; ++u) {
      const uint32_t k = group_keys[wave][u];
      before += k > own || (k == own && u < lane);
    }
    const uint64_t stays = __ballot(lane < p.groups && before < p.group_topk);
    const uint32_t magic = (1u << 21) / size + 1;  // e / size = e magic >> 21 for e < 1024, size <= 512
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = min(lane + 64 * i, E - 1);
      if (!((stays >> (((uint32_t)e * magic) >> 21)) & 1)) x.key[i] = 0u;
    }
  }
  wave_lds_fence();

  // lane j keeps choice j (topk <= 64)
  x.refresh();
  int id = -1;
  for (int j = 0; j < p.topk; ++j) {
    uint32_t k;
    const int e = x.take(lane, &k);
    if (e < 0) break;
    if (lane == j) id = e;
  }
  const float chosen = id >= 0 ? scores[wave][id] : 0.f;
  float w = chosen;
  if (p.renorm) {
    const float sum = wave_sum_quarters(chosen);
    if (sum > 0.f) w = chosen / sum;
  }
  if (lane < p.topk) {
    p.ids[row * p.topk + lane] = id;
    p.w[row * p.topk + lane] = w * p.scale;
  }
}

// Many tokens: four to a wave, 16 lanes each; lane l of them holds experts l, l + 16, ...
// The choices, which walk the row topk times, then cost a wave a quarter as many steps.  Bound
// by issuing: 16383 x 160 reads and writes 6 MB, but a wave, four tokens, issues 1450 vector and
// 430 scalar instructions, and the vector units are busy for 5800 of the kernel's 8000 periods
// of four cycles.  The twelve exponentials a lane are 480 of them, half in 64 bits, the six
// choices 444.
template <int NPL>
__global__ void __launch_bounds__(256) route_quarters_kernel(RouteArgs p) {
  __shared__ uint32_t keys[16][16 * NPL];
  __shared__ float scores[16][16 * NPL];
  const int lane = threadIdx.x & 63, l = threadIdx.x & 15, at = threadIdx.x >> 4;
  const int64_t row = (int64_t)blockIdx.x * 16 + at;
  const int64_t from = row < p.t ? row : p.t - 1;  // (rows past the end write nothing)
  const int E = p.E;

  float v[NPL];
  auto load = [&](auto lt) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = load_logit<decltype(lt)::value>(p.logits, from * E + min(l + 16 * i, E - 1));
  };
  if (p.logit_type == 0) load(std::integral_constant<int, 0>{});
  else if (p.logit_type == 1) load(std::integral_constant<int, 1>{});
  else load(std::integral_constant<int, 2>{});

  float s[NPL];
  uint32_t key[NPL];
  auto live = [&](int i) { return l + 16 * i < E && v[i] > -__builtin_inff(); };
  if (p.softmax) {
    float most = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < NPL; ++i) most = fmaxf(most, live(i) ? v[i] : -__builtin_inff());
    const double top = (double)row_all(most, [](float a, float b) { return fmaxf(a, b); });
    double e[NPL], sum[4] = {};
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      e[i] = live(i) ? exp64(fmax((double)v[i] - top, -745.)) : 0.;
      sum[i & 3] += e[i];
    }
    const double per = inverse64(row_sum((sum[0] + sum[1]) + (sum[2] + sum[3])));
#pragma unroll
    for (int i = 0; i < NPL; ++i) s[i] = (float)(e[i] * per);
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) s[i] = sigmoid(v[i]);
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    key[i] = live(i) ? logit_key(s[i] + (p.bias ? p.bias[min(l + 16 * i, E - 1)] : 0.f)) : 0u;
    scores[at][l + 16 * i] = s[i];
  }

  if (p.group_topk < p.groups) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) keys[at][l + 16 * i] = key[i];
    wave_lds_fence();
    const int size = E / p.groups;  // a lane a group
    uint32_t first = 0u, second = 0u;
    if (l < p.groups)
      for (int c = 0; c < size; ++c) {
        const uint32_t k = keys[at][l * size + c];
        second = max(second, min(first, k));
        first = max(first, k);
      }
    uint32_t own = first;
    if (p.group_best == 2 && second) own = logit_key(key_logit(first) + key_logit(second));
    int before = 0;
    for (int u = 0; u < p.groups; ++u) {
      const uint32_t k = (uint32_t)__shfl((int)own, (lane & 48) + u, 64);
      before += k > own || (k == own && u < l);
    }
    const uint32_t stays = (uint32_t)(__ballot(l < p.groups && before < p.group_topk) >> (lane & 48)) & 0xFFFFu;
    const uint32_t magic = (1u << 21) / size + 1;  // e / size = e magic >> 21 for e < 1024, size <= 512
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = min(l + 16 * i, E - 1);
      if (!((stays >> (((uint32_t)e * magic) >> 21)) & 1)) key[i] = 0u;
    }
  }
  wave_lds_fence();

  int id = -1;  // lane j keeps choice j
  for (int j = 0; j < p.topk; ++j) {
    uint32_t head = key[0];
    int mine = 0;
#pragma unroll
    for (int i = 1; i < NPL; ++i) {
      mine = key[i] > head ? i : mine;
      head = max(head, key[i]);
    }
    const uint32_t best = row_all(head, [](uint32_t a, uint32_t b) { return max(a, b); });
    const uint32_t e = row_all(head == best ? (uint32_t)(mine * 16 + l) : 0xFFFFu, [](uint32_t a, uint32_t b) { return min(a, b); });
    if (l == j && best) id = (int)e;
    const int out = (e & 15) == (uint32_t)l ? (int)(e >> 4) : -1;
#pragma unroll
    for (int i = 0; i < NPL; ++i) key[i] = i == out ? 0u : key[i];
  }
  const float chosen = id >= 0 ? scores[at][id] : 0.f;
  float w = chosen;
  if (p.renorm) {
    const float sum = row_sum(chosen);
    if (sum > 0.f) w = chosen / sum;
  }
  if (l < p.topk && row < p.t) {
    p.ids[row * p.topk + l] = id;
    p.w[row * p.topk + l] = w * p.scale;
  }
}

}  // namespace

int launch_route_experts(const RouteArgs& a, void* stream) {
  if (a.t < 1 || a.E < 1 || a.E > 1024 || a.groups < 1 || a.groups > 64 || a.E % a.groups) return (int)hipErrorInvalidValue;
  const dim3 grid((unsigned)((a.t + 3) / 4)), block(256);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  // us in a graph with a wave / a quarter of one per token: 160 experts, top 6 of 3 of 8 groups: 4096 tokens
  // 7.3 / 7.5, 8192 11.1 / 8.8, 16383 18.7 / 12.8; 256, top 8 of 4 of 8: 8192 13.0 / 14.0, 16383
  // 22.2 / 18.9; 128, top 8: 4096 5.6 / 5.7, 8192 8.2 / 6.5; 64, top 6: 2048 3.5 / 3.9, 4096 4.2 / 3.9
  if (a.t >= 4096 && a.t >= 40 * a.E && a.topk <= 16 && a.groups <= 16 && a.E <= 256) {
    const dim3 quarters((unsigned)((a.t + 15) / 16));
    if (a.E <= 64) return (int)launch_timed(route_quarters_kernel<4>, quarters, block, 0, s, a);
    if (a.E <= 128) return (int)launch_timed(route_quarters_kernel<8>, quarters, block, 0, s, a);
    if (a.E <= 192) return (int)launch_timed(route_quarters_kernel<12>, quarters, block, 0, s, a);
    return (int)launch_timed(route_quarters_kernel<16>, quarters, block, 0, s, a);
  }
  if (a.E <= 64) return (int)launch_timed(route_experts_kernel<1>, grid, block, 0, s, a);
  if (a.E <= 128) return (int)launch_timed(route_experts_kernel<2>, grid, block, 0, s, a);
  if (a.E <= 192) return (int)launch_timed(route_experts_kernel<3>, grid, block, 0, s, a);
  if (a.E <= 256) return (int)launch_timed(route_experts_kernel<4>, grid, block, 0, s, a);
  if (a.E <= 512) return (int)launch_timed(route_experts_kernel<8>, grid, block, 0, s, a);
  return (int)launch_timed(route_experts_kernel<16>, grid, block, 0, s, a);
}

}  // namespace hq
