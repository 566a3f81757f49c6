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
// run 64-bit multiply-adds at the rate of 32-bit ones.
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include "launch.h"
#include "route.h"
#include "route_device.h"

namespace hq {

namespace {

__device__ inline double wave_sum64(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
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
      e[i] = live[i] ? exp((double)v[i] - top) : 0.;
      sum += e[i];
    }
    sum = wave_sum64(sum);
#pragma unroll
    for (int i = 0; i < NPL; ++i) s[i] = (float)(e[i] / sum);
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) s[i] = (float)(1. / (1. + exp(-(double)v[i])));
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
    const float sum = wave_sum(chosen);
    if (sum > 0.f) w = chosen / sum;
  }
  if (lane < p.topk) {
    p.ids[row * p.topk + lane] = id;
    p.w[row * p.topk + lane] = w * p.scale;
  }
}

}  // namespace

int launch_route_experts(const RouteArgs& a, void* stream) {
  if (a.t < 1 || a.E < 1 || a.E > 1024 || a.groups < 1 || a.groups > 64 || a.E % a.groups) return (int)hipErrorInvalidValue;
  const dim3 grid((unsigned)((a.t + 3) / 4)), block(256);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.E <= 64) return (int)launch_timed(route_experts_kernel<1>, grid, block, 0, s, a);
  if (a.E <= 128) return (int)launch_timed(route_experts_kernel<2>, grid, block, 0, s, a);
  if (a.E <= 192) return (int)launch_timed(route_experts_kernel<3>, grid, block, 0, s, a);
  if (a.E <= 256) return (int)launch_timed(route_experts_kernel<4>, grid, block, 0, s, a);
  if (a.E <= 512) return (int)launch_timed(route_experts_kernel<8>, grid, block, 0, s, a);
  return (int)launch_timed(route_experts_kernel<16>, grid, block, 0, s, a);
}

}  // namespace hq
