// Routing, and an experts' layer of fp8 weights with 128-block scales for a
// few tokens in two kernels, from the router's logits (or given ids) on.
//
//   route     p = softmax(l); the topk experts of largest logit, ties to the
//             lowest index; weight p, or p over the chosen ones' sum
//   gate_up   h = quant(x) . W1[e]^T, act = SiLU(h[:I]) * h[I:]   (fp32 rows)
//   down      y[t] = sum_j w[t, j] quant(act[t, j]) . W2[e]^T
//
// Both GEMMs are bound by reading the chosen experts' weights, which every
// workgroup streams straight to registers; tokens that picked the same expert
// share one read (they are the columns of the matrix instruction).  One token's
// expert is found inside the kernel: a workgroup row per slot takes the j-th
// best logit.  More tokens are routed by the routing kernel first: counting the
// slots of an expert from the logits in every workgroup took 9 us of 8 tokens'
// 76, the launch takes 4.
//
// 256 experts, top 8, H = 7168, I = 256, in a graph over four sets of inputs, and
// the bytes of the experts that those hit over a streaming read's 6 TB/s: 1 token 18.3
// us (7.3), 2 29.2 (14.5), 4 42.9 (27), 8 64 (47), 13 90 (67), 16 97 (76); 24 tokens
// 150 (96), where the aligned path takes 117 (16 tokens 106).  With fewer experts
// the two paths cross earlier: 64 experts, top 8, H = 2048, I = 768 at 4 tokens (8
// tokens 68 us against 51), 8 and 16 experts, top 2, H = 4096 between 10 and 16.
// More than one token's weights are read past the caches (4 tokens 42 us against
// 45, 13 88.6 against 93); one token's may stay there (17.3 against 18.4).
// About 9 us are the two kernels' launches and their chains of dependent loads
// (ids, weights); the rest runs at 4.5 .. 5 TB/s.
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "block8.h"
#include "block8_device.h"
#include "launch.h"

namespace hq {

namespace {

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

// One wave per token: the chain of a choice is short (a maximum over 64 lanes),
// 3.6 us for one token of 256 experts.
template <int NPL>
__global__ void __launch_bounds__(256) route_kernel(const void* __restrict__ logits, int lt, int t, int E, int topk,
                                                    int renorm, int32_t* __restrict__ ids, float* __restrict__ w) {
  const int row = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (row >= t) return;
  Logits<NPL> x;
  x.load(logits, row, E, lt, lane);
  const float top = key_logit(wave_max(x.head));
  float sum = renorm ? 0.f : x.exp_sum(top);
  // lane j keeps choice j (topk <= 64)
  int my_id = -1;
  float my_e = 0.f;
  for (int j = 0; j < topk; ++j) {
    uint32_t k;
    const int e = x.take(lane, &k);
    if (e < 0) break;
    const float v = routing_exp(key_logit(k) - top);
    if (renorm) sum += v;
    if (lane == j) {
      my_id = e;
      my_e = v;
    }
  }
  if (lane < topk) {
    ids[(int64_t)row * topk + lane] = my_id;
    w[(int64_t)row * topk + lane] = my_id < 0 ? 0.f : my_e / sum;
  }
}

__device__ inline uint32_t row_min(uint32_t v) { return ~b8_row_max(~v); }
__device__ inline float row_sum(float v) {
  auto ror = [&](auto c) {
    constexpr int ctrl = decltype(c)::value;
    v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), ctrl, 0xF, 0xF, false));
  };
  ror(std::integral_constant<int, 0x128>{});
  ror(std::integral_constant<int, 0x124>{});
  ror(std::integral_constant<int, 0x122>{});
  ror(std::integral_constant<int, 0x121>{});
  return v;
}

// Sixteen lanes per token, for many tokens: a choice costs the wave one maximum
// over 16 lanes for four tokens.  Lane l keeps experts l, l + 16, ...  16-bit
// logits carry their expert in the key's low half (the lower the larger), which
// makes the keys unique and a choice one comparison per key.  Bound by
// instructions: 16383 x 160 bf16 top 6, 7.1 us in a graph (a wave per token about
// twice that), 6 MB.
template <int LT, int NPL>
__global__ void __launch_bounds__(256) route_rows_kernel(const void* __restrict__ logits, int t, int E, int topk, int renorm,
                                                         int32_t* __restrict__ ids, float* __restrict__ w) {
  const int row = blockIdx.x * 16 + (threadIdx.x >> 4), lane = threadIdx.x & 15;
  const int r = min(row, t - 1);
  // 16-bit logits as float keys have their value in the high half (bf16) or
  // are kept as the order of their own bits (fp16)
  auto key16 = [](uint32_t b) -> uint32_t {  // 0 for -inf and NaN
    constexpr uint32_t inf = LT == 1 ? 0x7F80u : 0x7C00u;
    const uint32_t mag = b & 0x7FFFu;
    if (mag > inf || b == (0x8000u | inf)) return 0u;
    if (mag == 0u) b = 0u;  // -0 and 0 are equal
    return (b & 0x8000u) ? (~b & 0xFFFFu) : (b | 0x8000u);
  };
  auto value = [](uint32_t k) -> float {
    if constexpr (LT == 0) return key_logit(k);
    if ((k >> 16) == 0u) return -__builtin_inff();
    const uint32_t h = k >> 16, b = (h & 0x8000u) ? (h & 0x7FFFu) : (~h & 0xFFFFu);
    return LT == 1 ? bf16_bits_to_float(b) : f16_bits_to_float(b);
  };
  uint32_t key[NPL];
  {
    uint32_t raw[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int64_t at = (int64_t)r * E + min(lane + 16 * i, E - 1);
      raw[i] = LT == 0 ? static_cast<const uint32_t*>(logits)[at] : static_cast<const uint16_t*>(logits)[at];
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 16 * i;
      if constexpr (LT == 0)
        key[i] = e < E ? logit_key(__uint_as_float(raw[i])) : 0u;
      else {
        const uint32_t k = key16(raw[i]);
        key[i] = e < E && k ? (k << 16) | (0xFFFFu - e) : 0u;
      }
    }
  }
  auto largest = [&] {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) m = max(m, key[i]);
    return m;
  };
  uint32_t head = largest();
  uint32_t best = b8_row_max(head);
  const float top = value(best);
  float sum = 0.f;
  if (!renorm) {
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (key[i]) sum += routing_exp(value(key[i]) - top);
    sum = row_sum(sum);
  }
  int my_id = -1;
  float my_e = 0.f;
  for (int j = 0; j < topk; ++j) {
    const uint32_t m = best;  // zero once a token's row is used up
    int e;
    if constexpr (LT == 0) {
      int mine = NPL - 1;  // the lowest of this lane's that has the key
#pragma unroll
      for (int i = NPL - 2; i >= 0; --i) mine = key[i] == m ? i : mine;
      e = (int)row_min(head == m ? (uint32_t)(16 * mine + lane) : 0xFFFFu);
      const int strike = (e & 15) == lane ? e >> 4 : -1;
#pragma unroll
      for (int i = 0; i < NPL; ++i) key[i] = i == strike ? 0u : key[i];
    } else {
      e = (int)(0xFFFFu - (m & 0xFFFFu));
#pragma unroll
      for (int i = 0; i < NPL; ++i) key[i] = key[i] == m ? 0u : key[i];
    }
    const float v = m ? routing_exp(value(m) - top) : 0.f;
    if (renorm) sum += v;
    if (lane == j && m) {
      my_id = e;
      my_e = v;
    }
    head = largest();
    best = b8_row_max(head);
  }
  if (lane < topk && row < t) {
    ids[(int64_t)row * topk + lane] = my_id;
    w[(int64_t)row * topk + lane] = my_id < 0 ? 0.f : my_e / sum;
  }
}

// ---------------------------------------------------------------------------
// gate_up.  A workgroup row per slot; the first of the slots that share an
// expert does the work for all of them.  Two shapes:
//   narrow  16 outputs a workgroup, its waves share K (their sums meet in
//           LDS); the fp32 rows are quantised by the down kernel.  For up to 8
//           tokens, whose few experts would leave most CUs idle otherwise: one
//           token 12 us with 8 waves and all of a wave's loads in flight at
//           once, more with 4.
//   wide    128 outputs a workgroup, 16 a wave over all of K: no sums to join,
//           and the workgroup holds a whole scale block, so that it writes
//           codes and scales.  13 tokens 57 us, 4.8 TB/s (272 MB).
// The products go through fp16 (b8_mfma_exact): their sums are quantised again.
// One more row of workgroups writes the routing where there are logits, and
// otherwise the units that the down kernel walks.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;  // of a down workgroup
constexpr int kFewLds = 128 * 1024;  // most dynamic LDS of a workgroup

// The routing of slot z, for the down kernel and the caller (one wave).
template <int NPL>
__device__ inline void few_write_routing(const B8FewArgs& p, int z, int lane) {
  Logits<NPL> r;
  r.load(p.logits, 0, p.E, p.logit_type, lane);
  const float top = key_logit(wave_max(r.head));
  float sum = p.renorm ? 0.f : r.exp_sum(top);
  int e = -1;
  float mine = 0.f;
  for (int j = 0; j < p.topk; ++j) {
    uint32_t k;
    const int id = r.take(lane, &k);
    if (id < 0) break;
    const float v = routing_exp(key_logit(k) - top);
    if (p.renorm) sum += v;
    if (j == z) {
      e = id;
      mine = v;
      if (!p.renorm) break;
    }
  }
  if (lane == 0) {
    p.topk_ids[z] = e;
    p.topk_w[z] = e < 0 ? 0.f : mine / sum;
  }
}

// The expert of slot z, -1 for none.  Uniform over the workgroup.
template <int NPL>
__device__ inline int few_expert(const B8FewArgs& p, int z, int lane) {
  int e = -1;
  if (p.logits) {
    Logits<NPL> x;
    x.load(p.logits, 0, p.E, p.logit_type, lane);
    for (int j = z; j >= 0; --j) {
      uint32_t k;
      e = x.take(lane, &k);
      if (e < 0) break;
    }
  } else {
    e = p.topk_ids[z];
    if (e < 0 || e >= p.E) e = -1;
  }
  return __builtin_amdgcn_readfirstlane(e);
}

// The ids a wave's lanes scan for an expert's slots, the first kScan of them in
// flight before the expert is known.
constexpr int kScan = 4;
__device__ inline void few_ids(const B8FewArgs& p, int (&ids)[kScan], int lane) {
#pragma unroll
  for (int i = 0; i < kScan; ++i) ids[i] = p.topk_ids[min(64 * i + lane, p.t * p.topk - 1)];
}

// The slots that hold expert e, in order, into picks; returns how many.  Ends
// with a barrier.
__device__ inline int few_slots(const B8FewArgs& p, int e, const int (&ids)[kScan], int* picks, int* npicks, int lane, int wave) {
  if (wave == 0) {
    int n = 0;
    auto scan = [&](int b, int id) {
      const bool hit = b + lane < p.t * p.topk && id == e;
      const uint64_t has = __ballot(hit);
      if (hit) picks[n + __popcll(has & ((1ull << lane) - 1))] = b + lane;
      n += __popcll(has);
    };
#pragma unroll
    for (int i = 0; i < kScan; ++i) scan(64 * i, ids[i]);
    for (int b = 64 * kScan; b < p.t * p.topk; b += 64) scan(b, p.topk_ids[min(b + lane, p.t * p.topk - 1)]);
    if (lane == 0) *npicks = n;
  }
  __syncthreads();
  return *npicks;
}

// The units of a tile of 16 tokens, for the down kernel: the distinct experts of
// its slots.  A token may hold an expert more than once (given ids): each
// occurrence is a unit of its own, so that a unit has at most one slot per
// token.  One workgroup; key: 2 kMax + 4 ints of LDS.  Found here, beside the
// stream, as in every down workgroup it cost up to a third of its time (13
// tokens: 36 us against 31).
template <int NW>
__device__ inline void few_units(const B8FewArgs& p, int tile, int* key, int tid) {
  constexpr int kMax = 16 * kB8FewMaxTopk;  // slots of a tile
  static_assert(64 * NW >= kMax);
  int* unit_of = key + kMax;  // index of a slot's unit, at the unit's first slot
  int* wcount = unit_of + kMax;
  const int lane = tid & 63, wave = tid >> 6;
  const int topk = p.topk, t0 = tile * 16, ns = min(16, p.t - t0) * topk;
  int32_t* out = p.units + (int64_t)tile * kB8FewUnitInts;
  for (int i = tid; i < ns * 8; i += 64 * NW) out[16 + kMax + i] = -1;
  int id = -1;
  if (tid < ns) {
    id = p.topk_ids[t0 * topk + tid];
    if (id < 0 || id >= p.E) id = -1;
  }
  if (tid < kMax) key[tid] = id;
  __syncthreads();
  const int tok = tid / topk, from = tok * topk;
  const bool have = tid < ns && id >= 0;
  int occ = 0;
  for (int j = 0; j < topk; ++j) occ += have && from + j < tid && key[min(from + j, kMax - 1)] == id;
  __syncthreads();
  const int k = id | (occ << 16);  // E is below 2^16
  if (have) key[tid] = k;
  __syncthreads();
  int first = kMax;
  for (int s = 0; s < ns; s += 4) {  // four keys a read, no read waits for another's result
    const int4 v = *reinterpret_cast<const int4*>(key + s);
    const int c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) first = min(first, c[q] == k ? s + q : kMax);
  }
  const bool lead = have && first == tid;
  const uint64_t leads = __ballot(lead);
  if (lane == 0 && wave < 4) wcount[wave] = __popcll(leads);
  __syncthreads();
  if (tid == 0) out[0] = wcount[0] + wcount[1] + wcount[2] + wcount[3];
  if (lead) {
    int at = __popcll(leads & ((1ull << lane) - 1));
    for (int w = 0; w < wave; ++w) at += wcount[w];
    unit_of[tid] = at;
    out[16 + at] = id;
  }
  __syncthreads();
  if (have) reinterpret_cast<int16_t*>(out + 16 + kMax)[unit_of[first] * 16 + tok] = (int16_t)tid;
  __syncthreads();  // before the next tile
}

__device__ inline __amdgpu_buffer_rsrc_t few_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// One block of a row of x (16 lanes, 8 values each) -> codes and scale in LDS.
template <bool BF16>
__device__ inline void few_quantise(u4_t raw, uint8_t* codes, float* scale, int c16) {
  float v[8];
  b8_unpack<BF16>(raw, v);
  uint32_t top = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, b8_mag(v[j]));
  const float s = b8_scale(b8_row_max(top));
  const B8Div d(s);
  *reinterpret_cast<uint2*>(codes + c16 * 8) =
      uint2{b8_codes(v[0], v[1], v[2], v[3], d), b8_codes(v[4], v[5], v[6], v[7], d)};
  if (c16 == 0) *scale = s;
}

template <int NPL, bool BF16, bool WIDE, int NW, int ST>
__global__ void __launch_bounds__(64 * NW) few_gate_up(B8FewArgs p) {
#if defined(__HIP_DEVICE_COMPILE__)
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // rows: codes [R][pitch], scales [R][G]
  __shared__ f4_t red[WIDE ? 1 : NW][2][64];
  __shared__ uint32_t tops[NW][16];
  __shared__ __attribute__((aligned(16))) int picks[kB8FewMaxSlots];
  __shared__ int npicks;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kq = lane >> 4;
  const int z = blockIdx.y, K = p.H, G = K / 128;
  const int nbi = p.I / 16;
  if (z == p.t * p.topk) {  // the last row
    if (p.logits) {
      if (wave == 0)
        for (int j = blockIdx.x; j < p.topk; j += gridDim.x) few_write_routing<NPL>(p, j, lane);
    } else {
      for (int tile = blockIdx.x; tile * 16 < p.t; tile += gridDim.x) few_units<NW>(p, tile, picks, tid);
    }
    return;
  }
  // the slot's own row of x is the first of the rows below: its loads (up to
  // 64 blocks) start here, before the routing
  constexpr int XP = 16 / NW;
  u4_t xr[XP];
#pragma unroll
  for (int u = 0; u < XP; ++u) {
    const int g = min((tid >> 4) + 4 * NW * u, G - 1);
    xr[u] = static_cast<const u4_t*>(p.x)[(int64_t)(z / p.topk) * (K / 8) + g * 16 + c16];
  }
  int ids[kScan] = {};
  if (!p.logits && wave == 0) few_ids(p, ids, lane);
  const int e = few_expert<NPL>(p, z, lane);
  if (e < 0) return;

  // ---- weight stream: this wave's gate and up fragments of step i ----------------
  const int nb0 = WIDE ? blockIdx.x * 8 + wave : blockIdx.x;
  const int gs = WIDE ? 0 : wave, gd = WIDE ? 1 : NW;  // groups gs, gs + gd, ...
  const auto rw = few_rsrc(p.w1 + (int64_t)e * p.w1_expert, p.w1_expert);
  const auto rws = few_rsrc(p.s1 + (int64_t)e * p.s1_expert, p.s1_expert * 4);
  constexpr int AUX = WIDE || NW == 4 ? kReadOnce : 0;  // more than one token
  u4_t wr[ST][2][2];
  uint32_t sw[ST][2];
  auto issue = [&](int slot, int g) {
    const int past = g < G ? 0 : (int)0x80000000u;  // steps past the end read nothing and hold zeros
    g = min(g, G - 1);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int nb = u * nbi + nb0;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        wr[slot][u][h] = __builtin_bit_cast(
            u4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, (lane * 16 + 1024 * h) | past, (nb * G + g) * 2048, AUX));
      sw[slot][u] = __builtin_amdgcn_raw_buffer_load_b32(rws, past, ((nb / 8) * G + g) * 4, 0);
    }
  };
#pragma unroll
  for (int s = 0; s < ST; ++s) {
    issue(s, gs + s * gd);
    __builtin_amdgcn_sched_barrier(0);  // step by step, as the waits of the loop below count them
  }

  int n = 1;
  if (p.logits) {  // one token, whose experts differ
    if (tid == 0) picks[0] = z;
  } else {
    n = few_slots(p, e, ids, picks, &npicks, lane, wave);
    if (picks[0] != z) return;
  }

  const int pitch = K + 16, R = p.rows;
  float* sa = reinterpret_cast<float*>(lds + R * pitch);
  for (int c0 = 0; c0 < n; c0 += R) {
    const int nr = min(n - c0, R);
    if (c0) {
      __syncthreads();  // the rows and sums of the chunk before are read
    } else {
#pragma unroll
      for (int u = 0; u < XP; ++u) {
        const int g = (tid >> 4) + 4 * NW * u;
        if (g < G) few_quantise<BF16>(xr[u], lds + g * 128, sa + g, c16);
      }
    }
    // the rest of the rows' blocks: row i / G, block i % G
    const int done = c0 ? 0 : min(G, 4 * NW * XP);
#pragma unroll 1
    for (int i = done + (tid >> 4); i < nr * G; i += 4 * NW) {
      const int r = i / G, g = i - r * G;
      const int64_t row = (!c0 && !r) ? z / p.topk : picks[c0 + r] / p.topk;
      few_quantise<BF16>(static_cast<const u4_t*>(p.x)[row * (K / 8) + g * 16 + c16], lds + r * pitch + g * 128,
                         sa + r * G + g, c16);
    }
    __syncthreads();
    const int rl = min(c16, nr - 1);
    const uint8_t* ar = lds + rl * pitch + kq * 16;
    f4_t acc[2] = {f4_t{0.f, 0.f, 0.f, 0.f}, f4_t{0.f, 0.f, 0.f, 0.f}};
#pragma unroll 1
    for (int g = gs; g < G; g += ST * gd) {
#pragma unroll
      for (int s = 0; s < ST; ++s) {
        const int gg = min(g + s * gd, G - 1);
        const auto av = b8_halves(*reinterpret_cast<const u4_t*>(ar + gg * 128), *reinterpret_cast<const u4_t*>(ar + gg * 128 + 64));
        const float f = sa[rl * G + gg];  // past the end the weights and their scales are zero
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const f4_t P = b8_mfma_exact(b8_halves(wr[s][u][0], wr[s][u][1]), av);
          const float m = f * __uint_as_float(sw[s][u]);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[u][q] = fmaf(m, P[q], acc[u][q]);
        }
        // the ring goes on with the next groups, after the last ones with the
        // first ones again if there are more rows
        issue(s, g + ST * gd < G ? g + (s + ST) * gd : (c0 + R < n ? gs + s * gd : G));
        __builtin_amdgcn_sched_barrier(0);  // one step's operands at a time: the ring fills the registers
      }
    }
    if constexpr (WIDE) {
      uint32_t top = 0u;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        acc[0][q] = b8_silu_mul(acc[0][q], acc[1][q]);
        top = max(top, b8_mag(acc[0][q]));
      }
      top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
      top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
      if (kq == 0) tops[wave][c16] = top;
      __syncthreads();
      top = 0u;
#pragma unroll
      for (int w = 0; w < NW; ++w) top = max(top, tops[w][c16]);
      const float s = b8_scale(top);
      const B8Div d(s);
      if (c16 < nr) {
        const int64_t slot = picks[c0 + c16];
        *reinterpret_cast<uint32_t*>(p.act_codes + slot * p.I + nb0 * 16 + 4 * kq) =
            b8_codes(acc[0][0], acc[0][1], acc[0][2], acc[0][3], d);
        if (wave == 0 && kq == 0) p.act[slot * (p.I / 128) + blockIdx.x] = s;
      }
    } else {
      red[wave][0][lane] = acc[0];
      red[wave][1][lane] = acc[1];
      __syncthreads();
      if (tid < 64 && c16 < nr) {
        f4_t h[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          h[u] = red[0][u][lane];
#pragma unroll
          for (int w = 1; w < NW; ++w)
#pragma unroll
            for (int q = 0; q < 4; ++q) h[u][q] += red[w][u][lane][q];
        }
        f4_t a;
#pragma unroll
        for (int q = 0; q < 4; ++q) a[q] = b8_silu_mul(h[0][q], h[1][q]);
        *reinterpret_cast<f4_t*>(p.act + (int64_t)picks[c0 + c16] * p.I + nb0 * 16 + 4 * kq) = a;
      }
    }
  }
#endif
}

// ---------------------------------------------------------------------------
// down + combine: grid (16-column blocks, tiles of 16 tokens).  The tile's
// activation rows lie quantised in LDS (as many 128-k groups at a time as
// fit); the waves take the (expert, group) steps in turn.  One token 6.0 .. 6.5 us
// (14.7 MB), 13 tokens 30 us (136 MB).
// ---------------------------------------------------------------------------
template <bool WIDE, bool ONE, int ST>
__global__ void __launch_bounds__(64 * kFewWaves) __attribute__((amdgpu_waves_per_eu(4))) few_down(B8FewArgs p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kMax = 16 * kB8FewMaxTopk;  // slots of a tile
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // codes [ns][pitch], scales [ns][gmax]
  __shared__ f4_t red[kFewWaves][64];
  __shared__ int slots_of[ONE ? 1 : kMax * 8];  // [unit][token of the tile]: its slot as 16 bits, -1 none
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kq = lane >> 4;
  const int topk = p.topk, t0 = blockIdx.y * 16, nt = min(16, p.t - t0), ns = nt * topk;
  const int G = p.I / 128, N = p.H, nb = blockIdx.x;

  // A lane keeps the experts of four units (-1: none), so that a step finds its
  // own without a trip to LDS.  One token's slots are its units, those without
  // an expert too: their steps read nothing.
  int nu, ue[4] = {-1, -1, -1, -1};
  if constexpr (ONE) {
    nu = ns;
    ue[0] = lane < ns ? p.topk_ids[lane] : -1;
    if (ue[0] >= p.E) ue[0] = -1;
  } else {
    const int32_t* un = p.units + (int64_t)blockIdx.y * kB8FewUnitInts;
    nu = __builtin_amdgcn_readfirstlane(un[0]);
#pragma unroll
    for (int i = 0; i < 4; ++i) ue[i] = un[16 + lane + 64 * i];  // (past nu whatever lies there, not used)
    for (int i = tid; i < nu * 8; i += 64 * kFewWaves) slots_of[i] = un[16 + kMax + i];
  }

  const int gmax = p.down_groups, pitch = gmax * 128 + 16;
  float* sc = reinterpret_cast<float*>(lds + ns * pitch);  // [ns][gmax]
  constexpr int AUX = ONE ? 0 : kReadOnce;
  u4_t wr[ST][2];
  uint32_t sw[ST];
  f4_t acc = f4_t{0.f, 0.f, 0.f, 0.f};
  for (int gc0 = 0; gc0 < G && nu; gc0 += gmax) {
    const int gc = min(gmax, G - gc0), steps = nu * gc;
    // step i is (unit i / gc, group i % gc), kept as a pair that the waves'
    // stride moves on
    const int du = kFewWaves / gc, dg = kFewWaves - du * gc;
    struct Step {
      int u, g;
    };
    auto next = [&](Step& t) {
      t.u += du;
      t.g += dg;
      if (t.g >= gc) {
        t.g -= gc;
        ++t.u;
      }
    };
    Step ahead{wave / gc, wave % gc}, now = ahead;
    auto issue = [&](int slot) {
      bool in = ahead.u < nu;
      const int u = in ? ahead.u : 0, g = gc0 + ahead.g;
      int e = __builtin_amdgcn_readlane(ue[0], u & 63);
      if constexpr (ONE) {
        in &= e >= 0;
        e = max(e, 0);
      } else if (nu > 64) {
        const int e1 = __builtin_amdgcn_readlane(ue[1], u & 63);
        const int e2 = __builtin_amdgcn_readlane(ue[2], u & 63), e3 = __builtin_amdgcn_readlane(ue[3], u & 63);
        e = u < 128 ? (u < 64 ? e : e1) : (u < 192 ? e2 : e3);
      }
      const auto rw = few_rsrc(p.w2 + (int64_t)e * p.w2_expert, in ? p.w2_expert : 0);
      const auto rs = few_rsrc(p.s2 + (int64_t)e * p.s2_expert, in ? p.s2_expert * 4 : 0);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        wr[slot][h] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, lane * 16 + 1024 * h, (nb * G + g) * 2048, AUX));
      sw[slot] = __builtin_amdgcn_raw_buffer_load_b32(rs, 0, ((nb / 8) * G + g) * 4, 0);
      next(ahead);
    };
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      issue(s);
      __builtin_amdgcn_sched_barrier(0);  // step by step, as the waits of the loop below count them
    }
    if (gc0) __syncthreads();  // the groups before are multiplied
#pragma unroll 1
    for (int i = tid >> 4; i < ns * gc; i += 4 * kFewWaves) {
      const int s = i / gc, g = i - s * gc;
      // (the row of a slot without an expert was not written: what lies there
      // is quantised and not used)
      const int64_t slot = t0 * topk + s;
      const float ws = p.topk_w[slot];
      float f;
      uint2 q;
      if constexpr (WIDE) {
        q = *reinterpret_cast<const uint2*>(p.act_codes + slot * p.I + (gc0 + g) * 128 + c16 * 8);
        f = p.act[slot * G + gc0 + g];
      } else {
        const f4_t* src = reinterpret_cast<const f4_t*>(p.act + slot * p.I + (gc0 + g) * 128 + c16 * 8);
        const f4_t a = src[0], b = src[1];
        uint32_t top = 0u;
#pragma unroll
        for (int v = 0; v < 4; ++v) top = max(top, max(b8_mag(a[v]), b8_mag(b[v])));
        f = b8_scale(b8_row_max(top));
        const B8Div d(f);
        q = uint2{b8_codes(a[0], a[1], a[2], a[3], d), b8_codes(b[0], b[1], b[2], b[3], d)};
      }
      *reinterpret_cast<uint2*>(lds + s * pitch + g * 128 + c16 * 8) = q;
      if (c16 == 0) sc[s * gmax + g] = f * ws;  // the top-k weight rides on the scale
    }
    __syncthreads();
#pragma unroll 1
    for (int i = wave; i < steps; i += ST * kFewWaves) {
#pragma unroll
      for (int s = 0; s < ST; ++s) {
        const bool in = now.u < nu;
        int sl;
        if constexpr (ONE)
          sl = c16 == 0 && __builtin_amdgcn_readlane(ue[0], in ? now.u : 0) >= 0 ? now.u : -1;
        else
          sl = reinterpret_cast<const int16_t*>(slots_of)[(in ? now.u : 0) * 16 + c16];
        const bool has = in && sl >= 0;  // lanes of other tokens take nothing
        const int row = has ? sl : 0;
        const uint8_t* ar = lds + row * pitch + now.g * 128 + kq * 16;
        const f4_t P = b8_mfma(cat8(wr[s][0], wr[s][1]),
                               cat8(*reinterpret_cast<const u4_t*>(ar), *reinterpret_cast<const u4_t*>(ar + 64)));
        const float f = sc[row * gmax + now.g] * __uint_as_float(sw[s]);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = has ? fmaf(f, P[q], acc[q]) : acc[q];
        next(now);
        issue(s);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (tid < 64 && c16 < nt) {
    f4_t v = red[0][lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += red[w][lane][q];
    auto cv = [&](float x) -> uint32_t { return p.out_bf16 ? float_to_bf16_bits(x) : float_to_f16_bits(x); };
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (int64_t)(t0 + c16) * N + nb * 16 + 4 * kq) =
        uint2{cv(v[0]) | (cv(v[1]) << 16), cv(v[2]) | (cv(v[3]) << 16)};
  }
#endif
}

template <int NPL, bool BF16, bool WIDE, int NW, int ST>
hipError_t gate_up_k(const B8FewArgs& a, dim3 grid, size_t lds, hipStream_t s) {
  const hipError_t e = allow_lds<few_gate_up<NPL, BF16, WIDE, NW, ST>>(kFewLds);
  if (e != hipSuccess) return e;
  return launch_timed(few_gate_up<NPL, BF16, WIDE, NW, ST>, grid, dim3(64 * NW), lds, s, a);
}

template <bool BF16>
hipError_t gate_up_s(const B8FewArgs& a, dim3 grid, size_t lds, hipStream_t s) {
  if (a.act_codes) return gate_up_k<1, BF16, true, 8, 6>(a, grid, lds, s);
  if (a.t > 1) return gate_up_k<1, BF16, false, 4, 4>(a, grid, lds, s);
  if (!a.logits || a.E <= 64) return gate_up_k<1, BF16, false, 8, 7>(a, grid, lds, s);
  if (a.E <= 256) return gate_up_k<4, BF16, false, 8, 7>(a, grid, lds, s);
  return gate_up_k<16, BF16, false, 8, 7>(a, grid, lds, s);
}

}  // namespace

int launch_route(int64_t t, int E, int topk, int logit_type, const void* logits, int renorm, int32_t* ids, float* w,
                 void* stream) {
  const dim3 grid((unsigned)((t + 3) / 4)), block(256);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int ti = (int)t;
  // One token goes as the layer's gate_up routes it, whose weights are so the same
  // bits.  64 experts or fewer leave a wave per token nothing to gain; for more, a wave
  // has the shorter chain and sixteen lanes the fewer instructions (256 experts,
  // top 8, fp32: 4096 tokens 6.0 us by waves, 6.5 by rows, 16383 15.6 and 11.0).
  // The border was set for 256 experts; fewer would cross earlier (6143 tokens by
  // waves and 6144 by rows: 128 experts 6.4 and 4.2 us, 160 6.7 and 5.2, 192 7.1 and
  // 6.0, 256 7.1 both).
  if (t > 1 && topk <= 16 && (E <= 64 || (E <= 256 && t >= 6144))) {
    const dim3 rows((unsigned)((t + 15) / 16));
    auto go = [&]<int LT>() -> int {
      if (E <= 64) return (int)launch_timed(route_rows_kernel<LT, 4>, rows, block, 0, s, logits, ti, E, topk, renorm, ids, w);
      if (E <= 128) return (int)launch_timed(route_rows_kernel<LT, 8>, rows, block, 0, s, logits, ti, E, topk, renorm, ids, w);
      if (E <= 192) return (int)launch_timed(route_rows_kernel<LT, 12>, rows, block, 0, s, logits, ti, E, topk, renorm, ids, w);
      return (int)launch_timed(route_rows_kernel<LT, 16>, rows, block, 0, s, logits, ti, E, topk, renorm, ids, w);
    };
    return logit_type == 0 ? go.template operator()<0>() : (logit_type == 1 ? go.template operator()<1>() : go.template operator()<2>());
  }
  if (E <= 64) return (int)launch_timed(route_kernel<1>, grid, block, 0, s, logits, logit_type, ti, E, topk, renorm, ids, w);
  if (E <= 128) return (int)launch_timed(route_kernel<2>, grid, block, 0, s, logits, logit_type, ti, E, topk, renorm, ids, w);
  if (E <= 256) return (int)launch_timed(route_kernel<4>, grid, block, 0, s, logits, logit_type, ti, E, topk, renorm, ids, w);
  if (E <= 512) return (int)launch_timed(route_kernel<8>, grid, block, 0, s, logits, logit_type, ti, E, topk, renorm, ids, w);
  return (int)launch_timed(route_kernel<16>, grid, block, 0, s, logits, logit_type, ti, E, topk, renorm, ids, w);
}

// Rows of x a gate_up workgroup keeps quantised at a time (the weights are
// read again for each further so many): four cover an expert's tokens of a
// small batch nearly always, eight where a CU holds one workgroup anyway.
static int few_rows(const B8FewArgs& a) {
  const int64_t per = a.H + 16 + a.H / 128 * 4;
  return (int)std::max<int64_t>(1, std::min<int64_t>({(int64_t)a.t, a.act_codes ? 8 : 4, 96 * 1024 / per}));
}

// 128-k groups of a tile's activation rows a down workgroup holds at a time:
// two workgroups of a CU hold up to 48 KiB each.
static int few_down_groups(const B8FewArgs& a) {
  const int64_t ns = std::min(a.t, 16) * (int64_t)a.topk;
  return (int)std::max<int64_t>(1, std::min<int64_t>(a.I / 128, 48 * 1024 / (ns * 132)));
}

int launch_few_gate_up(const B8FewArgs& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  B8FewArgs b = a;
  b.rows = few_rows(a);
  const dim3 grid((unsigned)(a.I / (a.act_codes ? 128 : 16)), (unsigned)(a.t * a.topk + (a.logits || a.t > 1 ? 1 : 0)));
  const size_t lds = (size_t)b.rows * (a.H + 16 + a.H / 128 * 4);
  if (lds > kFewLds || (a.logits && a.t > 1)) return (int)hipErrorInvalidValue;
  return a.x_bf16 ? (int)gate_up_s<true>(b, grid, lds, s) : (int)gate_up_s<false>(b, grid, lds, s);
}

int launch_few_down(const B8FewArgs& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  B8FewArgs b = a;
  b.down_groups = few_down_groups(a);
  const size_t lds = (size_t)std::min(a.t, 16) * a.topk * (b.down_groups * 132 + 16);
  const dim3 grid((unsigned)(a.H / 16), (unsigned)((a.t + 15) / 16)), block(64 * kFewWaves);
  auto go = [&]<bool WIDE, bool ONE, int ST>() -> int {
    const hipError_t e = allow_lds<few_down<WIDE, ONE, ST>>(kFewLds);
    return e != hipSuccess ? (int)e : (int)launch_timed(few_down<WIDE, ONE, ST>, grid, block, lds, s, b);
  };
  // up to two steps a wave need no deeper ring
  const bool little = std::min(a.t, 16) * a.topk * b.down_groups <= 2 * kFewWaves;
  if (a.act_codes) return little ? go.template operator()<true, false, 2>() : go.template operator()<true, false, 6>();
  if (a.t == 1) return little ? go.template operator()<false, true, 2>() : go.template operator()<false, true, 6>();
  return little ? go.template operator()<false, false, 2>() : go.template operator()<false, false, 6>();
}

}  // namespace hq
