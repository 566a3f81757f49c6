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
// share one read (they are the columns of the matrix instruction).  The expert
// a slot stands for is found inside the kernels: a workgroup row per slot
// takes its token's j-th best logit, and the slots that share its expert are
// found by counting, per token, the logits that come before the expert's.
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <algorithm>

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

// LT: 0 fp32, 1 bf16, 2 fp16
template <int LT>
__device__ inline float load_logit(const void* p, int64_t i) {
  if constexpr (LT == 0) return static_cast<const float*>(p)[i];
  const uint32_t b = static_cast<const uint16_t*>(p)[i];
  return LT == 1 ? bf16_bits_to_float(b) : f16_bits_to_float(b);
}
__device__ inline float load_logit_rt(const void* p, int64_t i, int lt) {
  return lt == 0 ? load_logit<0>(p, i) : (lt == 1 ? load_logit<1>(p, i) : load_logit<2>(p, i));
}

// Wave-wide maximum, minimum and sum, uniform.
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

// The row of logits a wave holds: lane l keeps experts l, l + 64, ...
template <int NPL>
struct Logits {
  uint32_t key[NPL];
  __device__ inline void load(const void* p, int64_t row, int E, int lt, int lane) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 64 * i;
      key[i] = e < E ? logit_key(load_logit_rt(p, row * E + e, lt)) : 0u;
    }
  }
  // The best expert left (largest key, then lowest index), struck out; -1 if
  // none is left.  Uniform.
  __device__ inline int take(int lane, uint32_t* best) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) m = max(m, key[i]);
    m = wave_max(m);
    *best = m;
    if (m == 0u) return -1;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const uint64_t has = __ballot(key[i] == m);
      if (has) {
        const int l = __builtin_ctzll(has);
        if (lane == l) key[i] = 0u;
        return 64 * i + l;
      }
    }
    return -1;
  }
  // How many experts come before expert e with key k.  Uniform.
  __device__ inline int before(int lane, int e, uint32_t k) const {
    int n = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int o = lane + 64 * i;
      n += __popcll(__ballot(key[i] > k || (key[i] == k && o < e)));
    }
    return n;
  }
  __device__ inline float exp_sum(float top) const {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (key[i]) s += expf(key_logit(key[i]) - top);
    return wave_sum(s);
  }
};

// One wave per token.
template <int NPL>
__global__ void __launch_bounds__(256) route_kernel(const void* __restrict__ logits, int lt, int t, int E, int topk,
                                                    int renorm, int32_t* __restrict__ ids, float* __restrict__ w) {
  const int row = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (row >= t) return;
  Logits<NPL> x;
  x.load(logits, row, E, lt, lane);
  const uint32_t k0 = [&] {
    uint32_t m = x.key[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) m = max(m, x.key[i]);
    return wave_max(m);
  }();
  const float top = key_logit(k0);
  float sum = renorm ? 0.f : x.exp_sum(top);
  // lane j keeps choice j (topk <= 64)
  int my_id = -1;
  float my_e = 0.f;
  for (int j = 0; j < topk; ++j) {
    uint32_t k;
    const int e = x.take(lane, &k);
    if (e < 0) break;
    const float v = expf(key_logit(k) - top);
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

// ---------------------------------------------------------------------------
// gate_up: grid (16-column blocks of the outputs, slots); 8 waves over K
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;
constexpr int kFewLds = 128 * 1024;  // most dynamic LDS of a gate_up workgroup

template <int NPL, bool BF16>
__global__ void __launch_bounds__(64 * kFewWaves) few_gate_up(B8FewArgs p) {
#if defined(__HIP_DEVICE_COMPILE__)
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ f4_t red[kFewWaves][2][64];
  __shared__ int picks[kB8FewMaxSlots];  // slots that share this one's expert, in order
  __shared__ int npicks;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kq = lane >> 4;
  const int z = blockIdx.y, topk = p.topk, T = p.t, E = p.E, K = p.H, G = K / 128;
  const int tok = z / topk;

  // ---- the slot's expert -------------------------------------------------------
  int e = -1;
  uint32_t ekey = 0u;
  Logits<NPL> x;
  if (p.logits) {
    x.load(p.logits, tok, E, p.logit_type, lane);
    for (int j = z - tok * topk; j >= 0; --j) {
      e = x.take(lane, &ekey);
      if (e < 0) break;
    }
    e = __builtin_amdgcn_readfirstlane(e);
  } else {
    e = p.topk_ids[z];
    if (e < 0 || e >= E) e = -1;
  }
  if (p.logits && blockIdx.x == 0 && wave == kFewWaves - 1) {
    // this slot's routing, for the down kernel and the caller
    Logits<NPL> r;
    r.load(p.logits, tok, E, p.logit_type, lane);
    uint32_t k0 = r.key[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) k0 = max(k0, r.key[i]);
    const float top = key_logit(wave_max(k0));
    float sum = 0.f;
    if (p.renorm) {
      for (int j = 0; j < topk; ++j) {
        uint32_t k;
        if (r.take(lane, &k) < 0) break;
        sum += expf(key_logit(k) - top);
      }
    } else {
      sum = r.exp_sum(top);
    }
    if (lane == 0) {
      p.topk_ids[z] = e;
      p.topk_w[z] = e < 0 ? 0.f : expf(key_logit(ekey) - top) / sum;
    }
  }
  if (e < 0) return;

  // ---- first weight loads (they need the expert only) ---------------------------
  const int nbi = p.I / 16;
  const uint8_t* wbase = p.w1 + (int64_t)e * p.w1_expert;
  auto rsrc = [](const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
  };
  const auto rw = rsrc(wbase, p.w1_expert);
  const auto rws = rsrc(p.s1 + (int64_t)e * p.s1_expert, p.s1_expert * 4);
  int woff[2], swoff[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int nb = u * nbi + blockIdx.x;
    woff[u] = nb * G * 2048 + lane * 16;
    swoff[u] = (nb / 8) * G * 4;
  }
  constexpr int ST = 4;
  u4_t wr[ST][2][2];
  uint32_t sw[ST][2];
  auto issue = [&](int slot, int g) {
    const int past = g < G ? 0 : (int)0x80000000u;
    g = min(g, G - 1);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        wr[slot][u][h] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, (woff[u] + 1024 * h) | past, g * 2048, 0));
      sw[slot][u] = __builtin_amdgcn_raw_buffer_load_b32(rws, swoff[u] | past, g * 4, 0);
    }
  };
#pragma unroll
  for (int s = 0; s < ST; ++s) issue(s, wave + s * kFewWaves);

  // ---- the slots that share the expert ------------------------------------------
  if (p.logits) {
    // slot of token t' that holds e: how many logits come before e's
    for (int t = wave; t < T; t += kFewWaves) {
      Logits<NPL> y;
      y.load(p.logits, t, E, p.logit_type, lane);
      const uint32_t k = logit_key(load_logit_rt(p.logits, (int64_t)t * E + e, p.logit_type));
      const int rank = y.before(lane, e, k);
      if (lane == 0) picks[t] = (k && rank < topk) ? t * topk + rank : -1;
    }
    __syncthreads();
    if (wave == 0) {
      const int s = lane < T ? picks[lane] : -1;  // T <= 64
      const uint64_t has = __ballot(s >= 0);
      if (s >= 0) picks[__popcll(has & ((1ull << lane) - 1))] = s;
      if (lane == 0) npicks = __popcll(has);
    }
  } else if (wave == 0) {
    int n = 0;
    for (int b = 0; b < T * topk; b += 64) {
      const int s = b + lane;
      const bool hit = s < T * topk && p.topk_ids[s] == e;
      const uint64_t has = __ballot(hit);
      if (hit) picks[n + __popcll(has & ((1ull << lane) - 1))] = s;
      n += __popcll(has);
    }
    if (lane == 0) npicks = n;
  }
  __syncthreads();
  if (picks[0] != z) return;  // the first of them does the work
  const int n = npicks;

  const int pitch = K + 16, R = p.rows;
  float* sa = reinterpret_cast<float*>(lds + R * pitch);  // [R][G]
  for (int c0 = 0; c0 < n; c0 += R) {
    const int nr = min(n - c0, R);
    if (c0) {
      __syncthreads();  // the rows and sums of the chunk before are read
#pragma unroll
      for (int s = 0; s < ST; ++s) issue(s, wave + s * kFewWaves);
    }
    // ---- rows of x, quantised into LDS: 16 lanes a block ------------------------
    for (int i = tid >> 4; i < nr * G; i += 4 * kFewWaves) {
      const int r = i / G, g = i - r * G;
      const int64_t row = picks[c0 + r] / topk;
      float v[8];
      b8_unpack<BF16>(static_cast<const u4_t*>(p.x)[row * (K / 8) + g * 16 + c16], v);
      uint32_t top = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, b8_mag(v[j]));
      const float s = b8_scale(b8_row_max(top));
      const B8Div d(s);
      *reinterpret_cast<uint2*>(lds + r * pitch + g * 128 + c16 * 8) =
          uint2{b8_codes(v[0], v[1], v[2], v[3], d), b8_codes(v[4], v[5], v[6], v[7], d)};
      if (c16 == 0) sa[r * G + g] = s;
    }
    __syncthreads();
    // ---- K over the waves -------------------------------------------------------
    const int rl = min(c16, nr - 1);
    f4_t acc[2] = {f4_t{0.f, 0.f, 0.f, 0.f}, f4_t{0.f, 0.f, 0.f, 0.f}};
    for (int g = wave; g < G; g += ST * kFewWaves) {
#pragma unroll
      for (int s = 0; s < ST; ++s) {
        const int gg = min(g + s * kFewWaves, G - 1);  // past the end the weights and their scales are zero
        const u4_t a0 = *reinterpret_cast<const u4_t*>(lds + rl * pitch + gg * 128 + kq * 16);
        const u4_t a1 = *reinterpret_cast<const u4_t*>(lds + rl * pitch + gg * 128 + 64 + kq * 16);
        const float f = sa[rl * G + gg];
        const bool in = g + s * kFewWaves < G;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const f4_t P = b8_mfma(cat8(wr[s][u][0], wr[s][u][1]), cat8(a0, a1));
          const float m = in ? f * __uint_as_float(sw[s][u]) : 0.f;
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[u][q] = fmaf(m, P[q], acc[u][q]);
        }
        issue(s, g + (s + ST) * kFewWaves);
      }
    }
    red[wave][0][lane] = acc[0];
    red[wave][1][lane] = acc[1];
    __syncthreads();
    if (tid < 64 && c16 < nr) {
      f4_t h[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        h[u] = red[0][u][lane];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w)
#pragma unroll
          for (int q = 0; q < 4; ++q) h[u][q] += red[w][u][lane][q];
      }
      f4_t a;
#pragma unroll
      for (int q = 0; q < 4; ++q) a[q] = b8_silu_mul(h[0][q], h[1][q]);
      *reinterpret_cast<f4_t*>(p.act + (int64_t)picks[c0 + c16] * p.I + blockIdx.x * 16 + 4 * kq) = a;
    }
  }
#endif
}

// ---------------------------------------------------------------------------
// down + combine: grid (column blocks, tiles of 16 tokens); the waves take the
// (expert, group) steps in turn
// ---------------------------------------------------------------------------
template <int NB>
__global__ void __launch_bounds__(64 * kFewWaves) few_down(B8FewArgs p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kMaxTile = 16 * kB8FewMaxTopk;
  __shared__ f4_t red[kFewWaves][NB][64];
  __shared__ int key[kMaxTile];           // expert | occurrence << 16, -1: none
  __shared__ int units[kMaxTile];         // first slot of each distinct key, in slot order
  __shared__ short slot_of[kMaxTile][16]; // [first slot][token of the tile]: the slot with that key, -1 none
  __shared__ float wt[kMaxTile];
  __shared__ int wcount[4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kq = lane >> 4;
  const int topk = p.topk, t0 = blockIdx.y * 16, nt = min(16, p.t - t0), ns = nt * topk;
  const int G = p.I / 128, N = p.H;

  // ---- the distinct experts of the tile's slots --------------------------------
  // A token may hold an expert more than once (given ids): each occurrence is
  // a unit of its own, so that a unit has at most one slot per token.
  for (int i = tid; i < ns * 8; i += 64 * kFewWaves) reinterpret_cast<int*>(slot_of)[i] = -1;
  int id = -1;
  if (tid < ns) {
    id = p.topk_ids[t0 * topk + tid];
    if (id < 0 || id >= p.E) id = -1;
    key[tid] = id;
    wt[tid] = p.topk_w[t0 * topk + tid];
  }
  __syncthreads();
  const int my_tok = tid / topk;
  int occ = 0;
  if (tid < ns && id >= 0)
    for (int s = my_tok * topk; s < tid; ++s) occ += key[s] == id;
  __syncthreads();
  if (tid < ns && id >= 0) key[tid] = id | (occ << 16);
  __syncthreads();
  int first = -1;
  if (tid < ns && id >= 0) {
    const int k = id | (occ << 16);
    for (first = 0; key[first] != k; ++first) {
    }
    slot_of[first][my_tok] = (short)tid;
  }
  const bool lead = first >= 0 && first == tid;
  const uint64_t leads = __ballot(lead);
  if (lane == 0 && wave < 4) wcount[wave] = __popcll(leads);
  __syncthreads();
  if (lead) {
    int at = __popcll(leads & ((1ull << lane) - 1));
    for (int w = 0; w < wave; ++w) at += wcount[w];
    units[at] = tid;
  }
  __syncthreads();
  const int nu = wcount[0] + wcount[1] + wcount[2] + wcount[3];
  const int steps = nu * G;

  auto rsrc = [](const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
  };
  const auto ract = rsrc(p.act, (int64_t)p.t * topk * p.I * 4);
  const int nblocks = N / 16, nb0 = blockIdx.x * NB;
  constexpr int ST = 2;
  u4_t wr[ST][NB][2];
  u4_t av[ST][8];
  uint32_t sw[ST][NB];
  float tw[ST];
  bool has[ST];  // whether the lane's token holds the unit's expert
  auto issue = [&](int slot, int i) {
    const bool in = i < steps;
    const int ii = in ? i : 0;
    const int u = ii / G, g = ii - u * G;
    const int s0 = __builtin_amdgcn_readfirstlane(steps ? units[u] : 0);
    const int e = __builtin_amdgcn_readfirstlane(steps ? key[s0] & 0xFFFF : 0);
    const auto rw = rsrc(p.w2 + (int64_t)e * p.w2_expert, in ? p.w2_expert : 0);
    const auto rs = rsrc(p.s2 + (int64_t)e * p.s2_expert, in ? p.s2_expert * 4 : 0);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int nb = min(nb0 + j, nblocks - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        wr[slot][j][h] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, lane * 16 + 1024 * h, (nb * G + g) * 2048, 0));
      sw[slot][j] = __builtin_amdgcn_raw_buffer_load_b32(rs, 0, ((nb / 8) * G + g) * 4, 0);
    }
    const int s = in ? slot_of[s0][c16] : -1;
    has[slot] = s >= 0;
    tw[slot] = wt[max(s, 0)];
    const int off = s >= 0 ? ((t0 * topk + s) * p.I + g * 128 + 16 * kq) * 4 : (int)0x80000000u;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      av[slot][q] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(ract, off, (q & 3) * 16 + (q >> 2) * 256, 0));
  };
  f4_t acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = f4_t{0.f, 0.f, 0.f, 0.f};
  if (steps) {
#pragma unroll
    for (int s = 0; s < ST; ++s) issue(s, wave + s * kFewWaves);
    for (int i = wave; i < steps; i += ST * kFewWaves) {
#pragma unroll
      for (int s = 0; s < ST; ++s) {
        // quantise the token's 128 values: 32 in this lane, four lanes a block
        uint32_t top = 0u;
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
          for (int r = 0; r < 4; ++r) top = max(top, av[s][q][r] & 0x7FFFFFFFu);
        top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
        const float sc = b8_scale(top);
        const B8Div d(sc);
        i8_t a;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          a[q] = (int)b8_codes(__uint_as_float(av[s][q][0]), __uint_as_float(av[s][q][1]), __uint_as_float(av[s][q][2]),
                               __uint_as_float(av[s][q][3]), d);
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const f4_t P = b8_mfma(cat8(wr[s][j][0], wr[s][j][1]), a);
          const float f = tw[s] * (sc * __uint_as_float(sw[s][j]));
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[j][q] = has[s] ? fmaf(f, P[q], acc[j][q]) : acc[j][q];
        }
        issue(s, i + (s + ST) * kFewWaves);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) red[wave][j][lane] = acc[j];
  __syncthreads();
  for (int i = tid; i < NB * 64; i += 64 * kFewWaves) {
    const int j = i >> 6, l = i & 63;
    f4_t v = red[0][j][l];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += red[w][j][l][q];
    const int t = l & 15, nb = nb0 + j;
    if (t >= nt || nb >= nblocks) continue;
    auto cv = [&](float x) -> uint32_t { return p.out_bf16 ? float_to_bf16_bits(x) : float_to_f16_bits(x); };
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (int64_t)(t0 + t) * N + nb * 16 + 4 * (l >> 4)) =
        uint2{cv(v[0]) | (cv(v[1]) << 16), cv(v[2]) | (cv(v[3]) << 16)};
  }
#endif
}

template <int NPL>
hipError_t gate_up_t(const B8FewArgs& a, dim3 grid, size_t lds, hipStream_t s) {
  const dim3 block(64 * kFewWaves);
  const hipError_t e = a.x_bf16 ? allow_lds<few_gate_up<NPL, true>>(kFewLds) : allow_lds<few_gate_up<NPL, false>>(kFewLds);
  if (e != hipSuccess) return e;
  return a.x_bf16 ? launch_timed(few_gate_up<NPL, true>, grid, block, lds, s, a)
                  : launch_timed(few_gate_up<NPL, false>, grid, block, lds, s, a);
}

}  // namespace

int launch_route(int64_t t, int E, int topk, int logit_type, const void* logits, int renorm, int32_t* ids, float* w,
                 void* stream) {
  const dim3 grid((unsigned)((t + 3) / 4)), block(256);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int ti = (int)t;
  if (E <= 64) return (int)launch_timed(route_kernel<1>, grid, block, 0, s, logits, logit_type, ti, E, topk, renorm, ids, w);
  if (E <= 128) return (int)launch_timed(route_kernel<2>, grid, block, 0, s, logits, logit_type, ti, E, topk, renorm, ids, w);
  if (E <= 256) return (int)launch_timed(route_kernel<4>, grid, block, 0, s, logits, logit_type, ti, E, topk, renorm, ids, w);
  if (E <= 512) return (int)launch_timed(route_kernel<8>, grid, block, 0, s, logits, logit_type, ti, E, topk, renorm, ids, w);
  return (int)launch_timed(route_kernel<16>, grid, block, 0, s, logits, logit_type, ti, E, topk, renorm, ids, w);
}

// Rows of x a workgroup keeps quantised at a time: four cover an expert's
// tokens of a small batch nearly always (the weights are read again for each
// further four), fewer where K is long.
int b8_few_rows(int64_t t, int64_t K) {
  const int64_t per = K + 16 + K / 128 * 4;
  return (int)std::max<int64_t>(1, std::min<int64_t>({t, 4, 96 * 1024 / per}));
}

int launch_few_gate_up(const B8FewArgs& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)(a.I / 16), (unsigned)(a.t * a.topk));
  const size_t lds = (size_t)a.rows * (a.H + 16 + a.H / 128 * 4);
  if (lds > kFewLds) return (int)hipErrorInvalidValue;
  if (!a.logits || a.E <= 64) return (int)gate_up_t<1>(a, grid, lds, s);
  if (a.E <= 256) return (int)gate_up_t<4>(a, grid, lds, s);
  return (int)gate_up_t<16>(a, grid, lds, s);
}

int launch_few_down(const B8FewArgs& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const unsigned tiles = (unsigned)((a.t + 15) / 16);
  const int nblocks = a.H / 16;
  return (int)launch_timed(few_down<1>, dim3((unsigned)nblocks, tiles), dim3(64 * kFewWaves), 0, s, a);
}

}  // namespace hq
