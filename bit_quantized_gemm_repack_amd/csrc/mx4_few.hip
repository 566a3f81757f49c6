// An experts' layer in MXFP4 for a few tokens, in two kernels.
//
//   gate_up   h = q(x) W1[e]^T
//   down      y[t] = sum_j w[t, j] q(SiLU(h[:I]) * h[I:]) W2[e]^T
//
// Both are bound by reading the chosen experts' weights, which every workgroup streams
// straight to registers, its waves taking the steps along K in turn; tokens that picked the
// same expert share one read (they are the columns of the matrix instruction).  One token of
// top 8, H = 7168, I = 256: 6.6 + 6.1 us start to end, of which the 23 MB of weights take 3.7 at
// the 6.4 TB/s that plain reads reach and starting, ids, the row's quantisation and the sums over
// waves the rest; 4 tokens 15.3 + 8.9; 8 tokens 24.3 + 14.8 for 164 MB (26 us).
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <algorithm>

#include "few_device.h"
#include "launch.h"
#include "mx4.h"
#include "mx4_device.h"
#include "mx4_product.h"

namespace hq {

namespace {

// Columns of gate_up by 16 rather than by strip: while that makes at most two workgroups a
// CU (top 8, us a layer in a graph by column / by strip: H = 7168, I = 256: 2 tokens 19.7 / 22.5, 3 tokens
// 26.5 / 22.6, 4 tokens 31.8 / 25.0; H = 2048, I = 768: 1 token 16.7 / 15.8, 2 tokens 29.1 / 22.1).
bool narrow(int64_t t, int64_t topk, int64_t I) { return t * topk * (I / 8) <= 512; }

constexpr int kDownWaves = 8;
constexpr int kFewLds = 64 * 1024;  // most dynamic LDS of a workgroup

// Bytes of a row of k values in LDS, codes and then powers of two: a multiple of 16 that
// spreads the rows an operand reads over the banks.
__host__ __device__ constexpr int64_t row_bytes(int64_t k) { return (k / 2 + k / 32 + 31) / 16 * 16; }

// 128 values of a row (16 lanes, 8 each) -> its codes and powers of two.
__device__ inline void few_codes(const float (&v)[8], uint8_t* codes, uint8_t* scale, int c16) {
  uint32_t top = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, b8_mag(v[j]));
  const uint32_t s = mx4_scale(quad_max(top));
  *reinterpret_cast<uint32_t*>(codes + c16 * 4) = mx4_word(v, s);
  if ((c16 & 3) == 0) scale[c16 >> 2] = (uint8_t)s;
}

// ---------------------------------------------------------------------------
// gate_up.  A workgroup row per slot; the first of the slots that share an expert does the
// work for all of them.  NF = 1: 16 columns a workgroup, gate or up, fp32 sums out (where the slots' strips would leave most CUs idle); NF = 4: a strip,
// 32 outputs, one block of the intermediate, quantised.  One more row of workgroups finds
// the units that the down kernel walks.
// ---------------------------------------------------------------------------
template <int INPUT, int NF, int NW, int ST, int Q>
__global__ void __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(NF == 4 ? 2 : 4))) mx4_few_gate_up(Mx4FewArgs p) {
#if defined(__HIP_DEVICE_COMPILE__)
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // rows: codes and powers of two
  __shared__ f4_t red[NW][NF][64];
  __shared__ __attribute__((aligned(16))) int picks[kB8FewMaxSlots];
  __shared__ int npicks;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kq = lane >> 4;
  const int z = blockIdx.y, K = p.H, G = K / 128, steps = G / Q;
  if (z == p.t * p.topk) {  // the last row
    for (int tile = blockIdx.x; tile * 16 < p.t; tile += gridDim.x) few_units<NW>(p, tile, picks, tid);
    return;
  }
  // the slot's own row of x is the first of the rows below: its loads (up to 64 groups) come
  // before the weights', which return in order
  constexpr int XP = 16 / NW;
  u4_t xr[XP];
  uint32_t xc[XP], xs[XP];
  auto load_x = [&](int64_t row, int g, u4_t& raw, uint32_t& code, uint32_t& scale) {
    if constexpr (INPUT == MX4_CODES) {
      code = static_cast<const uint32_t*>(p.x)[row * (K / 8) + g * 16 + c16];
      scale = p.x_scale[(int64_t)g * p.t + row];
    } else {
      raw = static_cast<const u4_t*>(p.x)[row * (K / 8) + g * 16 + c16];
    }
  };
  const int scales = K / 2, pitch = (int)row_bytes(K);
  auto put_x = [&](int r, int g, u4_t raw, uint32_t code, uint32_t scale) {
    uint8_t* row = lds + r * pitch;
    if constexpr (INPUT == MX4_CODES) {
      *reinterpret_cast<uint32_t*>(row + g * 64 + c16 * 4) = code;
      if (c16 == 0) *reinterpret_cast<uint32_t*>(row + scales + g * 4) = scale;
    } else {
      float v[8];
      b8_unpack<INPUT == MX4_BF16>(raw, v);
      few_codes(v, row + g * 64, row + scales + g * 4, c16);
    }
  };
#pragma unroll
  for (int u = 0; u < XP; ++u) load_x(z / p.topk, min((tid >> 4) + 4 * NW * u, G - 1), xr[u], xc[u], xs[u]);
  int ids[kScan] = {};
  if (p.t > 1 && wave == 0) few_ids(p, ids, lane);
  int e = p.topk_ids[z];
  e = __builtin_amdgcn_readfirstlane(e);
  if (e < 0 || e >= p.E) return;

  // ---- weight stream: steps wave, wave + NW, ... of this workgroup's fragments ----
  const int strip = NF == 4 ? blockIdx.x : blockIdx.x >> 2, j0 = NF == 4 ? 0 : blockIdx.x & 3;
  const auto rw = few_rsrc(p.w1 + (int64_t)e * p.w1_expert, p.w1_expert);
  const int first = strip * G * kMx4GroupBytes;
  u4_t wr[ST][Q][NF];
  Mx4Scales<Q> sw[ST];
  auto issue = [&](int slot, int s) {
    const int past = s < steps ? 0 : (int)0x80000000u;  // steps past the end read nothing and hold zeros
    const int at = first + min(s, steps - 1) * Q * kMx4GroupBytes;
#pragma unroll
    for (int u = 0; u < Q; ++u)
#pragma unroll
      for (int j = 0; j < NF; ++j)
        wr[slot][u][j] = __builtin_bit_cast(
            u4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, (lane * 16 + j * 1024) | past, at + u * 4096 + j0 * 1024, NF == 4 ? kReadOnce : 0));
    sw[slot].template load<0>(rw, lane, at);
  };
#pragma unroll
  for (int s = 0; s < ST; ++s) {
    issue(s, wave + s * NW);
    __builtin_amdgcn_sched_barrier(0);  // step by step, as the waits of the loop below count them
  }
  int n = 1;
  if (p.t == 1) {
    if (tid == 0) picks[0] = z;  // (an expert that comes twice is read twice)
  } else {
    n = few_slots(p, e, ids, picks, &npicks, lane, wave);
    if (picks[0] != z) return;
  }
  const int R = p.rows;
  for (int c0 = 0; c0 < n; c0 += R) {
    const int nr = min(n - c0, R);
    if (c0) {
      __syncthreads();  // the rows and sums of the chunk before are read
#pragma unroll
      for (int s = 0; s < ST; ++s) issue(s, wave + s * NW);
    } else {
#pragma unroll
      for (int u = 0; u < XP; ++u) {
        const int g = (tid >> 4) + 4 * NW * u;
        if (g < G) put_x(0, g, xr[u], xc[u], xs[u]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // the rest of the rows' groups: row i / G, group i % G
    const int done = c0 ? 0 : min(G, 4 * NW * XP);
#pragma unroll 1
    for (int i = done + (tid >> 4); i < nr * G; i += 4 * NW) {
      const int r = i / G, g = i - r * G;
      u4_t raw;
      uint32_t code, scale;
      load_x((!c0 && !r) ? z / p.topk : picks[c0 + r] / p.topk, g, raw, code, scale);
      put_x(r, g, raw, code, scale);
    }
    __syncthreads();
    const uint8_t* ar = lds + min(c16, nr - 1) * pitch;
    f4_t acc[NF];
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[j] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int s0 = wave; s0 < steps; s0 += ST * NW) {
#pragma unroll
      for (int s = 0; s < ST; ++s) {
        const int g = min(s0 + s * NW, steps - 1) * Q;  // past the end the weights are zeros
#pragma unroll
        for (int u = 0; u < Q; ++u) {
          const u4_t a = *reinterpret_cast<const u4_t*>(ar + (g + u) * 64 + kq * 16);
          const uint32_t sa = ar[scales + (g + u) * 4 + kq];
          if constexpr (NF == 4)
            mx4_strip(wr[s][u], a, acc, sw[s].v[u], sa);
          else
            acc[0] = mx4_mfma<0>(wr[s][u][0], a, acc[0], sw[s].v[u] >> (8 * j0), sa);
        }
        issue(s, s0 + (s + ST) * NW);
        __builtin_amdgcn_sched_barrier(0);  // one step's operands at a time: the ring fills the registers
      }
    }
#pragma unroll
    for (int j = 0; j < NF; ++j) red[wave][j][lane] = acc[j];
    __syncthreads();
    if (wave < NF) {
      f4_t v = red[0][wave][lane];
#pragma unroll
      for (int w = 1; w < NW; ++w)
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += red[w][wave][lane][q];
      if constexpr (NF == 1) {
        if (c16 < nr)
          *reinterpret_cast<f4_t*>(p.h + (int64_t)picks[c0 + c16] * 2 * p.I + mx4_column(2 * p.I, true, strip, j0, 4 * kq)) = v;
      } else {
        red[0][wave][lane] = v;
      }
    }
    if constexpr (NF == 4) {
      __syncthreads();
      if (wave == 0) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = b8_silu_mul(red[0][i >> 2][lane][i & 3], red[0][2 + (i >> 2)][lane][i & 3]);
        uint32_t s;
        const uint32_t codes = mx4_block_codes(v, kq, s);
        if (c16 < nr) {
          const int64_t slot = picks[c0 + c16];
          *reinterpret_cast<uint32_t*>(p.act + slot * (p.I / 2) + strip * 16 + (kq & 1) * 8 + (kq >> 1) * 4) = codes;
          if (kq == 0) p.act_scale[slot * (p.I / 32) + strip] = (uint8_t)s;
        }
      }
    }
  }
#endif
}

// ---------------------------------------------------------------------------
// down and the sum: grid (blocks of 16 NF columns, tiles of 16 tokens).  The tile's
// activation rows lie in LDS; the waves take the (expert, step) pairs in turn, and each
// product is weighted on its way into one fp32 sum.
// ---------------------------------------------------------------------------
template <bool NARROW, bool ONE, int NF, int ST, int Q>
__global__ void __launch_bounds__(64 * kDownWaves) mx4_few_down(Mx4FewArgs p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kMax = 16 * kB8FewMaxTopk;  // slots of a tile
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ f4_t red[kDownWaves][NF][64];
  __shared__ int slots_of[ONE ? 1 : kMax * 8];  // [unit][token of the tile]: its slot as 16 bits, -1 none
  __shared__ float ltw[kMax];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kq = lane >> 4;
  const int topk = p.topk, t0 = blockIdx.y * 16, nt = min(16, p.t - t0), ns = nt * topk;
  const int G = p.I / 128, N = p.H;

  // A lane keeps the experts of four units (-1: none), so that a step finds its own without
  // a trip to LDS.  One token's slots are its units, those without an expert too: their
  // steps read nothing.
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
    for (int i = tid; i < nu * 8; i += 64 * kDownWaves) slots_of[i] = un[16 + kMax + i];
  }
  const int f0 = blockIdx.x * NF, strip = f0 >> 2, j0 = f0 & 3;
  const int first = strip * G * kMx4GroupBytes, per = G / Q, steps = nu * per;
  u4_t wr[ST][Q][NF];
  Mx4Scales<Q> sw[ST];
  auto issue = [&](int slot, int i) {
    bool in = i < steps;
    const int u = in ? i / per : 0, s = in ? i - u * per : 0;
    int e = __builtin_amdgcn_readlane(ue[0], u & 63);
    if constexpr (ONE) {
      in &= e >= 0;
      e = max(e, 0);
    } else if (nu > 64) {
      const int e1 = __builtin_amdgcn_readlane(ue[1], u & 63);
      const int e2 = __builtin_amdgcn_readlane(ue[2], u & 63), e3 = __builtin_amdgcn_readlane(ue[3], u & 63);
      e = u < 128 ? (u < 64 ? e : e1) : (u < 192 ? e2 : e3);
    }
    if (!in) e = 0;  // (no unit at all: what the lanes hold is no expert)
    const auto rw = few_rsrc(p.w2 + (int64_t)e * p.w2_expert, in ? p.w2_expert : 0);
    const int at = first + s * Q * kMx4GroupBytes;
#pragma unroll
    for (int g = 0; g < Q; ++g)
#pragma unroll
      for (int j = 0; j < NF; ++j)
        wr[slot][g][j] = __builtin_bit_cast(
            u4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, lane * 16 + j * 1024, at + g * 4096 + j0 * 1024, 0));
    sw[slot].template load<0>(rw, lane, at);
  };
#pragma unroll
  for (int s = 0; s < ST; ++s) {
    issue(s, wave + s * kDownWaves);
    __builtin_amdgcn_sched_barrier(0);  // step by step, as the waits of the loop below count them
  }
  const int scales = p.I / 2, pitch = (int)row_bytes(p.I);
#pragma unroll 1
  for (int i = tid >> 4; i < ns * G; i += 4 * kDownWaves) {
    const int s = i / G, g = i - s * G;
    // (the row of a slot without an expert was not written: what lies there is not used)
    const int64_t slot = (int64_t)t0 * topk + s;
    uint8_t* row = lds + s * pitch;
    if constexpr (NARROW) {
      const f4_t* gate = reinterpret_cast<const f4_t*>(p.h + slot * 2 * p.I + g * 128 + c16 * 8);
      const f4_t* up = reinterpret_cast<const f4_t*>(p.h + slot * 2 * p.I + p.I + g * 128 + c16 * 8);
      const f4_t ga[2] = {gate[0], gate[1]}, ua[2] = {up[0], up[1]};
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = b8_silu_mul(ga[q >> 2][q & 3], ua[q >> 2][q & 3]);
      few_codes(v, row + g * 64, row + scales + g * 4, c16);
    } else {
      *reinterpret_cast<uint32_t*>(row + g * 64 + c16 * 4) = *reinterpret_cast<const uint32_t*>(p.act + slot * (p.I / 2) + g * 64 + c16 * 4);
      if (c16 == 0) *reinterpret_cast<uint32_t*>(row + scales + g * 4) = *reinterpret_cast<const uint32_t*>(p.act_scale + slot * (p.I / 32) + g * 4);
    }
    if (g == 0 && c16 == 0) ltw[s] = p.topk_w[slot];
  }
  __syncthreads();
  f4_t acc[NF];
#pragma unroll
  for (int j = 0; j < NF; ++j) acc[j] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int i = wave; i < steps; i += ST * kDownWaves) {
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      const int at = i + s * kDownWaves;
      const bool in = at < steps;
      const int u = in ? at / per : 0, g0 = in ? (at - u * per) * Q : 0;
      int sl;
      if constexpr (ONE)
        sl = c16 == 0 && __builtin_amdgcn_readlane(ue[0], u) >= 0 ? u : -1;
      else
        sl = reinterpret_cast<const int16_t*>(slots_of)[u * 16 + c16];
      if constexpr (!ONE) sl = sl >= 0 ? sl : -1;
      const bool has = in && sl >= 0;  // lanes of other tokens take nothing
      const int row = has ? sl : 0;
      const uint8_t* ar = lds + row * pitch;
      f4_t P[NF];
#pragma unroll
      for (int j = 0; j < NF; ++j) P[j] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int g = 0; g < Q; ++g) {
        const u4_t a = *reinterpret_cast<const u4_t*>(ar + (g0 + g) * 64 + kq * 16);
        const uint32_t sa = ar[scales + (g0 + g) * 4 + kq], ws = sw[s].v[g] >> (8 * j0);
        P[0] = mx4_mfma<0>(wr[s][g][0], a, P[0], ws, sa);
        if constexpr (NF > 1) P[1] = mx4_mfma<1>(wr[s][g][1], a, P[1], ws, sa);
      }
      const float f = ltw[row];
#pragma unroll
      for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[j][q] = has ? fmaf(f, P[j][q], acc[j][q]) : acc[j][q];
      issue(s, at + ST * kDownWaves);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int j = 0; j < NF; ++j) red[wave][j][lane] = acc[j];
  __syncthreads();
  if (wave < NF && c16 < nt) {
    f4_t v = red[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kDownWaves; ++w)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += red[w][wave][lane][q];
    auto cv = [&](float x) -> uint32_t { return p.out_bf16 ? float_to_bf16_bits(x) : float_to_f16_bits(x); };
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (int64_t)(t0 + c16) * N + (f0 + wave) * 16 + 4 * kq) =
        uint2{cv(v[0]) | (cv(v[1]) << 16), cv(v[2]) | (cv(v[3]) << 16)};
  }
#endif
}

template <int INPUT, int Q>
hipError_t gate_up(const Mx4FewArgs& a, hipStream_t s) {
  const size_t lds = (size_t)a.rows * row_bytes(a.H);
  const unsigned slots = (unsigned)(a.t * a.topk) + (a.t > 1 ? 1 : 0);
  auto go = [&]<int NF, int NW, int ST>() -> hipError_t {
    const hipError_t e = allow_lds<mx4_few_gate_up<INPUT, NF, NW, ST, Q>>(kFewLds);
    if (e != hipSuccess) return e;
    return launch_timed(mx4_few_gate_up<INPUT, NF, NW, ST, Q>, dim3((unsigned)(NF == 4 ? a.I / 32 : a.I / 8), slots), dim3(64 * NW), lds, s, a);
  };
  if (!a.h) return go.template operator()<4, 4, 3>();
  return a.H / (128 * Q) > 16 ? go.template operator()<1, 8, 4>() : go.template operator()<1, 4, 4>();
}

template <int Q>
hipError_t down(const Mx4FewArgs& a, hipStream_t s) {
  const size_t lds = (size_t)std::min(a.t, 16) * a.topk * row_bytes(a.I);
  auto go = [&]<bool NARROW, bool ONE, int NF, int ST>() -> hipError_t {
    const hipError_t e = allow_lds<mx4_few_down<NARROW, ONE, NF, ST, Q>>(kFewLds);
    if (e != hipSuccess) return e;
    return launch_timed(mx4_few_down<NARROW, ONE, NF, ST, Q>, dim3((unsigned)(a.H / (16 * NF)), (unsigned)((a.t + 15) / 16)), dim3(64 * kDownWaves),
                        lds, s, a);
  };
  // one token has no units: its slots take their place (few_units did not run)
  if (a.h) return a.t == 1 ? go.template operator()<true, true, 1, 2>() : go.template operator()<true, false, 1, 2>();
  return a.t == 1 ? go.template operator()<false, true, 2, 4>() : go.template operator()<false, false, 2, 4>();
}

}  // namespace

bool mx4_few_ok(int64_t t, int64_t topk, int64_t E, int64_t H, int64_t I) {
  // The aligned path starts two kernels more, and its gate_up walks all of K in each wave; but
  // its workgroups are larger, which many slots pay for.  us a layer here / there (bf16, uniform
  // routing, in a graph), by what each limit below is drawn from:
  //   slots by H: top 8 of 256 experts, H = 7168, I = 256: 1 token 12.7 / 35.2, 4 tokens 25.0 /
  //     41.7, 9 tokens 46.8 / 48.7, 13 tokens 62 / 56; H = 2048, I = 768: 2 tokens 20.9 / 25.6,
  //     3 tokens 28.3 / 25.7
  //   slots by I, as a down workgroup forms all its tile's codes first: 8 experts, H = 4096, I =
  //     2048: top 1, 8 tokens 24.3 / 32.0, 12 tokens 31.6 / 33.1, 16 tokens 36.0 / 33.6; top 8,
  //     1 token 28.0 / 35.6, 2 tokens 38.9 / 35.8; 64 experts, H = 4096, I = 512, top 4: 8 tokens
  //     27.3 / 31.2, 10 tokens 34.3 / 32.9
  //   rows an expert, as its weights are read again for each four: 8 experts, H = 7168, I = 256:
  //     top 1, 17 tokens 27.9 / 31.4, 24 tokens 30.5 / 25.3; top 2, 10 tokens 26.1 / 30.5, 17
  //     tokens 35.3 / 30.1; 16 experts, top 2, 16 tokens 24.9 / 32.7, 24 tokens 38.7 / 32.1; four
  //     tokens are four rows at most: 8 experts, top 8 21.8 / 30.3
  //   tiles of 16 tokens, each of which reads down's weights: top 1, H = 7168, I = 256: 16 / 64 /
  //     256 experts, 32 tokens 27.9 / 32.5, 27.0 / 36.7, 27.9 / 39.6; 40 tokens 40.0 / 33.1, 35.4 /
  //     38.3, 36.9 / 41.7; 64 tokens 52.6 / 33.3, 47.7 / 41.3, 47.9 / 45.9
  const int64_t slots = t * topk;
  return t >= 1 && t <= kMx4FewTokens && topk >= 1 && topk <= kMx4FewTopk && slots * 96 <= H && slots * I <= 20000 &&
         (2 * slots <= 5 * E || t <= 4) && E <= 4096 && row_bytes(H) <= kFewLds && std::min<int64_t>(t, 16) * topk * row_bytes(I) <= kFewLds;
}

size_t mx4_few_act_bytes(int64_t t, int64_t topk, int64_t I) {
  return (size_t)(t * topk) * (size_t)(narrow(t, topk, I) ? 8 * I : I / 2 + I / 32);
}

int launch_mx4_few(const Mx4FewArgs& a, void* stream) {
  if (!mx4_few_ok(a.t, a.topk, a.E, a.H, a.I) || a.H % 128 || a.I % 128) return (int)hipErrorInvalidValue;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  Mx4FewArgs b = a;
  if (narrow(a.t, a.topk, a.I))
    b.act = b.act_scale = nullptr;
  else
    b.h = nullptr;
  // rows of x a gate_up workgroup keeps at a time (the weights are read again for each
  // further so many): four cover an expert's tokens where routing is even, as mx4_few_ok
  // allows 2.5 an expert
  b.rows = (int)std::max<int64_t>(1, std::min<int64_t>({(int64_t)a.t, 4, kFewLds / row_bytes(a.H)}));
  const TimingEvents ev = take_timing();
  arm_timing({ev.start, nullptr});
  auto up = [&]<int Q>() {
    return a.input == MX4_CODES ? gate_up<MX4_CODES, Q>(b, s) : (a.input == MX4_BF16 ? gate_up<MX4_BF16, Q>(b, s) : gate_up<MX4_F16, Q>(b, s));
  };
  hipError_t e = mx4_groups(a.H / 128) == 2 ? up.template operator()<2>() : up.template operator()<1>();
  if (e != hipSuccess) return (int)e;
  arm_timing({nullptr, ev.stop});
  e = mx4_groups(a.I / 128) == 2 ? down<2>(b, s) : down<1>(b, s);
  return (int)e;
}

}  // namespace hq
