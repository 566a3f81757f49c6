// fp8 x fp8 GEMM with 128-block scales, few rows: bound by reading the weight
// once.  A workgroup owns NB 16-column blocks and 16 rows; its waves take
// the 128-k groups of its K range in turn, weights straight from memory to
// registers (no other wave needs them), ST groups of loads in flight per wave.
// The waves' partial sums meet in LDS in wave order; with K split over
// workgroups each stores fp32 partials for the reduce kernel, so results do
// not depend on timing.
//
//   C[m, n] = sum_g sa[g, m] sw[n / 128, g] P_g[m, n]
//
// P_g over the 128 k of group g is one matrix instruction; the promotion to fp32
// is four multiply-adds a lane and free beside the loads.  One row of (4096,
// 7168), 29.4 MB: 7.0 .. 7.8 us as a kernel, of which about 2 are the launch and the
// first loads' latency; 33 rows of (576, 7168) with three row blocks 7.8 us, latency
// alone: a wave's 14 groups come in two rings of loads.
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include "block8.h"
#include "block8_device.h"
#include "launch.h"

namespace hq {

namespace {

template <int NB, int ST, bool ONCE>
__global__ void __launch_bounds__(512) b8_skinny(B8Args p) {
#if defined(__HIP_DEVICE_COMPILE__)
  extern __shared__ __attribute__((aligned(16))) f4_t red[];  // [waves][NB][64]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int c16 = lane & 15, kq = lane >> 4;
  const int N = p.N, K = p.K, G = p.G;
  const int m0 = blockIdx.z * 16;
  const int g0 = blockIdx.y * p.gps, g1 = min(G, g0 + p.gps);
  const int nblocks = N / 16;
  const int nb0 = blockIdx.x * NB;

  auto rsrc = [](const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
  };
  const int abytes = p.a_rows * K, sbytes = G * p.a_rows * 4;
  const auto ra = rsrc(p.a, abytes);
  const auto rs = rsrc(p.a_scale, sbytes);
  const auto rw = rsrc(p.w, (int64_t)N * K);
  const auto rws = rsrc(p.w_scale, (int64_t)((N + 127) / 128) * G * 4);
  // rows past M load zeros without touching memory (offset past the range)
  const int am = m0 + c16;
  const int aoff = am < p.M ? am * K + kq * 16 : (int)0x80000000u;
  const int soff = am < p.M ? am * 4 : (int)0x80000000u;
  int woff[NB], swoff[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int nb = min(nb0 + j, nblocks - 1);
    woff[j] = nb * G * 2048 + lane * 16;
    swoff[j] = (nb / 8) * G * 4;
  }

  u4_t wr[ST][NB][2], ar[ST][2];
  uint32_t sw[ST][NB], sa[ST];
  // Loads are issued without branches, so that the wait before each step's math
  // is for that step's loads alone; steps past the end take offsets past the
  // range, which read nothing.
  auto issue = [&](int slot, int g) {
    const int past = g < g1 ? 0 : (int)0x80000000u;
    g = min(g, g1 - 1);
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        wr[slot][j][h] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, (woff[j] + 1024 * h) | past, g * 2048, ONCE ? kReadOnce : 0));
#pragma unroll
    for (int h = 0; h < 2; ++h)
      ar[slot][h] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(ra, (aoff + 64 * h) | past, g * 128, 0));
    sa[slot] = __builtin_amdgcn_raw_buffer_load_b32(rs, soff | past, g * p.a_rows * 4, 0);
#pragma unroll
    for (int j = 0; j < NB; ++j) sw[slot][j] = __builtin_amdgcn_raw_buffer_load_b32(rws, swoff[j] | past, g * 4, 0);
  };
  f4_t acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = f4_t{0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int s = 0; s < ST; ++s) {
    issue(s, g0 + wave + s * waves);
    __builtin_amdgcn_sched_barrier(0);  // step by step, as the waits of the loop below count them
  }
  for (int g = g0 + wave; g < g1; g += ST * waves) {
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      // a step past the end holds zero codes and zero scales: it adds nothing
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const f4_t P = b8_mfma(cat8(wr[s][j][0], wr[s][j][1]), cat8(ar[s][0], ar[s][1]));
        const float f = __uint_as_float(sa[s]) * __uint_as_float(sw[s][j]);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[j][q] = fmaf(f, P[q], acc[j][q]);
      }
      issue(s, g + (s + ST) * waves);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) red[(wave * NB + j) * 64 + lane] = acc[j];
  __syncthreads();
  for (int e = tid; e < NB * 64; e += blockDim.x) {
    f4_t v = red[e];
    for (int w = 1; w < waves; ++w) {
      const f4_t u = red[w * NB * 64 + e];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += u[q];
    }
    const int l = e & 63, m = m0 + (l & 15), nb = nb0 + (e >> 6);
    if (m >= p.M || nb >= nblocks) continue;
    const int n = nb * 16 + 4 * (l >> 4);
    if (p.part) {
      *reinterpret_cast<f4_t*>(p.part + ((int64_t)blockIdx.y * p.M + m) * N + n) = v;
    } else {
      auto cv = [&](float x) -> uint32_t { return p.out_bf16 ? float_to_bf16_bits(x) : float_to_f16_bits(x); };
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (int64_t)m * N + n) =
          uint2{cv(v[0]) | (cv(v[1]) << 16), cv(v[2]) | (cv(v[3]) << 16)};
    }
  }
#endif
}

template <int NB, int ST>
hipError_t launch_t(const B8Skinny& c, const B8Args& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.N / 16 + NB - 1) / NB), (unsigned)c.split, (unsigned)((a.M + 15) / 16));
  const dim3 block(64 * c.waves);
  const size_t lds = (size_t)c.waves * NB * 1024;
  // A large weight that one row block reads goes past the caches, which it would
  // sweep (one row of (4096, 7168), 28 MiB: 8.3 us against 8.7 from memory, 7.65
  // against 7.7 from the last-level cache; (7168, 2048), 14 MiB: 5.4 against 5.7
  // and 4.9 against 4.5)
  if (grid.z == 1 && (int64_t)a.N * a.K >= (int64_t(24) << 20)) return launch_timed(b8_skinny<NB, ST, true>, grid, block, lds, s, a);
  return launch_timed(b8_skinny<NB, ST, false>, grid, block, lds, s, a);
}

}  // namespace

bool b8_skinny_ok(const B8Skinny& c) {
  return (c.nb == 1 || c.nb == 2) && c.waves >= 1 && c.waves <= 8 && c.split >= 1 && c.split <= 64;
}

int launch_b8_skinny(const B8Skinny& c, const B8Args& a, void* stream) {
  if (!b8_skinny_ok(c) || a.G < 1 || a.gps < 1 || a.M > 16 * 65535) return (int)hipErrorInvalidValue;
  if ((int64_t)(c.split - 1) * a.gps >= a.G || (int64_t)c.split * a.gps < a.G) return (int)hipErrorInvalidValue;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return c.nb == 1 ? (int)launch_t<1, 8>(c, a, s) : (int)launch_t<2, 4>(c, a, s);
}

}  // namespace hq
