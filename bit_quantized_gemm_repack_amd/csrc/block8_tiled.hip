// fp8 x fp8 GEMM with 128-block scales, many rows: dense, and the two grouped
// products of an experts' layer.
//
//   C[m, n] = sum_g sa[g, m] sw[n / 128, g] P_g[m, n]
//
// Each 16 x 16 x 128 matrix instruction forms P_g from zero; its four results
// per lane are one token's, so the promotion to the fp32 accumulator is four
// fused multiply-adds with one factor sa * sw.
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <type_traits>
#include <utility>

#include "block8.h"
#include "block8_device.h"
#include "launch.h"
#include "qgemm_tiled_kernel.h"

namespace hq {

namespace {

// A workgroup of WM x 4 waves computes BM = 16 MB WM rows by BN = 64 NB
// columns: wave (wm, wn) owns rows [16 MB wm, + 16 MB) and 16 NB columns.
template <int MB, int NB, int WM, int ST>
struct B8Cfg {
  static constexpr int WAVES = 4 * WM;
  static constexpr int THREADS = 64 * WAVES;
  static constexpr int BM = 16 * MB * WM;
  static constexpr int BN = 64 * NB;
  static constexpr int NSEG = BM / 8;  // 1 KiB loads of the activation tile per step
  static constexpr int SEGW = NSEG > WAVES ? NSEG / WAVES : 1;
  static constexpr int SROWS = BM < 64 ? 64 : BM;  // row scales per step (whole 64-lane loads)
  static constexpr int STAGE = BM * 128 + SROWS * 4;
  static constexpr int LDS = ST * STAGE > 4 * BM * 4 ? ST * STAGE : 4 * BM * 4;
};

template <int MB, int NB, int WM, int ST, int MODE>
__global__ void __launch_bounds__(256 * WM) __attribute__((amdgpu_waves_per_eu(2))) b8_tiled(B8Args p) {
#if defined(__HIP_DEVICE_COMPILE__)
  using C = B8Cfg<MB, NB, WM, ST>;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c16 = lane & 15, kq = lane >> 4;
  const int wn = wave & 3, wm = wave >> 2;
  const int N = p.N, K = p.K, G = p.G;

  int tm, tn;
  if constexpr (MODE == B8_DENSE) {
    // ids dealt round-robin to the 8 XCDs get consecutive logical tiles on
    // each; logical tiles run in groups of group_m row tiles, column by column
    const int nwg = gridDim.x;
    int lid = blockIdx.x;
    if ((nwg & 7) == 0) lid = (blockIdx.x & 7) * (nwg >> 3) + (blockIdx.x >> 3);
    const int per = p.group_m * p.tiles_n;
    const int grp = lid / per, first = grp * p.group_m;
    const int gsz = min(p.tiles_m - first, p.group_m);
    const int r = lid - grp * per;
    tm = first + r % gsz;
    tn = r / gsz;
  } else {
    tm = blockIdx.x / p.tiles_n;
    tn = blockIdx.x - tm * p.tiles_n;
  }
  const int m0 = tm * C::BM;
  const int split = MODE == B8_DENSE ? (int)blockIdx.y : 0;
  const int gb = split * p.gps;
  const int Gl = min(G - gb, p.gps);

  const uint8_t* wbytes = p.w;
  const float* wsc = p.w_scale;
  if constexpr (MODE != B8_DENSE) {
    if (m0 >= *p.num_padded) return;
    const int64_t ex = p.block_expert[tm];
    if (ex < 0) {
      // slots whose expert id is out of range: the down GEMM's rows are zero
      if constexpr (MODE == B8_DOWN) {
        for (int e = tid; e < C::BM * C::BN; e += C::THREADS) {
          const int id = p.sorted_ids[m0 + e / C::BN];
          const int n = tn * C::BN + e % C::BN;
          if (id < p.n_slots && n < N) p.rows16[(int64_t)id * N + n] = 0;
        }
      }
      return;
    }
    wbytes += ex * p.w_expert;
    wsc += ex * p.s_expert;
  }

  // 16-column block of this wave's fragment j.  gate_up: the wave's first
  // NB / 2 fragments are gate columns, the others the up columns of the same
  // outputs (N/2 is a multiple of 128, the tile a whole 128-block of outputs).
  const int nblocks = N / 16;
  auto nblk = [&](int j) -> int {
    if constexpr (MODE == B8_GATE_UP) {
      const int b = tn * (C::BN / 32) + wn * (NB / 2) + (j % (NB / 2));
      return j < NB / 2 ? b : nblocks / 2 + b;
    }
    return tn * (C::BN / 16) + wn * NB + j;
  };

  auto rsrc = [](const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
  };
  const auto ra = rsrc(p.a, (int64_t)p.a_rows * K);
  const auto rs = rsrc(p.a_scale, (int64_t)G * p.a_rows * 4);
  const auto rw = rsrc(wbytes, (int64_t)N * K);
  const auto rws = rsrc(wsc, (int64_t)((N + 127) / 128) * G * 4);

  auto row_of = [&](int r) -> int {
    if constexpr (MODE == B8_DENSE) return min(m0 + r, p.M - 1);
    if constexpr (MODE == B8_GATE_UP) {
      const int id = p.sorted_ids[m0 + r];
      return id < p.n_slots ? id / p.topk : 0;
    }
    return m0 + r;
  };
  // activation rows: segment seg holds rows 8 seg .. 8 seg + 7, lane l writes
  // physical chunk l % 8 of row 8 seg + l / 8 (waves beyond the segments
  // repeat one, so that every wave has the same loads in flight)
  int aoff[C::SEGW], alds[C::SEGW];
#pragma unroll
  for (int s = 0; s < C::SEGW; ++s) {
    const int seg = (wave + C::WAVES * s) % C::NSEG;
    const int r = seg * 8 + (lane >> 3);
    aoff[s] = row_of(r) * K + swz<8>(r, lane & 7) * 16;
    alds[s] = __builtin_amdgcn_readfirstlane(seg * 1024);
  }
  const int sseg = __builtin_amdgcn_readfirstlane(wave % (C::SROWS / 64));
  const int soff = row_of(min(sseg * 64 + lane, C::BM - 1)) * 4;
  // Weight fragments: lane offset 16 l, the fragment's place in a scalar
  // offset.  Columns past N read the last block (their results are not stored).
  const int woff = lane * 16;
  int wsc_off[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) wsc_off[j] = __builtin_amdgcn_readfirstlane(min(nblk(j), nblocks - 1) * G * 2048);
  constexpr int NSW = MODE == B8_GATE_UP ? 2 : 1;  // weight scales a wave needs per step
  int swoff[NSW];
#pragma unroll
  for (int u = 0; u < NSW; ++u)
    swoff[u] = __builtin_amdgcn_readfirstlane((min(nblk(u * (NB / 2)), nblocks - 1) * 16 / 128) * G * 4);

  u4_t braw[ST][NB][2];
  uint32_t sraw[ST][NSW];
  constexpr int LPS = C::SEGW + 1 + 2 * NB + NSW;
  static_assert(LPS * (ST - 2) < 64, "loads in flight exceed the wait counter");

  auto issue = [&](auto slot_c, int g) {
    constexpr int slot = decltype(slot_c)::value;
    const int gg = gb + g;
#pragma unroll
    for (int s = 0; s < C::SEGW; ++s)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(lds + slot * C::STAGE + alds[s]), 16, aoff[s], gg * 128, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(lds + slot * C::STAGE + C::BM * 128 + sseg * 256), 4, soff,
                                             gg * p.a_rows * 4, 0, 0);
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        braw[slot][j][h] =
            __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, woff + 1024 * h, wsc_off[j] + gg * 2048, 0));
#pragma unroll
    for (int u = 0; u < NSW; ++u) sraw[slot][u] = __builtin_amdgcn_raw_buffer_load_b32(rws, 0, swoff[u] + gg * 4, 0);
  };

  f4_t acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[mb][j] = f4_t{0.f, 0.f, 0.f, 0.f};

  // The step's MB x NB matrix instructions, row block by row block, as one
  // pipeline: the operand of the next row block is read while the current
  // one multiplies, and the four multiply-adds that promote a product follow
  // two instructions behind it, so that they issue in the shadow of the matrix
  // instruction then running (32 cycles against 16) instead of waiting for
  // their own.
  auto compute = [&](auto slot_c) {
    constexpr int slot = decltype(slot_c)::value;
    const uint8_t* at = lds + slot * C::STAGE + wm * (16 * MB) * 128 + c16 * 128;
    const float* st = reinterpret_cast<const float*>(lds + slot * C::STAGE + C::BM * 128) + wm * 16 * MB + c16;
    float sw[NSW];
#pragma unroll
    for (int u = 0; u < NSW; ++u) sw[u] = __uint_as_float(sraw[slot][u]);
    i8_t a[2];
    float sa[2];
    auto read = [&](int mb) {  // the row blocks start at multiples of 16: the swizzle sees c16 alone
      a[mb & 1] = cat8(*reinterpret_cast<const u4_t*>(at + mb * 2048 + swz<8>(c16, kq) * 16),
                       *reinterpret_cast<const u4_t*>(at + mb * 2048 + swz<8>(c16, 4 + kq) * 16));
      sa[mb & 1] = st[16 * mb];
    };
    constexpr int D = NB == 4 && MB > 1 ? 3 : (MB * NB > 2 ? 2 : 1);  // products in flight ahead of their promotion (fewer than NB, or both of two)
    f4_t P[D + 1];
    float f[2][NSW];
    auto promote = [&](int i) {
      const int mb = i / NB, j = i - mb * NB;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        acc[mb][j][q] = fmaf(f[mb & 1][NSW == 2 ? j / (NB / 2) : 0], P[i % (D + 1)][q], acc[mb][j][q]);
    };
    read(0);
#pragma unroll
    for (int i = 0; i < MB * NB; ++i) {
      const int mb = i / NB, j = i - mb * NB;
      if (j == 0 && mb + 1 < MB) read(mb + 1);
      P[i % (D + 1)] = b8_mfma(cat8(braw[slot][j][0], braw[slot][j][1]), a[mb & 1]);
      if (j == (NB > D ? D - 1 : 0)) {
#pragma unroll
        for (int u = 0; u < NSW; ++u) f[mb & 1][u] = sa[mb & 1] * sw[u];
      }
      if (i >= D) promote(i - D);
      __builtin_amdgcn_sched_barrier(0);  // keeps this order: left to itself the scheduler puts each product's promotion right behind it
    }
#pragma unroll
    for (int i = MB * NB - D; i < MB * NB; ++i) promote(i);
  };

  auto gclamp = [&](int g) { return g < Gl ? g : Gl - 1; };
  auto step = [&](auto slot_c, int g) {
    constexpr int cur = decltype(slot_c)::value;
    using Ahead = std::integral_constant<int, (cur + ST - 1) % ST>;
    __builtin_amdgcn_sched_barrier(0);
    wait_vm_lds<LPS*(ST - 2)>();  // this wave's loads of step g have landed
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) pin(braw[cur][j][h]);
#pragma unroll
    for (int u = 0; u < NSW; ++u) pin(sraw[cur][u]);
    issue(Ahead{}, gclamp(g + ST - 1));  // into the slot every wave finished with at step g - 1
    if (g < Gl) compute(slot_c);
  };
  [&]<int... I>(std::integer_sequence<int, I...>) {
    ((issue(std::integral_constant<int, I>{}, gclamp(I)), __builtin_amdgcn_sched_barrier(0)), ...);
  }(std::make_integer_sequence<int, ST - 1>{});
  for (int g = 0; g < Gl; g += ST) {
    [&]<int... I>(std::integer_sequence<int, I...>) {
      (step(std::integral_constant<int, I>{}, g + I), ...);
    }(std::make_integer_sequence<int, ST>{});
  }
  __builtin_amdgcn_s_waitcnt(0);  // no load into LDS may outlive its use here

  // ---- epilogue: lane (c16, kq) holds token c16 of each row block, columns
  // 4 kq .. 4 kq + 3 of each column block --------------------------------------
  const int mw = m0 + 16 * MB * wm;
  if constexpr (MODE == B8_GATE_UP) {
    // one tile row holds the 128 outputs of one scale block: SiLU(gate) * up,
    // its largest magnitude over the four column waves, the codes
    uint32_t* red = reinterpret_cast<uint32_t*>(lds);  // [4][BM]
    __syncthreads();                              // every wave is done with the stage ring
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      uint32_t top = 0u;
#pragma unroll
      for (int j = 0; j < NB / 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float v = b8_silu_mul(acc[mb][j][q], acc[mb][j + NB / 2][q]);
          acc[mb][j][q] = v;
          top = max(top, b8_mag(v));
        }
      top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
      top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
      if (kq == 0) red[wn * C::BM + 16 * MB * wm + 16 * mb + c16] = top;
    }
    __syncthreads();
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const int rl = 16 * MB * wm + 16 * mb + c16;
      const float s = b8_scale(max(max(red[rl], red[C::BM + rl]), max(red[2 * C::BM + rl], red[3 * C::BM + rl])));
      if (p.sorted_ids[m0 + rl] >= p.n_slots) continue;
      const int64_t row = m0 + rl;
      const B8Div d(s);
#pragma unroll
      for (int j = 0; j < NB / 2; ++j)
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + row * (N / 2) + nblk(j) * 16 + 4 * kq) =
            b8_codes(acc[mb][j][0], acc[mb][j][1], acc[mb][j][2], acc[mb][j][3], d);
      if (wn == 0 && kq == 0) p.out_scale[(int64_t)tn * p.out_rows + row] = s;
    }
  } else {
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const int m = mw + 16 * mb + c16;
      float f = 1.f;
      int64_t orow = m;
      if constexpr (MODE == B8_DENSE) {
        if (m >= p.M) continue;
      } else {
        const int id = p.sorted_ids[m];
        if (id >= p.n_slots) continue;
        f = p.topk_w[id];
        orow = id;
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int b = nblk(j);
        if (b >= nblocks) continue;
        const f4_t v = acc[mb][j];
        const int n = b * 16 + 4 * kq;
        if constexpr (MODE == B8_DENSE) {
          if (p.part) {
            *reinterpret_cast<f4_t*>(p.part + ((int64_t)split * p.M + orow) * N + n) = v;
            continue;
          }
        }
        const int bf16 = MODE == B8_DOWN ? 1 : p.out_bf16;
        uint16_t* o = (MODE == B8_DOWN ? p.rows16 : static_cast<uint16_t*>(p.out)) + orow * N + n;
        auto cv = [&](float x) -> uint32_t { return bf16 ? float_to_bf16_bits(x * f) : float_to_f16_bits(x * f); };
        *reinterpret_cast<uint2*>(o) = uint2{cv(v[0]) | (cv(v[1]) << 16), cv(v[2]) | (cv(v[3]) << 16)};
      }
    }
  }
#endif
}

template <int MB, int NB, int WM, int ST, int MODE>
hipError_t launch_t(const B8Args& a, dim3 grid, hipStream_t s) {
  using C = B8Cfg<MB, NB, WM, ST>;
  const hipError_t e = allow_lds<b8_tiled<MB, NB, WM, ST, MODE>>(C::LDS);
  if (e != hipSuccess) return e;
  return launch_timed(b8_tiled<MB, NB, WM, ST, MODE>, grid, dim3(C::THREADS), (size_t)C::LDS, s, a);
}

template <int MODE>
hipError_t dispatch(const B8Tile& t, const B8Args& a, dim3 grid, hipStream_t s) {
#define HQ_B8(bm_, bn_, st_, MB, NB, WM) \
  if (t.bm == bm_ && t.bn == bn_ && t.stages == st_) return launch_t<MB, NB, WM, st_, MODE>(a, grid, s);
  HQ_B8(16, 256, 3, 1, 4, 1)
  HQ_B8(32, 256, 3, 2, 4, 1)
  HQ_B8(64, 256, 2, 4, 4, 1)
  HQ_B8(64, 256, 3, 4, 4, 1)
  HQ_B8(128, 256, 2, 8, 4, 1)
  if constexpr (MODE == B8_DENSE) {
    HQ_B8(256, 256, 2, 8, 4, 2)
    HQ_B8(128, 128, 2, 8, 2, 1)
    HQ_B8(128, 128, 3, 8, 2, 1)
    HQ_B8(64, 128, 3, 4, 2, 1)
    HQ_B8(64, 128, 4, 4, 2, 1)
    HQ_B8(32, 128, 4, 2, 2, 1)
    HQ_B8(16, 128, 4, 1, 2, 1)
  }
#undef HQ_B8
  return hipErrorInvalidValue;
}

}  // namespace

bool b8_tile_ok(int mode, const B8Tile& t) {
  if (t.bn == 256) {
    if (t.bm == 16 || t.bm == 32) return t.stages == 3;
    if (t.bm == 64) return t.stages == 2 || t.stages == 3;
    return (t.bm == 128 || (t.bm == 256 && mode == B8_DENSE)) && t.stages == 2;
  }
  if (t.bn != 128 || mode != B8_DENSE) return false;
  if (t.bm == 128) return t.stages == 2 || t.stages == 3;
  if (t.bm == 64) return t.stages == 3 || t.stages == 4;
  return (t.bm == 16 || t.bm == 32) && t.stages == 4;
}

int launch_b8_tiled(int mode, const B8Tile& t, const B8Args& a, int64_t blocks, void* stream) {
  if (!b8_tile_ok(mode, t) || a.G < 1 || a.gps < 1) return (int)hipErrorInvalidValue;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  B8Args b = a;
  if (mode == B8_DENSE) {
    // every split holds at least one group and together they cover K
    if ((int64_t)(t.split - 1) * a.gps >= a.G || (int64_t)t.split * a.gps < a.G) return (int)hipErrorInvalidValue;
    return (int)dispatch<B8_DENSE>(t, b, dim3((unsigned)(a.tiles_m * a.tiles_n), (unsigned)t.split), s);
  }
  if (a.gps != a.G || a.N % (mode == B8_GATE_UP ? 256 : 16) || blocks < 1 || blocks * a.tiles_n > INT32_MAX)
    return (int)hipErrorInvalidValue;
  const dim3 grid((unsigned)(blocks * a.tiles_n));
  return mode == B8_GATE_UP ? (int)dispatch<B8_GATE_UP>(t, b, grid, s) : (int)dispatch<B8_DOWN>(t, b, grid, s);
}

}  // namespace hq
