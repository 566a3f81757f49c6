// The two grouped products of an experts' layer in MXFP4.
//
//   gate_up   h = a W1[e]^T, q(SiLU(h[:, :I]) * h[:, I:])   codes and powers of two out
//   down      o = a W2[e]^T, the slots' rows on their way into the sum over experts
//
// One 16 x 16 x 128 matrix instruction multiplies E2M1 codes with both sides' powers of
// two and adds into fp32, so that a step is its instructions, one 16-byte read of LDS
// per row block, and loads.
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "grouped_device.h"
#include "launch.h"
#include "mx4.h"
#include "mx4_device.h"
#include "qgemm_tiled_kernel.h"

namespace hq {

namespace {

// acc += W . A^T over 128 k: the weight is the first operand, so a lane (token l % 16)
// holds four consecutive columns.  sw, sa: the power of two of this lane's 32 k of its
// weight column and of its activation row, in the lowest byte.
__device__ __forceinline__ f4_t mx4_mfma(u4_t w, u4_t a, f4_t acc, uint32_t sw, uint32_t sa) {
#if defined(__HIP_DEVICE_COMPILE__)
  const i8_t wv = i8_t{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  const i8_t av = i8_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, acc, 4, 4, 0, (int)sw, 0, (int)sa);
#else
  return acc;
#endif
}

// A workgroup of 4 waves computes BM = 16 MB rows by 256 columns, each wave all the rows
// and 64 columns, so that every weight is read once a tile, straight to registers.
constexpr int kWaves = 4;
template <int MB, int ST>
struct Mx4Cfg {
  static constexpr int BM = 16 * MB;
  static constexpr int SEGW = MB > kWaves ? MB / kWaves : 1;  // 1 KiB loads of 16 rows a wave and step
  static constexpr int SROWS = BM < 64 ? 64 : BM;             // row scales per step (whole 64-lane loads)
  static constexpr int STAGE = BM * 64 + SROWS * 4;
  static constexpr int EPI = BM * 8 + kWaves * rows_lds(4);   // what down's epilogue keeps in the ring's place
  static constexpr int LDS = ST * STAGE > EPI ? ST * STAGE : EPI;
};

__device__ inline __amdgpu_buffer_rsrc_t mx4_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// One tile: rows m0 .. m0 + 16 MB - 1, column tile tn.
template <int MB, int ST, int MODE>
__device__ __forceinline__ void mx4_tile(const Mx4Args& p, uint8_t* lds, int m0, int64_t ex, int tn) {
#if defined(__HIP_DEVICE_COMPILE__)
  using C = Mx4Cfg<MB, ST>;
  constexpr int NB = 4;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kq = lane >> 4;
  const int N = p.N, G = p.G, kb = p.K / 2;

  // 16-column block of this wave's fragment j: gate_up takes two of gate and the two of up
  // that belong to the same 32 outputs, one block of the intermediate
  const int nblocks = N / 16;
  auto nblk = [&](int j) -> int {
    if constexpr (MODE == MX4_GATE_UP) return (j < 2 ? 0 : nblocks / 2) + tn * 8 + wave * 2 + (j & 1);
    return p.col0 / 16 + tn * 16 + wave * 4 + j;
  };

  const auto ra = mx4_rsrc(p.a, (int64_t)p.a_rows * kb);
  const auto rs = mx4_rsrc(p.a_scale, (int64_t)G * p.a_rows * 4);
  const auto rw = mx4_rsrc(p.w + ex * p.w_expert, p.w_expert);
  const auto rws = mx4_rsrc(p.w_scale + ex * p.s_expert, p.s_expert);

  auto row_of = [&](int r) -> int {
    if constexpr (MODE == MX4_GATE_UP) {
      const int id = p.sorted_ids[m0 + r];
      return id < p.n_slots ? id / p.topk : 0;
    }
    return m0 + r;
  };
  // activation rows: segment seg holds rows 16 seg .. 16 seg + 15, lane l writes physical
  // chunk l % 4 of row 16 seg + l / 4 (waves beyond the segments repeat one, so that every
  // wave has the same loads in flight)
  int aoff[C::SEGW], alds[C::SEGW];
#pragma unroll
  for (int s = 0; s < C::SEGW; ++s) {
    const int seg = (wave + kWaves * s) % MB;
    const int r = seg * 16 + (lane >> 2);
    aoff[s] = row_of(r) * kb + swz<4>(r, lane & 3) * 16;
    alds[s] = seg * 1024;
  }
  const int sseg = wave % (C::SROWS / 64);
  const int soff = row_of(min(sseg * 64 + lane, C::BM - 1)) * 4;
  int wfrag[NB];  // columns past N read the last block (their results are not stored)
#pragma unroll
  for (int j = 0; j < NB; ++j) wfrag[j] = __builtin_amdgcn_readfirstlane(min(nblk(j), nblocks - 1) * G);

  u4_t braw[ST][NB];
  uint32_t sraw[ST][NB];
  constexpr int LPS = C::SEGW + 1 + 2 * NB;
  static_assert(LPS * (ST - 2) < 64, "loads in flight exceed the wait counter");

  auto issue = [&](auto slot_c, int g) {
    constexpr int slot = decltype(slot_c)::value;
#pragma unroll
    for (int s = 0; s < C::SEGW; ++s)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(lds + slot * C::STAGE + alds[s]), 16, aoff[s], g * 64, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(lds + slot * C::STAGE + C::BM * 64 + sseg * 256), 4, soff,
                                             g * p.a_rows * 4, 0, 0);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      braw[slot][j] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, lane * 16, (wfrag[j] + g) * 1024, 0));
      sraw[slot][j] = __builtin_amdgcn_raw_buffer_load_b32(rws, lane & ~3, (wfrag[j] + g) * 64, 0);
    }
  };

  f4_t acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[mb][j] = f4_t{0.f, 0.f, 0.f, 0.f};

  auto compute = [&](auto slot_c) {
    constexpr int slot = decltype(slot_c)::value;
    const uint8_t* at = lds + slot * C::STAGE + c16 * 64 + swz<4>(c16, kq) * 16;
    const uint8_t* st = lds + slot * C::STAGE + C::BM * 64 + c16 * 4 + kq;
    uint32_t sw[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) sw[j] = sraw[slot][j] >> (8 * (lane & 3));
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const u4_t av = *reinterpret_cast<const u4_t*>(at + mb * 1024);
      const uint32_t sa = st[mb * 64];
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[mb][j] = mx4_mfma(braw[slot][j], av, acc[mb][j], sw[j], sa);
    }
  };

  auto gclamp = [&](int g) { return g < G ? g : G - 1; };
  auto step = [&](auto slot_c, int g) {
    constexpr int cur = decltype(slot_c)::value;
    using Ahead = std::integral_constant<int, (cur + ST - 1) % ST>;
    __builtin_amdgcn_sched_barrier(0);
    wait_vm_lds<LPS*(ST - 2)>();  // this wave's loads of step g have landed
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      pin(braw[cur][j]);
      pin(sraw[cur][j]);
    }
    issue(Ahead{}, gclamp(g + ST - 1));  // into the slot every wave finished with at step g - 1
    if (g < G) compute(slot_c);
  };
  [&]<int... I>(std::integer_sequence<int, I...>) {
    ((issue(std::integral_constant<int, I>{}, gclamp(I)), __builtin_amdgcn_sched_barrier(0)), ...);
  }(std::make_integer_sequence<int, ST - 1>{});
  for (int g = 0; g < G; g += ST) {
    [&]<int... I>(std::integer_sequence<int, I...>) {
      (step(std::integral_constant<int, I>{}, g + I), ...);
    }(std::make_integer_sequence<int, ST>{});
  }
  __builtin_amdgcn_s_waitcnt(0);  // no load into LDS may outlive its use here

  // ---- epilogue: lane (c16, kq) holds token c16 of each row block, columns
  // 4 kq .. 4 kq + 3 of each column block --------------------------------------
  if constexpr (MODE == MX4_GATE_UP) {
    // a wave's 32 outputs are one block of the intermediate
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      float v[8];
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = b8_silu_mul(acc[mb][i >> 2][i & 3], acc[mb][2 + (i >> 2)][i & 3]);
        top = max(top, b8_mag(v[i]));
      }
      top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
      top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
      const uint32_t s = mx4_scale(top);
      // columns 4 kq of the first 16 in the low half, of the second in the high half; lanes
      // of odd kq give the first to their neighbour and take the second: four bytes each
      const uint32_t word = mx4_word(v, s);
      const uint32_t give = kq & 1 ? word & 0xFFFFu : word >> 16;
      const uint32_t got = (uint32_t)__shfl_xor((int)give, 16, 64);
      const uint32_t codes = kq & 1 ? got | (word & 0xFFFF0000u) : (word & 0xFFFFu) | (got << 16);
      const int row = m0 + 16 * mb + c16;
      if (p.sorted_ids[row] >= p.n_slots) continue;
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + (int64_t)row * (N / 4) + tn * 64 + wave * 16 + (kq & 1) * 8 + (kq >> 1) * 4) = codes;
      if (kq == 0) p.out_scale[((int64_t)tn * p.out_rows + row) * 4 + wave] = (uint8_t)s;
    }
  } else {
    const int col = nblk(0) * 16;
    // the rows' slots and weights, into LDS first: a load per row block between
    // the stores would wait for each in turn
    int32_t* lid = reinterpret_cast<int32_t*>(lds);
    float* ltw = reinterpret_cast<float*>(lid + C::BM);
    __syncthreads();  // every wave is done with the stage ring
    load_slots(p, m0, C::BM, lid, ltw, tid, 64 * kWaves);
    __syncthreads();
    uint8_t* buf = lds + C::BM * 8 + wave * rows_lds(4);
    if (col < p.col0 + p.ncol) store_slot_rows<MB>(p, lid, ltw, buf, col, lane, acc);
  }
#endif
}

constexpr int mx4_stages(int MB) { return MB <= 4 ? 4 : 3; }

// An aligned block is run with as many row blocks (a power of two) as hold slots, so that
// the half-empty blocks that end each expert's segment cost what they hold.
template <int MB, int MODE>
__device__ __forceinline__ void mx4_tile_rows(const Mx4Args& p, uint8_t* lds, int m0, int64_t ex, int tn, int rows) {
  if constexpr (MB > 1) {
    if (rows <= 8 * MB) {
      mx4_tile_rows<MB / 2, MODE>(p, lds, m0, ex, tn, rows);
      return;
    }
  }
  mx4_tile<MB, mx4_stages(MB), MODE>(p, lds, m0, ex, tn);
}

template <int MB, int MODE>
__global__ void __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2))) mx4_grouped(Mx4Args p) {
#if defined(__HIP_DEVICE_COMPILE__)
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  int tm, tn;
  if (!grouped_place(p, 16 * MB, tm, tn)) return;
  const int m0 = tm * 16 * MB;
  const int64_t ex = p.block_expert[tm];
  if (ex < 0 || ex >= p.experts) {
    if constexpr (MODE == MX4_DOWN)
      zero_slot_rows(p, m0, 16 * MB, p.col0 + tn * 256, min(p.col0 + p.ncol, p.col0 + tn * 256 + 256), threadIdx.x, 256);
    return;
  }
  mx4_tile_rows<MB, MODE>(p, lds, m0, ex, tn, block_rows(p, m0, 16 * MB, threadIdx.x & 63));
#endif
}

// The down product with short K: the block's activation rows lie in LDS whole, and the
// workgroup walks its column tiles in one stream of weight loads, with no barrier and no
// refill between tiles.
constexpr int short_lds(int rows, int G) { return rows * (G * 68 + 8) + kWaves * rows_lds(4); }
constexpr int kShortLds = 72 * 1024;  // two workgroups a CU

template <int MB>
__device__ __forceinline__ void mx4_down_tiles(const Mx4Args& p, uint8_t* lds, int m0, int64_t ex, int c0, int c1) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int ROWS = 16 * MB, ST = 3;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kq = lane >> 4;
  const int G = p.G, kb = p.K / 2;
  const auto ra = mx4_rsrc(p.a, (int64_t)p.a_rows * kb);
  const auto rw = mx4_rsrc(p.w + ex * p.w_expert, p.w_expert);
  const auto rws = mx4_rsrc(p.w_scale + ex * p.s_expert, p.s_expert);
  // rows: group g at g * ROWS * 64, chunks swizzled; their powers of two [G][ROWS] behind
  uint32_t* ls = reinterpret_cast<uint32_t*>(lds + G * ROWS * 64);
  for (int s = wave; s < G * MB; s += kWaves) {
    const int g = s / MB, seg = s - g * MB;
    const int r = seg * 16 + (lane >> 2);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(lds + s * 1024), 16, (m0 + r) * kb + swz<4>(r, lane & 3) * 16, g * 64, 0, 0);
  }
  for (int i = tid; i < G * ROWS; i += 64 * kWaves) {
    const int g = i / ROWS;
    ls[i] = p.a_scale[(int64_t)g * p.a_rows + m0 + i - g * ROWS];
  }
  int32_t* lid = reinterpret_cast<int32_t*>(ls + G * ROWS);
  float* ltw = reinterpret_cast<float*>(lid + ROWS);
  load_slots(p, m0, ROWS, lid, ltw, tid, 64 * kWaves);
  uint8_t* buf = reinterpret_cast<uint8_t*>(ltw + ROWS) + wave * rows_lds(4);

  u4_t braw[ST][4];
  uint32_t sraw[ST][4];
  int col = c0 + 64 * wave, g = 0;  // of the step being multiplied
  int acol = col, ag = 0;           // of the step being loaded
  auto issue = [&](auto slot_c) {
    constexpr int slot = decltype(slot_c)::value;
    const int nb = min(acol, c1 - 64) / 16;  // past the end: loaded again, not stored
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int f = (nb + j) * G + ag;
      braw[slot][j] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, lane * 16, f * 1024, 0));
      sraw[slot][j] = __builtin_amdgcn_raw_buffer_load_b32(rws, lane & ~3, f * 64, 0);
    }
    if (++ag == G) {
      ag = 0;
      acol += 256;
    }
  };
  f4_t acc[MB][4];
  auto zero = [&] {
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[mb][j] = f4_t{0.f, 0.f, 0.f, 0.f};
  };
  zero();
  [&]<int... I>(std::integer_sequence<int, I...>) {
    (issue(std::integral_constant<int, I>{}), ...);
  }(std::make_integer_sequence<int, ST - 1>{});
  __builtin_amdgcn_s_waitcnt(0);  // this wave's loads into LDS have landed
  __syncthreads();
  auto step = [&](auto slot_c) {
    constexpr int slot = decltype(slot_c)::value;
    issue(std::integral_constant<int, (slot + ST - 1) % ST>{});
    __builtin_amdgcn_sched_barrier(0);
    uint32_t sw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) sw[j] = sraw[slot][j] >> (8 * (lane & 3));
    const uint8_t* at = lds + g * ROWS * 64 + c16 * 64 + swz<4>(c16, kq) * 16;
    const uint8_t* st = reinterpret_cast<const uint8_t*>(ls + g * ROWS + c16) + kq;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const u4_t av = *reinterpret_cast<const u4_t*>(at + mb * 1024);
      const uint32_t sa = st[mb * 64];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[mb][j] = mx4_mfma(braw[slot][j], av, acc[mb][j], sw[j], sa);
    }
    if (++g == G) {
      if (col < c1) store_slot_rows<MB>(p, lid, ltw, buf, col, lane, acc);
      zero();
      g = 0;
      col += 256;
    }
  };
  const int steps = (c1 - c0 + 255) / 256 * G;
  for (int s = 0; s < steps; s += ST) {
    [&]<int... I>(std::integer_sequence<int, I...>) {
      ((s + I < steps ? step(std::integral_constant<int, I>{}) : void()), ...);
    }(std::make_integer_sequence<int, ST>{});
  }
#endif
}

template <int MB>
__device__ __forceinline__ void mx4_down_rows(const Mx4Args& p, uint8_t* lds, int m0, int64_t ex, int c0, int c1, int rows) {
  if constexpr (MB > 1) {
    if (rows <= 8 * MB) {
      mx4_down_rows<MB / 2>(p, lds, m0, ex, c0, c1, rows);
      return;
    }
  }
  mx4_down_tiles<MB>(p, lds, m0, ex, c0, c1);
}

template <int MB>
__global__ void __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2))) mx4_down_short(Mx4Args p) {
#if defined(__HIP_DEVICE_COMPILE__)
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  int tm, tn;
  if (!grouped_place(p, 16 * MB, tm, tn)) return;
  const int m0 = tm * 16 * MB;
  const int64_t ex = p.block_expert[tm];
  const int c0 = p.col0 + tn * p.cols_wg, c1 = min(c0 + p.cols_wg, p.col0 + p.ncol);
  if (ex < 0 || ex >= p.experts) {
    zero_slot_rows(p, m0, 16 * MB, c0, c1, threadIdx.x, 256);
    return;
  }
  mx4_down_rows<MB>(p, lds, m0, ex, c0, c1, block_rows(p, m0, 16 * MB, threadIdx.x & 63));
#endif
}

template <int MB, int MODE>
hipError_t launch_tiles(const Mx4Args& a, dim3 grid, hipStream_t s) {
  // the largest ring of the row counts a block may run with
  constexpr int LOW = MB < 4 ? MB : 4;
  constexpr size_t lds = std::max<size_t>(Mx4Cfg<MB, mx4_stages(MB)>::LDS, Mx4Cfg<LOW, mx4_stages(LOW)>::LDS);
  const hipError_t e = allow_lds<mx4_grouped<MB, MODE>>(lds);
  return e != hipSuccess ? e : launch_timed(mx4_grouped<MB, MODE>, grid, dim3(64 * kWaves), lds, s, a);
}

template <int MB>
hipError_t launch_short(const Mx4Args& a, dim3 grid, hipStream_t s) {
  const hipError_t e = allow_lds<mx4_down_short<MB>>(kShortLds);
  return e != hipSuccess ? e : launch_timed(mx4_down_short<MB>, grid, dim3(64 * kWaves), (size_t)short_lds(16 * MB, a.G), s, a);
}

template <int MB>
hipError_t launch_block(int mode, bool whole, const Mx4Args& a, dim3 grid, hipStream_t s) {
  if (whole) return launch_short<MB>(a, grid, s);
  return mode == MX4_DOWN ? launch_tiles<MB, MX4_DOWN>(a, grid, s) : launch_tiles<MB, MX4_GATE_UP>(a, grid, s);
}

}  // namespace

int launch_mx4_grouped(int mode, int bm, const Mx4Args& a, int64_t blocks, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.G < 1 || a.N % (mode == MX4_GATE_UP ? 256 : 64) || blocks < 1) return (int)hipErrorInvalidValue;
  if (mode == MX4_DOWN && (a.ncol < 64 || a.ncol % 64 || a.col0 % 256 || a.col0 + a.ncol > a.N)) return (int)hipErrorInvalidValue;
  Mx4Args b = a;
  const bool whole = mode == MX4_DOWN && short_lds(bm, a.G) <= kShortLds;
  if (whole) {
    const int64_t tiles = (a.ncol + 255) / 256;
    const int64_t per = tiles * blocks >= 1536 ? 2 : 1;  // column tiles a workgroup walks
    b.cols_wg = (int)(256 * per);
    b.tiles_n = (int)((tiles + per - 1) / per);
  } else {
    b.tiles_n = (int)((mode == MX4_DOWN ? a.ncol : a.N) + 255) / 256;
  }
  if (blocks * b.tiles_n > INT32_MAX) return (int)hipErrorInvalidValue;
  const dim3 grid((unsigned)(blocks * b.tiles_n));
  switch (bm) {
    case 16: return (int)launch_block<1>(mode, whole, b, grid, s);
    case 64: return (int)launch_block<4>(mode, whole, b, grid, s);
    case 128: return (int)launch_block<8>(mode, whole, b, grid, s);
  }
  return (int)hipErrorInvalidValue;
}

}  // namespace hq
