// fp8 x fp8 GEMM with 128-block scales, many rows: dense, and the two grouped
// products of an experts' layer.
//
//   C[m, n] = sum_g sa[g, m] sw[n / 128, g] P_g[m, n]
//
// Each 16 x 16 x 128 matrix instruction forms P_g from zero; its four results
// per lane are one token's, so the promotion to the fp32 accumulator is four
// fused multiply-adds with one factor sa * sw.
//
// What bounds it: 4096 x 4096 x 7168 takes 104 .. 106 us, 2320 TFLOP/s (the library's
// product with one scale per tensor takes 83, the instruction alone would take
// 53): the operand reads from LDS beside the matrix and vector instructions, and
// the clock, which the same product of zeros keeps higher (88 us).  200 x 14336
// x 4096 takes 22.6 us, 30 with its weight from memory: every row tile reads the
// weight again; without its loads 17, without its products 21.  Up to 64
// rows an expert the grouped products read weights at 4.8 .. 5.3 TB/s.
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "block8.h"
#include "block8_device.h"
#include "grouped_device.h"
#include "launch.h"
#include "qgemm_tiled_kernel.h"

namespace hq {

namespace {

// One 128-k step of a wave's 16 MB rows by 16 NB columns as one pipeline: the
// operand of the next row block is read while the current one multiplies, and
// the four multiply-adds that promote a product follow up to three matrix
// instructions behind it, so that they issue in the shadow of the one then
// running (32 cycles against 16) instead of waiting for their own.
//   at, st  the step's activation rows and row scales in LDS, this lane's row
//           (c16) of the first row block
//   b, sw   weight operands and scales (NSW = 2: gate columns, up columns)
template <int MB, int NB, int NSW>
__device__ __forceinline__ void b8_step(const uint8_t* at, const float* st, int c16, int kq, const u4_t (&b)[NB][2],
                                        const float (&sw)[NSW], f4_t (&acc)[MB][NB]) {
#if defined(__HIP_DEVICE_COMPILE__)
  i8_t a[2];
  float sa[2];
  auto read = [&](int mb) {  // row blocks start at multiples of 16: the swizzle sees c16 alone
    a[mb & 1] = cat8(*reinterpret_cast<const u4_t*>(at + mb * 2048 + swz<8>(c16, kq) * 16),
                     *reinterpret_cast<const u4_t*>(at + mb * 2048 + swz<8>(c16, 4 + kq) * 16));
    sa[mb & 1] = st[16 * mb];
  };
  // products in flight ahead of their promotion (fewer than NB, or both of two)
  constexpr int D = NB == 4 && MB > 1 ? 3 : (MB * NB > 2 ? 2 : 1);
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
    P[i % (D + 1)] = b8_mfma(cat8(b[j][0], b[j][1]), a[mb & 1]);
    if (j == (NB > D ? D - 1 : 0)) {
#pragma unroll
      for (int u = 0; u < NSW; ++u) f[mb & 1][u] = sa[mb & 1] * sw[u];
    }
    if (i >= D) promote(i - D);
    // keeps this order: left to itself the scheduler puts each product's promotion right behind it
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int i = MB * NB - D; i < MB * NB; ++i) promote(i);
#endif
}

// The step of the gate_up GEMM, whose sums are quantised again: products through
// fp16 (b8_mfma_exact).  The two weight fragments are converted once, each row
// block as it comes; its promotion follows behind the next one's products.
template <int MB>
__device__ __forceinline__ void b8_step_exact(const uint8_t* at, const float* st, int c16, int kq, const u4_t (&b)[2][2],
                                              const float (&sw)[2], f4_t (&acc)[MB][2]) {
#if defined(__HIP_DEVICE_COMPILE__)
  u4_t a[2][2];
  float sa[2];
  auto read = [&](int mb) {
    a[mb & 1][0] = *reinterpret_cast<const u4_t*>(at + mb * 2048 + swz<8>(c16, kq) * 16);
    a[mb & 1][1] = *reinterpret_cast<const u4_t*>(at + mb * 2048 + swz<8>(c16, 4 + kq) * 16);
    sa[mb & 1] = st[16 * mb];
  };
  f4_t P[2][2];
  float f[2][2];
  auto promote = [&](int mb) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[mb][u][q] = fmaf(f[mb & 1][u], P[mb & 1][u][q], acc[mb][u][q]);
  };
  read(0);
  const B8Halves w[2] = {b8_halves(b[0][0], b[0][1]), b8_halves(b[1][0], b[1][1])};
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    if (mb + 1 < MB) read(mb + 1);
    const B8Halves v = b8_halves(a[mb & 1][0], a[mb & 1][1]);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      P[mb & 1][u] = f4_t{0.f, 0.f, 0.f, 0.f};
      f[mb & 1][u] = sa[mb & 1] * sw[u];
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        P[mb & 1][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[u].v[s], v.v[s], P[mb & 1][u], 0, 0, 0);
    if (mb) promote(mb - 1);
    __builtin_amdgcn_sched_barrier(0);
  }
  promote(MB - 1);
#endif
}

// A workgroup of WV waves computes BM = 16 MB rows by BN = 16 NB WV columns,
// each wave all the rows and 16 NB columns, so that every weight is read once a
// tile, straight to registers.
template <int MB, int NB, int ST, int WV = 4>
struct B8Cfg {
  static constexpr int WAVES = WV;
  static constexpr int THREADS = 64 * WAVES;
  static constexpr int BM = 16 * MB;
  static constexpr int BN = 16 * NB * WV;
  static constexpr int NSEG = BM / 8;  // 1 KiB loads of the activation tile per step
  static constexpr int SEGW = NSEG > WAVES ? NSEG / WAVES : 1;
  static constexpr int SROWS = BM < 64 ? 64 : BM;  // row scales per step (whole 64-lane loads)
  static constexpr int STAGE = BM * 128 + SROWS * 4;
  // the ring, or what the epilogues keep in its place
  static constexpr int EPI = std::max(BM * 16, WAVES * rows_lds(NB));
  static constexpr int LDS = ST * STAGE > EPI ? ST * STAGE : EPI;
};

// One tile: rows m0 .. m0 + C::BM - 1, column tile tn.
template <int MB, int NB, int ST, int MODE, int WV = 4, bool ONCE = false>
__device__ __forceinline__ void b8_tile(const B8Args& p, uint8_t* lds, int m0, int64_t ex, int tn) {
#if defined(__HIP_DEVICE_COMPILE__)
  using C = B8Cfg<MB, NB, ST, WV>;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c16 = lane & 15, kq = lane >> 4;
  const int wn = wave;
  const int N = p.N, K = p.K, G = p.G;

  const int split = MODE == B8_DENSE ? (int)blockIdx.y : 0;
  const int gb = split * p.gps;
  const int Gl = min(G - gb, p.gps);
  const uint8_t* wbytes = p.w + (MODE == B8_DENSE ? 0 : ex * p.w_expert);
  const float* wsc = p.w_scale + (MODE == B8_DENSE ? 0 : ex * p.s_expert);

  // 16-column block of this wave's fragment j.  gate_up: the wave's first
  // NB / 2 fragments are gate columns, the others the up columns of the same
  // outputs (N/2 is a multiple of 128, the tile a whole 128-block of outputs).
  const int nblocks = N / 16;
  auto nblk = [&](int j) -> int {
    if constexpr (MODE == B8_GATE_UP) {
      const int b = tn * (C::BN / 32) + wn * (NB / 2) + (j % (NB / 2));
      return j < NB / 2 ? b : nblocks / 2 + b;
    }
    return (MODE == B8_DOWN ? p.col0 / 16 : 0) + tn * (C::BN / 16) + wn * NB + j;
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
            __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, woff + 1024 * h, wsc_off[j] + gg * 2048, ONCE ? kReadOnce : 0));
#pragma unroll
    for (int u = 0; u < NSW; ++u) sraw[slot][u] = __builtin_amdgcn_raw_buffer_load_b32(rws, 0, swoff[u] + gg * 4, 0);
  };

  f4_t acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[mb][j] = f4_t{0.f, 0.f, 0.f, 0.f};

  auto compute = [&](auto slot_c) {
    constexpr int slot = decltype(slot_c)::value;
    float sw[NSW];
#pragma unroll
    for (int u = 0; u < NSW; ++u) sw[u] = __uint_as_float(sraw[slot][u]);
    const uint8_t* at = lds + slot * C::STAGE + c16 * 128;
    const float* st = reinterpret_cast<const float*>(lds + slot * C::STAGE + C::BM * 128) + c16;
    if constexpr (MODE == B8_GATE_UP && NB == 2)
      b8_step_exact<MB>(at, st, c16, kq, braw[slot], sw, acc);
    else
      b8_step<MB, NB, NSW>(at, st, c16, kq, braw[slot], sw, acc);
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
  if constexpr (MODE == B8_GATE_UP) {
    // one tile row holds the 128 outputs of one scale block: SiLU(gate) * up,
    // its largest magnitude over the column waves, the codes
    uint32_t* red = reinterpret_cast<uint32_t*>(lds);  // [WAVES][BM]
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
      if (kq == 0) red[wn * C::BM + 16 * mb + c16] = top;
    }
    __syncthreads();
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const int rl = 16 * mb + c16;
      uint32_t top = 0u;
#pragma unroll
      for (int w = 0; w < C::WAVES; ++w) top = max(top, red[w * C::BM + rl]);
      const float s = b8_scale(top);
      if (p.sorted_ids[m0 + rl] >= p.n_slots) continue;
      const int64_t row = m0 + rl;
      const B8Div d(s);
#pragma unroll
      for (int j = 0; j < NB / 2; ++j)
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + row * (N / 2) + nblk(j) * 16 + 4 * kq) =
            b8_codes(acc[mb][j][0], acc[mb][j][1], acc[mb][j][2], acc[mb][j][3], d);
      if (wn == 0 && kq == 0) p.out_scale[(int64_t)tn * p.out_rows + row] = s;
    }
  } else if constexpr (MODE == B8_DOWN) {
    const int col = nblk(0) * 16;
    // the rows' slots and weights, into LDS first: a load per row block between
    // the stores would wait for each in turn
    int32_t* lid = reinterpret_cast<int32_t*>(lds);
    float* ltw = reinterpret_cast<float*>(lid + C::BM);
    __syncthreads();  // every wave is done with the stage ring
    load_slots(p, m0, C::BM, lid, ltw, tid, C::THREADS);
    __syncthreads();
    if (col < p.col0 + p.ncol) store_slot_rows<MB>(p, lid, ltw, col, lane, acc);
  } else if (p.part) {
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const int m = m0 + 16 * mb + c16;
      if (m >= p.M) continue;
#pragma unroll
      for (int j = 0; j < NB; ++j)
        if (nblk(j) < nblocks)
          *reinterpret_cast<f4_t*>(p.part + ((int64_t)split * p.M + m) * N + nblk(j) * 16 + 4 * kq) = acc[mb][j];
    }
  } else {
    __syncthreads();  // every wave is done with the stage ring
    uint8_t* buf = lds + wave * rows_lds(NB);
    const int col = nblk(0) * 16, cols = min(16 * NB, N - col);
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const int m = m0 + 16 * mb + c16;
      char* o = reinterpret_cast<char*>(static_cast<uint16_t*>(p.out) + (int64_t)m * N + col);
      rows16_out<NB>(
          buf, lane,
          [&](int j) {
            auto cv = [&](float x) -> uint32_t { return p.out_bf16 ? float_to_bf16_bits(x) : float_to_f16_bits(x); };
            const f4_t v = acc[mb][j];
            return uint2{cv(v[0]) | (cv(v[1]) << 16), cv(v[2]) | (cv(v[3]) << 16)};
          },
          [&](int byte, uint4 v) {
            if (m < p.M && byte < 2 * cols) *reinterpret_cast<uint4*>(o + byte) = v;
          });
    }
  }
#endif
}

template <int MB, int NB, int ST>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) b8_dense(B8Args p) {
#if defined(__HIP_DEVICE_COMPILE__)
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  // logical tiles run in groups of group_m row tiles, column by column
  const int lid = xcd_order(blockIdx.x, gridDim.x);
  const int per = p.group_m * p.tiles_n;
  const int grp = lid / per, first = grp * p.group_m;
  const int gsz = min(p.tiles_m - first, p.group_m);
  const int r = lid - grp * per;
  b8_tile<MB, NB, ST, B8_DENSE>(p, lds, (first + r % gsz) * B8Cfg<MB, NB, ST>::BM, 0, r / gsz);
#endif
}

// gate_up through fp16 (EXACT) takes 8 waves of 16 gate and 16 up columns, one
// workgroup a CU; otherwise 4 waves of twice as many, as the down GEMM.
constexpr int b8_grouped_waves(bool exact) { return exact ? 8 : 4; }
constexpr int b8_grouped_stages(int MB) { return MB <= 4 ? 3 : 2; }

// A grouped tile of up to 16 MB rows: an aligned block is run with as many row
// blocks (a power of two) as hold slots, so that the half-empty blocks that end
// each expert's segment cost what they hold.
template <int MB, int MODE, bool EXACT, bool ONCE>
__device__ __forceinline__ void b8_grouped_tile(const B8Args& p, uint8_t* lds, int m0, int64_t ex, int tn, int rows) {
  if constexpr (MB > 1) {
    if (rows <= 8 * MB) {
      b8_grouped_tile<MB / 2, MODE, EXACT, ONCE>(p, lds, m0, ex, tn, rows);
      return;
    }
  }
  b8_tile<MB, EXACT ? 2 : 4, b8_grouped_stages(MB), MODE, b8_grouped_waves(EXACT), ONCE>(p, lds, m0, ex, tn);
}

template <int MB, int MODE, bool EXACT, bool ONCE>
__global__ void __launch_bounds__(64 * b8_grouped_waves(EXACT)) __attribute__((amdgpu_waves_per_eu(2))) b8_grouped(B8Args p) {
#if defined(__HIP_DEVICE_COMPILE__)
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  int tm, tn;
  if (!grouped_place(p, 16 * MB, tm, tn)) return;
  const int m0 = tm * 16 * MB;
  const int64_t ex = p.block_expert[tm];
  if (ex < 0 || ex >= p.experts) {
    if constexpr (MODE == B8_DOWN)
      zero_slot_rows(p, m0, 16 * MB, p.col0 + tn * 256, min(p.col0 + p.ncol, p.col0 + tn * 256 + 256), threadIdx.x, 256);
    return;
  }
  b8_grouped_tile<MB, MODE, EXACT, ONCE>(p, lds, m0, ex, tn, block_rows(p, m0, 16 * MB, threadIdx.x & 63));
#endif
}

// The down GEMM with short K: the block's activation rows lie in LDS whole, and
// the workgroup walks its column tiles in one stream of weight loads, with no
// barrier and no refill between tiles (with two or four groups of K per tile
// the loads' latency at each tile's start would cost as much as its math).
// 256 experts, top 8, H = 7168, I = 256: 509 tokens 105 us (444 MB of weights and
// 58 of rows, 4.8 TB/s), 4096 tokens two windows of 118 us (5 TB/s).
template <int MB>
__device__ __forceinline__ void b8_down_tiles(const B8Args& p, uint8_t* lds, int m0, int64_t ex, int c0, int c1) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kq = lane >> 4;
  const int K = p.K, G = p.G;
  constexpr int ROWS = 16 * MB;
  auto rsrc = [](const void* base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
  };
  const auto ra = rsrc(p.a, (int64_t)p.a_rows * K);
  const auto rw = rsrc(p.w + ex * p.w_expert, p.w_expert);
  const auto rws = rsrc(p.w_scale + ex * p.s_expert, p.s_expert * 4);
  // rows: group g at g * ROWS * 128, chunks swizzled; scales [G][ROWS] behind
  float* ls = reinterpret_cast<float*>(lds + G * ROWS * 128);
  for (int s = wave; s < G * ROWS / 8; s += 4) {
    const int g = s / (ROWS / 8), seg = s - g * (ROWS / 8);
    const int r = seg * 8 + (lane >> 3);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(lds + s * 1024), 16, (m0 + r) * K + swz<8>(r, lane & 7) * 16,
                                             g * 128, 0, 0);
  }
  for (int i = tid; i < G * ROWS; i += 256) {
    const int g = i / ROWS;
    ls[i] = p.a_scale[(int64_t)g * p.a_rows + m0 + i - g * ROWS];
  }
  int32_t* lid = reinterpret_cast<int32_t*>(ls + G * ROWS);
  float* ltw = reinterpret_cast<float*>(lid + ROWS);
  load_slots(p, m0, ROWS, lid, ltw, tid, 256);

  u4_t braw[2][4][2];
  float sw[2][1];
  int col = c0 + 64 * wave, g = 0;      // of the step being multiplied
  int acol = col, ag = 0;               // of the step being loaded
  auto issue = [&](auto slot_c) {
    constexpr int slot = decltype(slot_c)::value;
    const int cc = min(acol, c1 - 64);  // past the end: loaded again, not stored
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        braw[slot][j][h] = __builtin_bit_cast(
            u4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, lane * 16 + 1024 * h, ((cc / 16 + j) * G + ag) * 2048, 0));
    sw[slot][0] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rws, 0, ((cc / 128) * G + ag) * 4, 0));
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
  issue(std::integral_constant<int, 0>{});
  __builtin_amdgcn_s_waitcnt(0);  // this wave's loads into LDS have landed
  __syncthreads();
  auto step = [&](auto slot_c) {
    constexpr int slot = decltype(slot_c)::value;
    issue(std::integral_constant<int, slot ^ 1>{});
    __builtin_amdgcn_sched_barrier(0);
    b8_step<MB, 4, 1>(lds + g * ROWS * 128 + c16 * 128, ls + g * ROWS + c16, c16, kq, braw[slot], sw[slot], acc);
    if (++g == G) {
      if (col < c1) store_slot_rows<MB>(p, lid, ltw, col, lane, acc);
      zero();
      g = 0;
      col += 256;
    }
  };
  const int steps = (c1 - c0 + 255) / 256 * G;
  for (int s = 0; s < steps; s += 2) {
    step(std::integral_constant<int, 0>{});
    if (s + 1 < steps) step(std::integral_constant<int, 1>{});
  }
#endif
}

template <int MB>
__device__ __forceinline__ void b8_down_dispatch(const B8Args& p, uint8_t* lds, int m0, int64_t ex, int c0, int c1, int rows) {
  if constexpr (MB > 1) {
    if (rows <= 8 * MB) {
      b8_down_dispatch<MB / 2>(p, lds, m0, ex, c0, c1, rows);
      return;
    }
  }
  b8_down_tiles<MB>(p, lds, m0, ex, c0, c1);
}

template <int MB>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) b8_down_short(B8Args p) {
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
  b8_down_dispatch<MB>(p, lds, m0, ex, c0, c1, block_rows(p, m0, 16 * MB, threadIdx.x & 63));
#endif
}

// y[t][col0 + c] = RNE(sum over the token's topk slots of row * scale), in slot
// order; eight columns a thread, the rows as store_slot_rows leaves them.  Bound by
// reading the rows: a window of 4096 tokens, 235 MB, 43 us, 6.1 TB/s with its output.
// The rows are done with once read: loads that do not keep them leave the cache to
// the next window's (a layer of 4096 tokens 648 us against 661).
template <bool WIDE>
__global__ void __launch_bounds__(256) b8_combine_kernel(const u4_t* __restrict__ rows, const u2_t* __restrict__ low, const float* __restrict__ scale,
                                                         int topk, int n, int col0, int ncol, int64_t elems,
                                                         uint4* __restrict__ y, int out_bf16) {
  const int ncol8 = ncol / 8, strips = ncol / 64;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < elems; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / ncol8;
    const int c = (int)(i - t * ncol8);
    float v[8] = {};
    for (int j = 0; j < topk; ++j) {
      const u4_t w = __builtin_nontemporal_load(rows + (t * topk + j) * ncol8 + c);
      const float f = scale[(t * topk + j) * strips + c / 8];
      if constexpr (WIDE) {
        const u2_t l = __builtin_nontemporal_load(low + (t * topk + j) * ncol8 + c);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t hi = q & 1 ? w[q >> 1] & 0xFFFF0000u : w[q >> 1] << 16;
          v[q] = fmaf(__uint_as_float(hi | ((l[q >> 2] >> (8 * (q & 3))) & 0xFFu) << 8), f, v[q]);
        }
        continue;
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = fmaf(f16_bits_to_float((w[q >> 1] >> (16 * (q & 1))) & 0xFFFFu), f, v[q]);
    }
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      o[q] = out_bf16 ? (uint32_t)float_to_bf16_bits(v[2 * q]) | ((uint32_t)float_to_bf16_bits(v[2 * q + 1]) << 16)
                      : (uint32_t)float_to_f16_bits(v[2 * q]) | ((uint32_t)float_to_f16_bits(v[2 * q + 1]) << 16);
    y[t * (n / 8) + col0 / 8 + c] = uint4{o[0], o[1], o[2], o[3]};
  }
}

template <int MB, int NB, int ST>
hipError_t launch_dense(const B8Args& a, dim3 grid, hipStream_t s) {
  using C = B8Cfg<MB, NB, ST>;
  const hipError_t e = allow_lds<b8_dense<MB, NB, ST>>(C::LDS);
  if (e != hipSuccess) return e;
  return launch_timed(b8_dense<MB, NB, ST>, grid, dim3(C::THREADS), (size_t)C::LDS, s, a);
}

hipError_t dispatch_dense(const B8Tile& t, const B8Args& a, dim3 grid, hipStream_t s) {
#define HQ_B8(bm_, bn_, st_, MB, NB) \
  if (t.bm == bm_ && t.bn == bn_ && t.stages == st_) return launch_dense<MB, NB, st_>(a, grid, s);
  HQ_B8(128, 256, 2, 8, 4)
  HQ_B8(128, 128, 2, 8, 2)
  HQ_B8(64, 128, 3, 4, 2)
  HQ_B8(32, 128, 4, 2, 2)
  HQ_B8(16, 128, 4, 1, 2)
#undef HQ_B8
  return hipErrorInvalidValue;
}

template <int MB, int MODE, bool EXACT, bool ONCE = false>
hipError_t launch_grouped_k(const B8Args& a, dim3 grid, hipStream_t s) {
  // the largest ring of the row counts a block may run with
  constexpr int LOW = MB < 4 ? MB : 4, NB = EXACT ? 2 : 4, WV = b8_grouped_waves(EXACT);
  constexpr size_t lds = std::max<size_t>(B8Cfg<MB, NB, b8_grouped_stages(MB), WV>::LDS, B8Cfg<LOW, NB, b8_grouped_stages(LOW), WV>::LDS);
  const hipError_t e = allow_lds<b8_grouped<MB, MODE, EXACT, ONCE>>(lds);
  return e != hipSuccess ? e : launch_timed(b8_grouped<MB, MODE, EXACT, ONCE>, grid, dim3(64 * WV), lds, s, a);
}

template <int MB>
hipError_t launch_grouped(int mode, const B8Args& a, dim3 grid, hipStream_t s) {
  if (mode == B8_DOWN) return launch_grouped_k<MB, B8_DOWN, false>(a, grid, s);
  // The sums of gate_up are quantised again, where what the fp8 instruction
  // drops decides codes (b8_mfma_exact).  With up to 64 rows a block the
  // weights' loads bound both forms (256 experts, top 8, H = 7168, I = 256: 509
  // tokens 172 us through fp16 and 170 through fp8, 1024 208 and 194); with 128
  // fp16 has half the rate (4096 tokens 381 and 277), for what an output of
  // bf16, itself off by 1.7e-3, shows as 2.3e-3 at most, and one of fp16 as
  // five times its rounding.
  if constexpr (MB == 8)
    if (a.out_bf16) return launch_grouped_k<MB, B8_GATE_UP, false>(a, grid, s);
  // Weights that one block reads go past the caches (509 tokens of 256 experts
  // 161 us against 179); where blocks share an expert they stay (700 tokens of 16
  // experts in 16-row blocks 38 us, past the caches 59).
  if constexpr (MB <= 4)
    if (a.once) return launch_grouped_k<MB, B8_GATE_UP, true, true>(a, grid, s);
  return launch_grouped_k<MB, B8_GATE_UP, true>(a, grid, s);
}

constexpr int kShortLds = 63 * 1024;  // two workgroups a CU

template <int MB>
hipError_t launch_short(const B8Args& a, dim3 grid, hipStream_t s) {
  const hipError_t e = allow_lds<b8_down_short<MB>>(kShortLds);
  return e != hipSuccess ? e : launch_timed(b8_down_short<MB>, grid, dim3(256), (size_t)(16 * MB * (a.G * 132 + 8)), s, a);
}

}  // namespace

bool b8_tile_ok(const B8Tile& t) {
  if (t.stages != b8_stages(t.bm)) return false;
  if (t.bn == 256) return t.bm == 128;
  return t.bn == 128 && (t.bm == 16 || t.bm == 32 || t.bm == 64 || t.bm == 128);
}

int launch_b8_dense(const B8Tile& t, const B8Args& a, void* stream) {
  if (!b8_tile_ok(t) || a.G < 1 || a.gps < 1) return (int)hipErrorInvalidValue;
  // every split holds at least one group and together they cover K
  if ((int64_t)(t.split - 1) * a.gps >= a.G || (int64_t)t.split * a.gps < a.G) return (int)hipErrorInvalidValue;
  return (int)dispatch_dense(t, a, dim3((unsigned)(a.tiles_m * a.tiles_n), (unsigned)t.split), static_cast<hipStream_t>(stream));
}

int launch_b8_grouped(int mode, int bm, const B8Args& a, int64_t blocks, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.G < 1 || a.gps != a.G || a.N % (mode == B8_GATE_UP ? 256 : 64) || blocks < 1) return (int)hipErrorInvalidValue;
  if (mode == B8_DOWN && (a.ncol < 64 || a.ncol % 64 || a.col0 % 64 || a.col0 + a.ncol > a.N)) return (int)hipErrorInvalidValue;
  B8Args b = a;
  const bool whole = mode == B8_DOWN && bm * (a.G * 132 + 8) <= kShortLds;
  if (whole) {
    // column tiles a workgroup walks: two where there are plenty (they share
    // the rows' staging; more leave the last workgroups a long tail).  256
    // experts, H = 7168, I = 256, by 1 / 2 / 4 / 7 / 14 tiles: 100 tokens 78.1 /
    // 77.8 / 79.7 / 86.5 / 85.9 us, 509 122 / 118 / 121 / 127 / 134, 4096 340 /
    // 323 / 347 / 364 / 399; 64 experts of H = 2048, 1000 tokens 27.2 / 28.4 / 33.2.
    const int64_t tiles = (a.ncol + 255) / 256;
    const int64_t per = tiles * blocks >= 1536 ? 2 : 1;
    b.cols_wg = (int)(256 * per);
    b.tiles_n = (int)((tiles + per - 1) / per);
  } else {
    b.tiles_n = (int)((mode == B8_DOWN ? a.ncol : a.N) + 255) / 256;
  }
  if (blocks * b.tiles_n > INT32_MAX) return (int)hipErrorInvalidValue;
  const dim3 grid((unsigned)(blocks * b.tiles_n));
  switch (bm) {
    case 16: return whole ? (int)launch_short<1>(b, grid, s) : (int)launch_grouped<1>(mode, b, grid, s);
    case 64: return whole ? (int)launch_short<4>(b, grid, s) : (int)launch_grouped<4>(mode, b, grid, s);
    case 128: return whole ? (int)launch_short<8>(b, grid, s) : (int)launch_grouped<8>(mode, b, grid, s);
  }
  return (int)hipErrorInvalidValue;
}

int launch_b8_combine(const B8Args& a, int64_t t, void* stream, const uint8_t* rows8) {
  const int64_t elems = t * a.ncol / 8;
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((elems + 255) / 256, 16384));
  auto go = [&](auto kernel) {
    return (int)launch_timed(kernel, dim3((unsigned)blocks), dim3(256), 0, static_cast<hipStream_t>(stream),
                             reinterpret_cast<const u4_t*>(a.rows16), reinterpret_cast<const u2_t*>(rows8), a.row_scale, a.topk, a.N, a.col0, a.ncol, elems, static_cast<uint4*>(a.out), a.out_bf16);
  };
  return rows8 ? go(b8_combine_kernel<true>) : go(b8_combine_kernel<false>);
}

}  // namespace hq
