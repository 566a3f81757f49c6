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
#include "mx4_product.h"
#include "qgemm_tiled_kernel.h"

namespace hq {

namespace {

// A workgroup of four waves computes BM = 16 MB rows by 256 columns: each wave the rows by a
// strip of 64 columns, whose weights go straight to registers.  A step covers Q groups of 128
// k: with two, an activation row is a whole 128-byte line.  (Blocks of 256 rows by eight waves
// read an expert's weights less often, but wait more for their rows: 4096 tokens of 256 experts
// gate_up 196 us against 160.)
constexpr int kWaves = 4;
template <int MB, int ST, int Q>
struct Mx4Cfg {
  static constexpr int BM = 16 * MB;
  static constexpr int CHUNKS = 4 * Q;                                    // 16-byte chunks of a row
  static constexpr int SEG_ROWS = 64 / CHUNKS;                            // rows of a 1 KiB load
  static constexpr int SEGS = BM / SEG_ROWS;
  static constexpr int SEGW = SEGS > kWaves ? SEGS / kWaves : 1;            // such loads a wave
  static constexpr int SROWS = BM < 64 ? 64 : BM;                         // row scales a group (whole 64-lane loads)
  static constexpr int SCALES = BM * 64 * Q;                              // where they lie in a stage
  static constexpr int STAGE = SCALES + Q * SROWS * 4;
  static constexpr int LDS = ST * STAGE;                                  // (more than the slots of down's epilogue)
};

__device__ inline __amdgpu_buffer_rsrc_t mx4_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// One tile: rows m0 .. m0 + 16 MB - 1, column tile tn.
template <int MB, int ST, int Q, int MODE, int AUX>
__device__ __forceinline__ void mx4_tile(const Mx4Args& p, uint8_t* lds, int m0, int64_t ex, int tn) {
#if defined(__HIP_DEVICE_COMPILE__)
  using C = Mx4Cfg<MB, ST, Q>;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kq = lane >> 4;
  const int N = p.N, G = p.G, kb = p.K / 2, steps = G / Q;
  const int strip = (MODE == MX4_DOWN ? p.col0 / 64 : 0) + tn * 4 + wave;
  const int first = __builtin_amdgcn_readfirstlane(min(strip, N / 64 - 1) * steps * Q * kMx4GroupBytes);  // past N: loaded again, not stored

  const auto ra = mx4_rsrc(p.a, (int64_t)p.a_rows * kb);
  const auto rs = mx4_rsrc(p.a_scale, (int64_t)G * p.a_rows * 4);
  const auto rw = mx4_rsrc(p.w + ex * p.w_expert, p.w_expert);

  auto row_of = [&](int r) -> int {
    if constexpr (MODE == MX4_GATE_UP) {
      const int id = p.sorted_ids[m0 + r];
      return id < p.n_slots ? id / p.topk : 0;
    }
    return m0 + r;
  };
  // activation rows: lane l of segment seg writes physical chunk l % CHUNKS of row
  // SEG_ROWS seg + l / CHUNKS (waves beyond the segments repeat one, so that every wave has
  // the same loads in flight)
  int aoff[C::SEGW], alds[C::SEGW];
#pragma unroll
  for (int s = 0; s < C::SEGW; ++s) {
    const int seg = (wave + kWaves * s) % C::SEGS;
    const int r = seg * C::SEG_ROWS + lane / C::CHUNKS;
    aoff[s] = row_of(r) * kb + swz<C::CHUNKS>(r, lane % C::CHUNKS) * 16;
    alds[s] = seg * 1024;
  }
  constexpr int HALVES = C::SROWS / 64;
  const int sgroup = wave / HALVES % Q, shalf = wave % HALVES;
  const int soff = row_of(min(shalf * 64 + lane, C::BM - 1)) * 4;
  const int slds = C::SCALES + sgroup * C::SROWS * 4 + shalf * 256;

  u4_t braw[ST][Q][4];
  Mx4Scales<Q> sraw[ST];
  constexpr int LPS = C::SEGW + 1 + 4 * Q + 1;
  static_assert(LPS * (ST - 2) < 64, "loads in flight exceed the wait counter");

  auto issue = [&](auto slot_c, int s) {
    constexpr int slot = decltype(slot_c)::value;
#pragma unroll
    for (int i = 0; i < C::SEGW; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(lds + slot * C::STAGE + alds[i]), 16, aoff[i], s * 64 * Q, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(lds + slot * C::STAGE + slds), 4, soff, (s * Q + sgroup) * p.a_rows * 4, 0, 0);
#pragma unroll
    for (int u = 0; u < Q; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        braw[slot][u][j] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, lane * 16 + j * 1024, first + s * Q * kMx4GroupBytes + u * 4096, AUX));
    sraw[slot].template load<AUX>(rw, lane, first + s * Q * kMx4GroupBytes);
  };

  f4_t acc[MB][4];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[mb][j] = f4_t{0.f, 0.f, 0.f, 0.f};

  auto compute = [&](auto slot_c) {
    constexpr int slot = decltype(slot_c)::value;
    const uint8_t* at = lds + slot * C::STAGE + c16 * 64 * Q;
    const uint8_t* st = lds + slot * C::STAGE + C::SCALES + c16 * 4 + kq;
#pragma unroll
    for (int u = 0; u < Q; ++u)
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
        mx4_strip(braw[slot][u], *reinterpret_cast<const u4_t*>(at + mb * 1024 * Q + swz<C::CHUNKS>(c16, 4 * u + kq) * 16), acc[mb],
                  sraw[slot].v[u], st[u * C::SROWS * 4 + mb * 64]);
  };

  auto sclamp = [&](int s) { return s < steps ? s : steps - 1; };
  auto step = [&](auto slot_c, int s) {
    constexpr int cur = decltype(slot_c)::value;
    using Ahead = std::integral_constant<int, (cur + ST - 1) % ST>;
    __builtin_amdgcn_sched_barrier(0);
    wait_vm_lds<LPS*(ST - 2)>();  // this wave's loads of step s have landed
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < Q; ++u) {
#pragma unroll
      for (int j = 0; j < 4; ++j) pin(braw[cur][u][j]);
      pin(sraw[cur].v[u]);
    }
    issue(Ahead{}, sclamp(s + ST - 1));  // into the slot every wave finished with at step s - 1
    if (s < steps) compute(slot_c);
  };
  [&]<int... I>(std::integer_sequence<int, I...>) {
    ((issue(std::integral_constant<int, I>{}, sclamp(I)), __builtin_amdgcn_sched_barrier(0)), ...);
  }(std::make_integer_sequence<int, ST - 1>{});
  for (int s = 0; s < steps; s += ST) {
    [&]<int... I>(std::integer_sequence<int, I...>) {
      (step(std::integral_constant<int, I>{}, s + I), ...);
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
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = b8_silu_mul(acc[mb][i >> 2][i & 3], acc[mb][2 + (i >> 2)][i & 3]);
      uint32_t s;
      const uint32_t codes = mx4_block_codes(v, kq, s);
      const int row = m0 + 16 * mb + c16;
      if (p.sorted_ids[row] >= p.n_slots) continue;
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + (int64_t)row * (N / 4) + tn * 64 + wave * 16 + (kq & 1) * 8 + (kq >> 1) * 4) = codes;
      if (kq == 0) p.out_scale[((int64_t)tn * p.out_rows + row) * 4 + wave] = (uint8_t)s;
    }
  } else {
    const int col = strip * 64;
    // the rows' slots and weights, into LDS first: a load per row block between
    // the stores would wait for each in turn
    int32_t* lid = reinterpret_cast<int32_t*>(lds);
    float* ltw = reinterpret_cast<float*>(lid + C::BM);
    __syncthreads();  // every wave is done with the stage ring
    load_slots(p, m0, C::BM, lid, ltw, tid, 64 * kWaves);
    __syncthreads();
    if (col >= p.col0 + p.ncol) return;
    if (p.rows8)
      store_slot_rows24<MB>(p, lid, ltw, col, lane, acc);
    else
      store_slot_rows<MB>(p, lid, ltw, col, lane, acc);
  }
#endif
}

constexpr int mx4_stages(int MB) { return MB <= 4 ? 3 : 2; }

// An aligned block is run with as many row blocks (a power of two) as hold slots, so that
// the half-empty blocks that end each expert's segment cost what they hold.
template <int MB, int Q, int MODE, int AUX>
__device__ __forceinline__ void mx4_tile_rows(const Mx4Args& p, uint8_t* lds, int m0, int64_t ex, int tn, int rows) {
  if constexpr (MB > 1) {
    if (rows <= 8 * MB) {
      mx4_tile_rows<MB / 2, Q, MODE, AUX>(p, lds, m0, ex, tn, rows);
      return;
    }
  }
  mx4_tile<MB, mx4_stages(MB), Q, MODE, AUX>(p, lds, m0, ex, tn);
}

// gate_up is bound by its weights' way from beyond L2: 509 tokens of 256 experts (top 8, H =
// 7168, I = 256) 84 us, 5.9 TB/s, 13 tokens 28; 4096 tokens 159, 0.75 GB for 0.5 of need,
// as an expert's further blocks seldom find them there.  64 experts, H = 2048, I = 768, 1000
// tokens: 43, eight steps a tile whose start and end take as long.  Three workgroups a CU with
// a ring of two are level (82 and 42), but 13 tokens take 39.
template <int MB, int Q, int MODE>
__global__ void __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2))) mx4_grouped(Mx4Args p) {
#if defined(__HIP_DEVICE_COMPILE__)
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  int tm, tn;
  if (!grouped_place(p, 16 * MB, tm, tn)) return;
  const int m0 = tm * 16 * MB;
  const int64_t ex = p.block_expert[tm];
  if (ex < 0 || ex >= p.experts) {
    if constexpr (MODE == MX4_DOWN)
      zero_slot_rows(p, m0, 16 * MB, p.col0 + tn * 256, min(p.col0 + p.ncol, p.col0 + tn * 256 + 256), threadIdx.x, 64 * kWaves);
    return;
  }
  const int rows = block_rows(p, m0, 16 * MB, threadIdx.x & 63);
  // weights that no other block reads go past the caches
  const bool alone = (tm == 0 || p.block_expert[tm - 1] != ex) && ((tm + 1) * 16 * MB >= *p.num_padded || p.block_expert[tm + 1] != ex);
  if (alone)
    mx4_tile_rows<MB, Q, MODE, kReadOnce>(p, lds, m0, ex, tn, rows);
  else
    mx4_tile_rows<MB, Q, MODE, 0>(p, lds, m0, ex, tn, rows);
#endif
}

// The down product with short K (G groups, up to kShortGroups): each wave keeps its strip's
// weights in registers whole, the block's activation rows lie in LDS, and sixteen of them
// at a time are multiplied and stored.  Past its start a wave loads nothing more: loads and
// stores return in one order, so that a load's wait would cover the stores before it (rows
// straight from memory, a ring of three: 105 us a window of 4096 tokens, now 91: 125 MB of weights
// read and 235 of slot rows written; 509 tokens 59; 1000 of 64 experts to fp16 30.9, 49 MB of
// rows of 24 bits, with rows of 16 26.5).
constexpr int kShortGroups = 8;
constexpr int short_lds(int bm, int G) { return bm * (G * 68 + 8); }

template <int G>
__global__ void __launch_bounds__(64 * kWaves) mx4_down_short(Mx4Args p, int bm) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int Q = mx4_groups(G), CHUNKS = 4 * Q, SEG_ROWS = 64 / CHUNKS;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // rows [G / Q][bm][64 Q], chunks swizzled
  int tm, tn;
  if (!grouped_place(p, bm, tm, tn)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kq = lane >> 4;
  const int m0 = tm * bm, kb = p.K / 2;
  const int64_t ex = p.block_expert[tm];
  const int c0 = p.col0 + tn * 256, c1 = min(c0 + 256, p.col0 + p.ncol);
  if (ex < 0 || ex >= p.experts) {
    zero_slot_rows(p, m0, bm, c0, c1, tid, 64 * kWaves);
    return;
  }
  uint32_t* ls = reinterpret_cast<uint32_t*>(lds + G * bm * 64);  // powers of two [G][bm]
  int32_t* lid = reinterpret_cast<int32_t*>(ls + G * bm);
  float* ltw = reinterpret_cast<float*>(lid + bm);
  const int id = tid < bm ? p.sorted_ids[m0 + tid] : p.n_slots;
  const auto ra = mx4_rsrc(p.a, (int64_t)p.a_rows * kb);
  for (int i = wave; i < G * bm / 16; i += kWaves) {
    const int s = i / (bm / SEG_ROWS), r = (i - s * (bm / SEG_ROWS)) * SEG_ROWS + lane / CHUNKS;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(lds + i * 1024), 16, (m0 + r) * kb + swz<CHUNKS>(r, lane % CHUNKS) * 16, s * 64 * Q, 0, 0);
  }
  const int col = c0 + 64 * wave, at = min(col, c1 - 64) / 64 * G * kMx4GroupBytes;
  const auto rw = mx4_rsrc(p.w + ex * p.w_expert, p.w_expert);
  u4_t w[G][4];
  Mx4Scales<Q> sw[G / Q];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[g][j] = __builtin_bit_cast(u4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, lane * 16 + j * 1024, at + g / Q * Q * kMx4GroupBytes + g % Q * 4096, 0));
#pragma unroll
  for (int s = 0; s < G / Q; ++s) sw[s].template load<0>(rw, lane, at + s * Q * kMx4GroupBytes);
  if (tid < bm) {
#pragma unroll
    for (int g = 0; g < G; ++g) ls[g * bm + tid] = p.a_scale[(int64_t)g * p.a_rows + m0 + tid];
    lid[tid] = id;
    ltw[tid] = id < p.n_slots ? p.topk_w[id] : 0.f;
  }
  __builtin_amdgcn_s_waitcnt(0);  // this wave's loads into LDS have landed
  __syncthreads();
  if (col >= c1) return;
  int live = 0;  // rows that hold a slot: a prefix of the block
  for (int b = 0; b < bm; b += 64) live += __popcll(__ballot(b + lane < bm && lid[min(b + lane, bm - 1)] < p.n_slots));
  for (int r = 0; r < live; r += 16) {
    f4_t acc[1][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[0][j] = f4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const u4_t a = *reinterpret_cast<const u4_t*>(lds + ((g / Q) * bm + r + c16) * 64 * Q + swz<CHUNKS>(c16, 4 * (g % Q) + kq) * 16);
      mx4_strip(w[g], a, acc[0], sw[g / Q].v[g % Q], ls[g * bm + r + c16] >> (8 * kq));
    }
    if (p.rows8)
      store_slot_rows24<1>(p, lid + r, ltw + r, col, lane, acc);
    else
      store_slot_rows<1>(p, lid + r, ltw + r, col, lane, acc);
  }
#endif
}

__global__ void repack_mx4_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ e8m0, uint8_t* __restrict__ out, int64_t N,
                                  int64_t K, int paired, int64_t per, int64_t total) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t e = i / per;
    alignas(16) uint8_t v[16];
    mx4_repack_chunk(codes + e * N * (K / 2), e8m0 + e * N * (K / 32), N, K, paired, i - e * per, v);
    reinterpret_cast<u4_t*>(out)[i] = *reinterpret_cast<const u4_t*>(v);
  }
}

template <int MB, int Q, int MODE>
hipError_t launch_tiles(const Mx4Args& a, dim3 grid, hipStream_t s) {
  // the largest ring of the row counts a block may run with
  constexpr int LOW = MB < 4 ? MB : 4;
  constexpr size_t lds = std::max<size_t>(Mx4Cfg<MB, mx4_stages(MB), Q>::LDS, Mx4Cfg<LOW, mx4_stages(LOW), Q>::LDS);
  const hipError_t e = allow_lds<mx4_grouped<MB, Q, MODE>>(lds);
  return e != hipSuccess ? e : launch_timed(mx4_grouped<MB, Q, MODE>, grid, dim3(64 * kWaves), lds, s, a);
}

template <int MB>
hipError_t launch_block(int mode, const Mx4Args& a, dim3 grid, hipStream_t s) {
  if (mx4_groups(a.G) == 2) return mode == MX4_DOWN ? launch_tiles<MB, 2, MX4_DOWN>(a, grid, s) : launch_tiles<MB, 2, MX4_GATE_UP>(a, grid, s);
  return mode == MX4_DOWN ? launch_tiles<MB, 1, MX4_DOWN>(a, grid, s) : launch_tiles<MB, 1, MX4_GATE_UP>(a, grid, s);
}

template <int G>
hipError_t launch_short(const Mx4Args& a, int bm, dim3 grid, hipStream_t s) {
  if constexpr (G <= kShortGroups) {
    if (a.G != G) return launch_short<G + 1>(a, bm, grid, s);
    const hipError_t e = allow_lds<mx4_down_short<G>>(short_lds(128, G));
    return e != hipSuccess ? e : launch_timed(mx4_down_short<G>, grid, dim3(64 * kWaves), (size_t)short_lds(bm, G), s, a, bm);
  }
  return hipErrorInvalidValue;
}

}  // namespace

int launch_mx4_repack(int64_t N, int64_t K, int64_t E, bool paired, const void* codes, const void* e8m0, void* w_out, void* stream) {
  const int64_t per = mx4_weight_bytes(N, K) / 16;
  hipLaunchKernelGGL(repack_mx4_kernel, dim3((unsigned)std::min<int64_t>((per * E + 255) / 256, 65536)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(e8m0),
                     static_cast<uint8_t*>(w_out), N, K, (int)paired, per, per * E);
  return (int)hipGetLastError();
}

int launch_mx4_grouped(int mode, int bm, const Mx4Args& a, int64_t blocks, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.G < 1 || a.N % (mode == MX4_GATE_UP ? 256 : 64) || blocks < 1) return (int)hipErrorInvalidValue;
  if (mode == MX4_DOWN && (a.ncol < 64 || a.ncol % 64 || a.col0 % 64 || a.col0 + a.ncol > a.N)) return (int)hipErrorInvalidValue;
  if (bm != 16 && bm != 64 && bm != 128) return (int)hipErrorInvalidValue;
  Mx4Args b = a;
  b.tiles_n = (int)((mode == MX4_DOWN ? a.ncol : a.N) + 255) / 256;
  if (blocks * b.tiles_n > INT32_MAX) return (int)hipErrorInvalidValue;
  const dim3 grid((unsigned)(blocks * b.tiles_n));
  if (mode == MX4_DOWN && a.G <= kShortGroups) return (int)launch_short<1>(b, bm, grid, s);
  switch (bm) {
    case 16: return (int)launch_block<1>(mode, b, grid, s);
    case 64: return (int)launch_block<4>(mode, b, grid, s);
  }
  return (int)launch_block<8>(mode, b, grid, s);
}

}  // namespace hq
