// Device helpers of the grouped products (aligned blocks of an expert's slots): where a
// workgroup's tile lies, and the slots' rows on their way into the sum over a token's
// experts.  Args: the kernel's arguments (sorted_ids, num_padded, topk_w, n_slots,
// tiles_n, and for the rows col0, ncol, rows16, rows8, row_scale).
#pragma once

#include "block8_device.h"
#include "hq_internal.h"

namespace hq {

// Sixteen rows of 16 NB 16-bit values from the operand layout (lane (c16, kq),
// fragment j: columns 16 j + 4 kq .. + 3 of row c16) to 16 bytes a lane, so
// that a store instruction covers whole 64-byte runs of its rows; through the
// wave's own 16 x (32 NB + 16) bytes of LDS.  Stored 8 bytes a lane straight
// from the operand layout, the rows of the down GEMM took 129 us of 4096
// tokens' 340.
constexpr int rows_lds(int NB) { return 16 * (32 * NB + 16); }

template <int NB, typename V, typename S>
__device__ __forceinline__ void rows16_out(uint8_t* buf, int lane, V&& value, S&& store) {
  const int c16 = lane & 15, kq = lane >> 4;
  constexpr int PITCH = 32 * NB + 16;
#pragma unroll
  for (int j = 0; j < NB; ++j) *reinterpret_cast<uint2*>(buf + c16 * PITCH + 32 * j + 8 * kq) = value(j);
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int h = 0; h < NB / 2; ++h)
    store(64 * h + 16 * kq, *reinterpret_cast<const uint4*>(buf + c16 * PITCH + 64 * h + 16 * kq));
  __builtin_amdgcn_wave_barrier();
}

// Maximum over the lanes that differ in bit D (16, 32) of their number, in each of them.
template <int D>
__device__ __forceinline__ float lanes_max(float v) {
#if defined(__HIP_DEVICE_COMPILE__)
  const uint32_t b = __float_as_uint(v);
  if constexpr (D == 16) {
    const auto x = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    return fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
  } else {
    const auto x = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
  }
#else
  return v;
#endif
}

// A slot's row of the down GEMM, 64 columns a wave, on its way into the sum over
// the token's experts: fp16 values o / 2^e, with the 2^e that brings the 64 columns'
// largest finite one to [2^14, 2^15), and topk_w * 2^e as their scale.  Half the
// bytes of fp32 rows, which are a third of the layer's traffic (an fp8 block layer of 4096
// tokens with fp16 outputs: 980 us with fp32 rows, 725 with these).  Each value is off by at most
// 2^-11 of itself down to 2^-29 of the largest, and below that by 2^-39 of the
// largest: an eighth of bf16's rounding, and as much as fp16's own.  (Integers of
// one step for the 64 columns were finer beside a large column and lost the others.)
// What is not finite stays in its column.
template <int MB, typename Args>
__device__ __forceinline__ void store_slot_rows(const Args& p, const int32_t* ids, const float* tw, int col, int lane, const f4_t (&acc)[MB][4]) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int c16 = lane & 15, kq = lane >> 4;
  // Rows without a slot are stored past the end, which writes nothing: with a branch
  // around them the next loads' wait would cover these stores, each block's in turn.
  const auto rows = __builtin_amdgcn_make_buffer_rsrc(p.rows16, (short)0, (int)((uint32_t)p.n_slots * (uint32_t)(2 * p.ncol)), 0x00020000);
  const auto scales = __builtin_amdgcn_make_buffer_rsrc(p.row_scale, (short)0, (int)((uint32_t)p.n_slots * (uint32_t)(p.ncol / 16)), 0x00020000);
  const uint32_t at = 2 * (col - p.col0) + (kq & 1) * 32 + (kq >> 1) * 16;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; q += 2) top = fmaxf(fmaxf(fabsf(acc[mb][j][q]), fabsf(acc[mb][j][q + 1])), top);
    if (__ballot(top == __builtin_inff())) {  // the largest finite one
      top = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float m = fabsf(acc[mb][j][q]);
          top = m < __builtin_inff() ? fmaxf(top, m) : top;
        }
    }
    top = lanes_max<16>(top);
    top = lanes_max<32>(top);
    const int e = max((int)(__float_as_uint(top) >> 23) - 127 - 14, -126);  // the largest is below 2^(e + 15)
    const float inv = __builtin_amdgcn_ldexpf(1.f, -e);                     // (exact: e is at most 113)
    const int id = ids[16 * mb + c16];
    const bool live = id < p.n_slots;
    const uint32_t row = live ? (uint32_t)id * (uint32_t)(2 * p.ncol) + at : kSlotRowsMost;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t v[2][2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const f4_t& a = acc[mb][2 * h + j];
          v[j][q] = (uint32_t)float_to_f16_bits(a[2 * q] * inv) | ((uint32_t)float_to_f16_bits(a[2 * q + 1] * inv) << 16);
        }
      // lanes of odd kq give their first four columns for their neighbour's second four
      u4_t o;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const auto x = __builtin_amdgcn_permlane16_swap(v[0][q], v[1][q], false, false);
        o[q] = x[0];
        o[2 + q] = x[1];
      }
      __builtin_amdgcn_raw_buffer_store_b128(o, rows, row, 64 * h, 0);
    }
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(tw[16 * mb + c16] * __builtin_amdgcn_ldexpf(1.f, e)), scales,
                                          live && kq == 0 ? (uint32_t)id * (uint32_t)(p.ncol / 16) + (col - p.col0) / 16 : kSlotRowsMost, 0, 0);
  }
#endif
}

// The same rows in 24 bits a value, for sums that go on to fp16: the upper three bytes of the
// rounded fp32, two of them in rows16 and one in rows8, and topk_w as their scale.  Each value
// is off by at most 2^-16 of itself.  In an MXFP4 layer of 4096 tokens of 256 experts (H = 7168)
// 556 us against 457 with 16 bits and 692 with fp32; of 1000 tokens of 64 (H = 2048) 78 against
// 74 and 84.  (The lowest bytes in two stores of 8 a lane: 583, 79.)
template <int MB, typename Args>
__device__ __forceinline__ void store_slot_rows24(const Args& p, const int32_t* ids, const float* tw, int col, int lane, const f4_t (&acc)[MB][4]) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int c16 = lane & 15, kq = lane >> 4;
  const uint32_t ncol = (uint32_t)p.ncol, n = (uint32_t)p.n_slots;
  const auto high = __builtin_amdgcn_make_buffer_rsrc(p.rows16, (short)0, (int)(n * (2 * ncol)), 0x00020000);
  const auto low = __builtin_amdgcn_make_buffer_rsrc(p.rows8, (short)0, (int)(n * ncol), 0x00020000);
  const auto scales = __builtin_amdgcn_make_buffer_rsrc(p.row_scale, (short)0, (int)(n * (ncol / 16)), 0x00020000);
  const uint32_t at = (col - p.col0) + (kq & 1) * 16 + (kq >> 1) * 8;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const uint32_t id = (uint32_t)ids[16 * mb + c16];
    const bool live = id < n;
    uint32_t lows[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t hi[2][2], lo[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float v = acc[mb][2 * h + j][q];
          b[q] = v == v ? __float_as_uint(v) + 0x80u : 0x7FC00000u;
        }
        hi[j][0] = __builtin_amdgcn_perm(b[1], b[0], 0x07060302);
        hi[j][1] = __builtin_amdgcn_perm(b[3], b[2], 0x07060302);
        lo[j] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0C0C0501), __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0501), 0x05040100);
      }
      // lanes of odd kq give their first four columns for their neighbour's second four
      u4_t o;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const auto x = __builtin_amdgcn_permlane16_swap(hi[0][q], hi[1][q], false, false);
        o[q] = x[0];
        o[2 + q] = x[1];
      }
      const auto y = __builtin_amdgcn_permlane16_swap(lo[0], lo[1], false, false);
      lows[h][0] = y[0];
      lows[h][1] = y[1];
      __builtin_amdgcn_raw_buffer_store_b128(o, high, live ? id * (2 * ncol) + 2 * at : kSlotRowsMost, 64 * h, 0);
    }
    // lanes of kq >= 2 give their eight columns of the first half for their neighbour's of the second
    const auto y0 = __builtin_amdgcn_permlane32_swap(lows[0][0], lows[1][0], false, false);
    const auto y1 = __builtin_amdgcn_permlane32_swap(lows[0][1], lows[1][1], false, false);
    __builtin_amdgcn_raw_buffer_store_b128(u4_t{y0[0], y1[0], y0[1], y1[1]}, low,
                                           live ? id * ncol + (col - p.col0) + (kq & 1) * 16 + (kq >> 1) * 32 : kSlotRowsMost, 0, 0);
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(tw[16 * mb + c16]), scales,
                                          live && kq == 0 ? id * (ncol / 16) + (col - p.col0) / 16 : kSlotRowsMost, 0, 0);
  }
#endif
}

// Slots and top-k weights of a block's rows, into LDS.
template <typename Args>
__device__ inline void load_slots(const Args& p, int m0, int rows, int32_t* ids, float* tw, int tid, int threads) {
  for (int i = tid; i < rows; i += threads) {
    const int id = p.sorted_ids[m0 + i];
    ids[i] = id;
    tw[i] = id < p.n_slots ? p.topk_w[id] : 0.f;
  }
}

// The rows of slots whose expert id is out of range: zeros, columns [c0, c1).
template <typename Args>
__device__ inline void zero_slot_rows(const Args& p, int m0, int rows, int c0, int c1, int tid, int threads) {
  const int n = (c1 - c0) / 64;  // strips
  for (int i = tid; i < rows * n * 16; i += threads) {
    const int s = i >> 4, r = s / n, strip = s - r * n;
    const int id = p.sorted_ids[m0 + r];
    if (id >= p.n_slots) continue;
    const int col = c0 + 64 * strip - p.col0;
    const int64_t at = (int64_t)id * p.ncol + col + 4 * (i & 15);
    *reinterpret_cast<uint2*>(p.rows16 + at) = uint2{0u, 0u};
    if constexpr (requires { p.rows8; })
      if (p.rows8) *reinterpret_cast<uint32_t*>(p.rows8 + at) = 0u;
    if ((i & 15) == 0) p.row_scale[(int64_t)id * (p.ncol / 64) + col / 64] = 0.f;
  }
}

// Rows of the aligned block from m0 on that hold a slot: a prefix of it.
template <typename Args>
__device__ inline int block_rows(const Args& p, int m0, int bm, int lane) {
  int n = 0;
  for (int b = 0; b < bm; b += 64)
    n += __popcll(__ballot(b + lane < bm && p.sorted_ids[m0 + min(b + lane, bm - 1)] < p.n_slots));
  return n;
}

// Workgroup ids are dealt round-robin to the 8 XCDs, each with an L2 of its own:
// the id'th of n workgroups takes this logical tile, so that every XCD runs a
// consecutive run of them.
__device__ __forceinline__ int xcd_order(int id, int n) {
  const int xcd = id & 7, each = n >> 3, over = n & 7;
  return xcd * each + min(xcd, over) + (id >> 3);
}

// The tile of a grouped launch (row block tm, column tile tn), or false past the
// padded rows.  The column tiles of a row block and the row blocks of an expert
// follow each other on one XCD, so that its L2 fetches the rows and the expert's
// weights once where they keep pace (4096 tokens, 256 experts, top 8, H = 7168,
// I = 256: gate_up 303 us against 325 with ids in order).
template <typename Args>
__device__ __forceinline__ bool grouped_place(const Args& p, int bm, int& tm, int& tn) {
  const int n = *p.num_padded / bm * p.tiles_n;
  if ((int)blockIdx.x >= n) return false;
  const int lid = xcd_order(blockIdx.x, n);
  tm = lid / p.tiles_n;
  tn = lid - tm * p.tiles_n;
  return true;
}

}  // namespace hq
