// Device helpers of the grouped products (aligned blocks of an expert's slots): where a
// workgroup's tile lies, and the slots' rows on their way into the sum over a token's
// experts.  Args: the kernel's arguments (sorted_ids, num_padded, topk_w, n_slots,
// tiles_n, and for the rows col0, ncol, rows16, row_scale).
#pragma once

#include "block8_device.h"

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

// A slot's row of the down GEMM, 64 columns a wave, on its way into the sum over
// the token's experts: fp16 values o / 2^e, with the 2^e that brings the 64 columns'
// largest finite one to [2^14, 2^15), and topk_w * 2^e as their scale.  Half the
// bytes of fp32 rows, which are a third of the layer's traffic (4096 tokens with
// fp16 outputs: 980 us with fp32 rows, 739 with these).  Each value is off by at most
// 2^-11 of itself down to 2^-29 of the largest, and below that by 2^-39 of the
// largest: an eighth of bf16's rounding, and as much as fp16's own.  (Integers of
// one step for the 64 columns were finer beside a large column and lost the others.)
// What is not finite stays in its column.
template <int MB, typename Args>
__device__ __forceinline__ void store_slot_rows(const Args& p, const int32_t* ids, const float* tw, uint8_t* buf, int col,
                                              int lane, const f4_t (&acc)[MB][4]) {
  const int c16 = lane & 15;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    uint32_t top = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t m = b8_mag(acc[mb][j][q]);
        top = max(top, m < 0x7F800000u ? m : 0u);
      }
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    const int e = max((int)(top >> 23) - 127 - 14, -126);  // the largest is below 2^(e + 15)
    const float inv = __builtin_amdgcn_ldexpf(1.f, -e);    // (exact: e is at most 113)
    const int id = ids[16 * mb + c16];
    const bool live = id < p.n_slots;
    char* o = reinterpret_cast<char*>(p.rows16 + (int64_t)(live ? id : 0) * p.ncol + (col - p.col0));
    rows16_out<4>(
        buf, lane,
        [&](int j) {
          uint32_t v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = float_to_f16_bits(acc[mb][j][q] * inv);
          return uint2{v[0] | (v[1] << 16), v[2] | (v[3] << 16)};
        },
        [&](int byte, uint4 v) {
          if (live) *reinterpret_cast<uint4*>(o + byte) = v;
        });
    if (live && lane < 16)
      p.row_scale[(int64_t)id * (p.ncol / 64) + (col - p.col0) / 64] = tw[16 * mb + c16] * __builtin_amdgcn_ldexpf(1.f, e);
  }
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
    *reinterpret_cast<uint2*>(p.rows16 + (int64_t)id * p.ncol + col + 4 * (i & 15)) = uint2{0u, 0u};
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
