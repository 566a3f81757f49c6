// Internal interface of the experts' layers in MXFP4 (grouped FMT_F44): kernel arguments
// and launchers (they return a hipError_t as int).
//
// Activations and weights are E2M1 codes with one power of two per 32 k, which the
// scaled matrix instruction takes as they are: a product needs no promotion.
//
// Device weight layout, a private one of the grouped plans: strips of 64 columns, what one
// wave multiplies, each along K without a gap, so that a wave reads one stream (in the dense
// plans' order, 16 columns a stream and the powers of two apart, gate_up of 256 experts by
// 16 rows ran at 4.5 TB/s for 5.6).  A strip is four fragments of 16 columns; gate_up's
// holds 32 columns of gate and the 32 of up that belong to the same outputs.  It goes in
// steps of q groups of 128 k, q = 2 where K/128 is even, else 1, each
//   codes           [q][fragment 4][lane 64][16 bytes]: lane l has the 32 codes of column l %
//                   16 and block l / 16
//   powers of two   [lane 64][q][fragment 4] bytes, a fragment's by the matrix instruction's
//                   selector
// and all of it lies in the codes' buffer; the metadata is empty.
// Activation codes are row-major, their powers of two words [K/128][rows] of four blocks.
#pragma once

#include "hq_internal.h"

namespace hq {

struct Mx4Args {
  const uint8_t* a;          // codes, K / 2 bytes a row
  const uint32_t* a_scale;   // [G][a_rows]
  const uint8_t* w;
  void* out;                 // gate_up: codes [rows][N / 4]
  int N, K, G;
  int a_rows;                // rows of a and of each scale group
  int tiles_n;
  const int32_t* sorted_ids;
  const int32_t* block_expert;
  const int32_t* num_padded;
  const float* topk_w;
  int topk, n_slots;
  int experts;               // a block_expert outside [0, experts) is no expert
  int64_t w_expert;          // bytes per expert
  uint8_t* out_scale;        // gate_up: [N / 256][out_rows][4]
  int out_rows;
  // down: this launch's columns [col0, col0 + ncol) of N, col0 a multiple of
  // 64; the slots' rows with a scale per 64 columns
  int col0, ncol;
  uint16_t* rows16;          // [n_slots][ncol] fp16, or with rows8 the upper bytes of 24-bit values
  uint8_t* rows8;            // [n_slots][ncol] their lowest bytes, or null
  float* row_scale;          // [n_slots][ncol / 64]
};

enum Mx4Mode : int { MX4_GATE_UP = 0, MX4_DOWN = 1 };

// Groups of 128 k a step, and a step's bytes.
HQ_HD constexpr inline int mx4_groups(int64_t G) { return G % 2 ? 1 : 2; }
constexpr int kMx4GroupBytes = 4 * kFragBytes + 256;
HQ_HD constexpr inline int64_t mx4_weight_bytes(int64_t N, int64_t K) { return N / 64 * (K / kFragK) * kMx4GroupBytes; }
// Column of fragment j, lane column c of a strip.
HQ_HD inline int64_t mx4_column(int64_t N, bool paired, int64_t strip, int j, int c) {
  return paired ? (j < 2 ? 0 : N / 2) + strip * 32 + (j & 1) * 16 + c : strip * 64 + j * 16 + c;
}
// The 16 bytes that are chunk `at` of an expert's device weight <- canonical codes [N][K/2]
// and E8M0 [N][K/32].
HQ_HD inline void mx4_repack_chunk(const uint8_t* codes, const uint8_t* e8m0, int64_t N, int64_t K, bool paired, int64_t at, uint8_t* out) {
  const int64_t G = K / kFragK;
  const int q = mx4_groups(G), per = q * (kMx4GroupBytes / 16), c = (int)(at % per);
  const int64_t step = at / per, g0 = step % (G / q) * q, strip = step / (G / q);
  if (c < q * 256) {
    const int lane = c & 63, j = (c >> 6) & 3, u = c >> 8;
    const uint8_t* from = codes + mx4_column(N, paired, strip, j, lane & 15) * (K / 2) + (g0 + u) * 64 + (lane >> 4) * 16;
    for (int i = 0; i < 16; ++i) out[i] = from[i];
    return;
  }
  for (int i = 0; i < 16; ++i) {
    const int b = (c - q * 256) * 16 + i, j = b & 3, u = (b >> 2) % q, lane = (b >> 2) / q;
    out[i] = e8m0[mx4_column(N, paired, strip, j, lane & 15) * (K / 32) + 4 * (g0 + u) + (lane >> 4)];
  }
}
#ifndef __HIPCC_RTC__
// Whether a plan's weights have this layout.
inline bool mx4_layout(const hq_plan* p) { return p->fmt == FMT_F44 && p->compute.kind == HQ_GEMM_GROUPED; }
#endif
int launch_mx4_repack(int64_t N, int64_t K, int64_t E, bool paired, const void* codes, const void* e8m0, void* w_out, void* stream);

// Aligned blocks of bm rows (16, 64, 128) by 256 columns.
int launch_mx4_grouped(int mode, int bm, const Mx4Args& a, int64_t blocks, void* stream);

// Before the products of a layer (mx4_prepare.hip): x in MXFP4 (not where x is null), and the
// slots by expert in blocks of bm rows, as hq_moe_align sorts them.
struct Mx4PrepareArgs {
  const void* x;  // 16-bit [m][8 k8]
  uint32_t* codes;
  uint32_t* e8m0;
  const int32_t* ids;
  int32_t* sorted;
  int32_t* blocks;
  int32_t* padded;
  uint32_t m, k8;
  int x_bf16;
  int n_slots, E, bm;
  int sorters;  // set by the launcher
};
int launch_mx4_prepare(const Mx4PrepareArgs& a, void* stream);

// An experts' layer for a few tokens in two kernels (mx4_few.hip).
enum Mx4Input : int { MX4_F16 = 0, MX4_BF16 = 1, MX4_CODES = 2 };
constexpr int kMx4FewTokens = 32, kMx4FewTopk = 16;
struct Mx4FewArgs {
  const void* x;             // [t][H] 16-bit, or codes [t][H / 2]
  const uint32_t* x_scale;   // of codes: [H / 128][t]
  const int32_t* topk_ids;   // [t][topk]
  const float* topk_w;
  const uint8_t* w1;         // 2I x H per expert
  const uint8_t* w2;         // H x I
  float* h;                  // gate and up [t * topk][2 I], or
  uint8_t* act;              // codes [t * topk][I / 2] and, behind them, their
  uint8_t* act_scale;        // powers of two [t * topk][I / 32]: the launcher's choice, in the same place
  void* out;                 // [t][H]
  int32_t* units;            // per tile of 16 tokens kB8FewUnitInts, for t > 1
  int64_t w1_expert, w2_expert;
  int t, topk, E, H, I;
  int input, out_bf16;
  int rows;                  // rows of x a gate_up workgroup holds (set by its launcher)
};
// Whether the two kernels take t tokens of this layer.
bool mx4_few_ok(int64_t t, int64_t topk, int64_t E, int64_t H, int64_t I);
// Bytes of h, or of act and act_scale.
size_t mx4_few_act_bytes(int64_t t, int64_t topk, int64_t I);
int launch_mx4_few(const Mx4FewArgs& a, void* stream);

}  // namespace hq
