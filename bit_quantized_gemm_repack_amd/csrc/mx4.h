// Internal interface of the experts' layers in MXFP4 (grouped FMT_F44): kernel arguments
// and launchers (they return a hipError_t as int).
//
// Activations and weights are E2M1 codes with one power of two per 32 k, which the
// scaled matrix instruction takes as they are: a product needs no promotion.
//
// Device weight layout: codes as the dense plans have them (hq_internal.h: fragments of
// 16 columns x 128 k, 1 KiB, lane l the 32 codes of column l % 16 and block l / 16),
// powers of two [N/16][K/128][64 lanes] bytes.  Activation codes are row-major, their
// powers of two words [K/128][rows] of four blocks.
#pragma once

#include "hq_internal.h"

namespace hq {

struct Mx4Args {
  const uint8_t* a;          // codes, K / 2 bytes a row
  const uint32_t* a_scale;   // [G][a_rows]
  const uint8_t* w;
  const uint8_t* w_scale;
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
  int64_t w_expert;          // code bytes per expert
  int64_t s_expert;          // powers of two per expert
  uint8_t* out_scale;        // gate_up: [N / 256][out_rows][4]
  int out_rows;
  // down: this launch's columns [col0, col0 + ncol) of N, col0 a multiple of
  // 256; the slots' rows with a scale per 64 columns
  int col0, ncol;
  uint16_t* rows16;          // [n_slots][ncol] fp16
  float* row_scale;          // [n_slots][ncol / 64]
  int cols_wg;               // short K: columns a workgroup walks
};

enum Mx4Mode : int { MX4_GATE_UP = 0, MX4_DOWN = 1 };

// Aligned blocks of bm rows (16, 64, 128) by 256 columns.
int launch_mx4_grouped(int mode, int bm, const Mx4Args& a, int64_t blocks, void* stream);

}  // namespace hq
