// Internal interface of the fp8 x fp8 path with 128-block scales (FMT_B8):
// kernel arguments and launchers (they return a hipError_t as int).
//
// Value of a weight: w[n, k] = e4m3(code) * sw[n / 128, k / 128], of an
// activation: a[m, k] = e4m3(code) * sa[k / 128, m], so
//   C[m, n] = sum_g sa[g, m] * sw[n / 128, g] * P_g[m, n],
// P_g the product of the codes over the 128 k of group g, which one
// 16x16x128 matrix instruction forms for 16 x 16 outputs.
//
// Device weight layout: fragments of 16 columns x 128 k, 2 KiB, n-block major
// (fragment (nb, g) at ((nb * K/128) + g) * 2048).  Half h of a fragment holds
// for lane l the 16 codes of column l % 16, k = 64 h + 16 (l / 16) + [0, 16):
// one 16-byte load per lane, registers 4h .. 4h+3 of the operand.  The
// activation operand takes the same k in the same registers.  Weight scales
// stay fp32 [ceil(N/128)][K/128].
#pragma once

#include "hq_internal.h"

namespace hq {

struct B8Args {
  const uint8_t* a;        // codes, row-major, K bytes a row
  const float* a_scale;    // [G][a_rows]
  const uint8_t* w;
  const float* w_scale;    // [ceil(N/128)][G] per expert
  void* out;
  float* part;             // [split][M][N] fp32 partials (split > 1)
  int M, N, K, G;
  int a_rows;              // rows of a and of each scale group
  int out_bf16;
  int gps;                 // groups per split
  int tiles_m, tiles_n, group_m;
  // ---- grouped (MoE) ----
  const int32_t* sorted_ids;
  const int32_t* block_expert;
  const int32_t* num_padded;
  const float* topk_w;
  int once;                // most experts' rows lie in one block
  int topk, n_slots;
  int experts;             // a block_expert outside [0, experts) is no expert
  int64_t w_expert;        // code bytes per expert
  int64_t s_expert;        // weight scales per expert
  float* out_scale;        // gate_up: scales of the requantised rows [N/256][out_rows]
  int out_rows;
  // down: this launch's columns [col0, col0 + ncol) of N, col0 a multiple of
  // 256; the slots' rows with a scale per 64 columns
  int col0, ncol;
  uint16_t* rows16;        // [n_slots][ncol] fp16
  float* row_scale;        // [n_slots][ncol / 64]
  int cols_wg;             // short K: columns a workgroup walks
};

enum B8Mode : int { B8_DENSE = 0, B8_GATE_UP = 1, B8_DOWN = 2 };

// A dense tile: bm rows (16 .. 128) by bn columns (128, 256), K over `split`
// workgroups, `stages` groups in the load ring.
struct B8Tile {
  int bm, bn, split, stages;
};
inline int b8_stages(int bm) { return bm >= 128 ? 2 : (bm == 64 ? 3 : 4); }
bool b8_tile_ok(const B8Tile& t);
int launch_b8_dense(const B8Tile& t, const B8Args& a, void* stream);
// Grouped: aligned blocks of bm rows (16, 64, 128) by 256 columns.
int launch_b8_grouped(int mode, int bm, const B8Args& a, int64_t blocks, void* stream);
// y = the sum of a token's slot rows over the columns of a's window.
int launch_b8_combine(const B8Args& a, int64_t t, void* stream);

// Few rows: 16 rows by 16 nb columns a workgroup, K over its waves and over
// `split` workgroups.
struct B8Skinny {
  int nb, waves, split;
};
bool b8_skinny_ok(const B8Skinny& c);
int launch_b8_skinny(const B8Skinny& c, const B8Args& a, void* stream);

int launch_b8_repack(int64_t N, int64_t K, int64_t E, const void* codes, const void* scales, void* w_out,
                     void* meta_out, void* stream);

// x [m, k] (silu: [m, 2k], SiLU(x[:, :k]) * x[:, k:]) -> codes [m, k] and
// scales [k/128, m].
int launch_quantize_blocks(int64_t m, int64_t k, int in_bf16, int silu, const void* x, void* codes, float* scales,
                           void* stream);

// Routing: softmax top-k of each row of logits [t][E] (logit_type 0 fp32, 1
// bf16, 2 fp16), E <= 1024, topk <= 64.
int launch_route(int64_t t, int E, int topk, int logit_type, const void* logits, int renorm, int32_t* ids, float* w,
                 void* stream);

// An experts' layer for a few tokens in two kernels (block8_moe.hip).
constexpr int kB8FewMaxTokens = 64;
constexpr int kB8FewMaxTopk = 16;
constexpr int kB8FewMaxSlots = kB8FewMaxTokens * kB8FewMaxTopk;
// A tile's units: how many, their experts from int 16 on, then per unit the slot
// of each of the 16 tokens as 16-bit integers, -1 for none.
constexpr int kB8FewUnitInts = 16 + 16 * kB8FewMaxTopk * 9;

struct B8FewArgs {
  const void* x;        // [t][H]
  const void* logits;   // [t][E], or null: topk_ids and topk_w are given
  int32_t* topk_ids;    // [t][topk]
  float* topk_w;
  const uint8_t* w1;    // device layout, 2I x H per expert
  const float* s1;
  const uint8_t* w2;    // H x I per expert
  const float* s2;
  float* act;           // fp32 rows [t * topk][I], or with act_codes their scales [t * topk][I/128]
  uint8_t* act_codes;   // [t * topk][I], or null
  void* out;            // [t][H]
  int32_t* units;       // per tile of 16 tokens kB8FewUnitInts, for t > 1 (see few_units)
  int64_t w1_expert, s1_expert, w2_expert, s2_expert;
  int t, topk, E, H, I;
  int x_bf16, out_bf16, logit_type, renorm;
  int rows;             // rows of x a gate_up workgroup holds (set by its launcher)
  int down_groups;      // 128-k groups a down workgroup holds (set by its launcher)
};
int launch_few_gate_up(const B8FewArgs& a, void* stream);
int launch_few_down(const B8FewArgs& a, void* stream);

// One 32-bit word of the device layout <- canonical uint8 [N][K].
HQ_HD inline uint32_t repack_word_b8(const uint8_t* codes, int64_t K, int64_t widx) {
  const int64_t G = K / kFragK;
  const int u = (int)(widx & 3);
  const int lane = (int)((widx >> 2) & 63);
  const int h = (int)((widx >> 8) & 1);
  const int64_t frag = widx >> 9;
  const int64_t g = frag % G, nb = frag / G;
  const uint8_t* c = codes + (nb * kFragN + (lane & 15)) * K + g * kFragK + 64 * h + 16 * (lane >> 4) + 4 * u;
  return (uint32_t)c[0] | ((uint32_t)c[1] << 8) | ((uint32_t)c[2] << 16) | ((uint32_t)c[3] << 24);
}

}  // namespace hq
