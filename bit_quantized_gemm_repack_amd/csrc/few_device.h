// Device helpers of the two-kernel layers for a few tokens: which slots share an expert.
// Args: the layer's arguments (t, topk, E, topk_ids, units).
#pragma once

#include "block8.h"
#include "block8_device.h"

namespace hq {

// The ids a wave's lanes scan for an expert's slots, the first kScan of them in
// flight before the expert is known.
constexpr int kScan = 4;
template <typename Args>
__device__ inline void few_ids(const Args& p, int (&ids)[kScan], int lane) {
#pragma unroll
  for (int i = 0; i < kScan; ++i) ids[i] = p.topk_ids[min(64 * i + lane, p.t * p.topk - 1)];
}

// The slots that hold expert e, in order, into picks; returns how many.  Ends
// with a barrier.
template <typename Args>
__device__ inline int few_slots(const Args& p, int e, const int (&ids)[kScan], int* picks, int* npicks, int lane, int wave) {
  if (wave == 0) {
    int n = 0;
    auto scan = [&](int b, int id) {
      const bool hit = b + lane < p.t * p.topk && id == e;
      const uint64_t has = __ballot(hit);
      if (hit) picks[n + __popcll(has & ((1ull << lane) - 1))] = b + lane;
      n += __popcll(has);
    };
#pragma unroll
    for (int i = 0; i < kScan; ++i) scan(64 * i, ids[i]);
    for (int b = 64 * kScan; b < p.t * p.topk; b += 64) scan(b, p.topk_ids[min(b + lane, p.t * p.topk - 1)]);
    if (lane == 0) *npicks = n;
  }
  __syncthreads();
  return *npicks;
}

// The units of a tile of 16 tokens, for the down kernel: the distinct experts of
// its slots.  A token may hold an expert more than once (given ids): each
// occurrence is a unit of its own, so that a unit has at most one slot per
// token.  One workgroup; key: 2 kMax + 4 ints of LDS.  Found here, beside the
// stream, as in every down workgroup it cost up to a third of its time (13
// tokens: 36 us against 31).
template <int NW, typename Args>
__device__ inline void few_units(const Args& p, int tile, int* key, int tid) {
  constexpr int kMax = 16 * kB8FewMaxTopk;  // slots of a tile
  static_assert(64 * NW >= kMax);
  int* unit_of = key + kMax;  // index of a slot's unit, at the unit's first slot
  int* wcount = unit_of + kMax;
  const int lane = tid & 63, wave = tid >> 6;
  const int topk = p.topk, t0 = tile * 16, ns = min(16, p.t - t0) * topk;
  int32_t* out = p.units + (int64_t)tile * kB8FewUnitInts;
  for (int i = tid; i < ns * 8; i += 64 * NW) out[16 + kMax + i] = -1;
  int id = -1;
  if (tid < ns) {
    id = p.topk_ids[t0 * topk + tid];
    if (id < 0 || id >= p.E) id = -1;
  }
  if (tid < kMax) key[tid] = id;
  __syncthreads();
  const int tok = tid / topk, from = tok * topk;
  const bool have = tid < ns && id >= 0;
  int occ = 0;
  for (int j = 0; j < topk; ++j) occ += have && from + j < tid && key[min(from + j, kMax - 1)] == id;
  __syncthreads();
  const int k = id | (occ << 16);  // E is below 2^16
  if (have) key[tid] = k;
  __syncthreads();
  int first = kMax;
  for (int s = 0; s < ns; s += 4) {  // four keys a read, no read waits for another's result
    const int4 v = *reinterpret_cast<const int4*>(key + s);
    const int c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) first = min(first, c[q] == k ? s + q : kMax);
  }
  const bool lead = have && first == tid;
  const uint64_t leads = __ballot(lead);
  if (lane == 0 && wave < 4) wcount[wave] = __popcll(leads);
  __syncthreads();
  if (tid == 0) out[0] = wcount[0] + wcount[1] + wcount[2] + wcount[3];
  if (lead) {
    int at = __popcll(leads & ((1ull << lane) - 1));
    for (int w = 0; w < wave; ++w) at += wcount[w];
    unit_of[tid] = at;
    out[16 + at] = id;
  }
  __syncthreads();
  if (have) reinterpret_cast<int16_t*>(out + 16 + kMax)[unit_of[first] * 16 + tok] = (int16_t)tid;
  __syncthreads();  // before the next tile
}

__device__ inline __amdgpu_buffer_rsrc_t few_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

}  // namespace hq
