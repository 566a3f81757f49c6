// What an MXFP4 experts' layer needs before its products, in one launch: x in MXFP4 and the
// slots sorted by expert.  4096 x 7168 and 32768 slots of 256 experts 17.4 us, the quantiser's 74
// MB alone 15 and one sorting workgroup alone 25.6; 13 tokens 5.5, two launches before 9.
#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <algorithm>

#include "block8_device.h"
#include "launch.h"
#include "mx4.h"
#include "mx4_device.h"

namespace hq {

namespace {

constexpr int kThreads = 1024;
constexpr int kMostSorters = 16;

// Workgroup `w` of `of`, which sorts the w-th part of the slots.  Each counts every slot's
// expert, those before its part apart from the others, so that it knows where its own go
// without a word from the rest; the segments' tails and the blocks' experts are shared out
// as well.  A segment holds an expert's slots, up to whole blocks; the last those of no
// expert, whose blocks are marked -1.
__device__ void sort_slots(const Mx4PrepareArgs& p, int w, int of, int* lds) {
  const int S = p.E + 1, tid = threadIdx.x, n = p.n_slots;
  int* before = lds;      // then: the next place of the segment
  int* count = lds + S;   // slots from the part on; then: of all
  int* start = lds + 2 * S;  // [S + 1]
  for (int e = tid; e < S; e += kThreads) before[e] = count[e] = 0;
  __syncthreads();
  const int from = (int)((int64_t)n * w / of), to = (int)((int64_t)n * (w + 1) / of);
  auto segment = [&](int id) { return id >= 0 && id < p.E ? id : p.E; };
  constexpr int kBatch = 16;  // loads in flight
  for (int base = tid; base < n; base += kBatch * kThreads) {
    int id[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) id[u] = p.ids[min(base + u * kThreads, n - 1)];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = base + u * kThreads;
      if (i < n) atomicAdd((i < from ? before : count) + segment(id[u]), 1);
    }
  }
  __syncthreads();
  if (tid < 64) {  // each lane a run of segments
    const int per = (S + 63) / 64, e0 = min(S, tid * per), e1 = min(S, e0 + per);
    int run = 0;
    for (int e = e0; e < e1; ++e) {
      count[e] += before[e];
      run += (count[e] + p.bm - 1) / p.bm * p.bm;
    }
    int upto = run;
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d, 64);
      if (tid >= d) upto += v;
    }
    int at = upto - run;
    for (int e = e0; e < e1; ++e) {
      start[e] = at;
      before[e] += at;
      at += (count[e] + p.bm - 1) / p.bm * p.bm;
    }
    if (tid == 63) {
      start[S] = upto;
      if (w == 0) *p.padded = upto;
    }
  }
  __syncthreads();
  // tails and blocks: 16 lanes a segment
  for (int e = w + of * (tid >> 4); e < S; e += of * (kThreads / 16)) {
    for (int i = start[e] + count[e] + (tid & 15); i < start[e + 1]; i += 16) p.sorted[i] = n;
    for (int b = start[e] / p.bm + (tid & 15); b < start[e + 1] / p.bm; b += 16) p.blocks[b] = e < p.E ? e : -1;
  }
  for (int base = from + tid; base < to; base += kBatch * kThreads) {
    int id[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) id[u] = p.ids[min(base + u * kThreads, n - 1)];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = base + u * kThreads;
      if (i < to) p.sorted[atomicAdd(before + segment(id[u]), 1)] = i;
    }
  }
}

// Workgroups 0 .. sorters - 1 sort, the others quantise 8 rows by 8 words of four blocks
// (as the stand-alone quantiser, 16 lanes a word).
template <bool BF16>
__global__ void __launch_bounds__(kThreads) mx4_prepare(Mx4PrepareArgs p) {
  extern __shared__ int lds[];
  const int b = (int)blockIdx.x - p.sorters;
  if (b < 0) {
    sort_slots(p, blockIdx.x, p.sorters, lds);
    return;
  }
  const uint32_t G = p.k8 / 16, octs = (G + 7) / 8, rb = (uint32_t)b / octs;
  const uint32_t g = ((uint32_t)b - rb * octs) * 8 + (threadIdx.x >> 7), row = rb * 8 + ((threadIdx.x >> 4) & 7);
  if (g >= G || row >= p.m) return;
  const int64_t at = (int64_t)row * p.k8 + g * 16 + (threadIdx.x & 15);
  float v[8];
  b8_unpack<BF16>(static_cast<const u4_t*>(p.x)[at], v);
  uint32_t top = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, b8_mag(v[j]));
  const uint32_t s = mx4_scale(quad_max(top));
  p.codes[at] = mx4_word(v, s);
  const uint32_t all = mx4_scale_word(s);
  if ((threadIdx.x & 15) == 0) p.e8m0[(int64_t)g * p.m + row] = all;
}

}  // namespace

int launch_mx4_prepare(const Mx4PrepareArgs& a, void* stream) {
  Mx4PrepareArgs b = a;
  b.sorters = std::max(1, std::min(kMostSorters, (a.n_slots + 2047) / 2048));
  const size_t lds = (size_t)(3 * (a.E + 1) + 1) * sizeof(int);
  const unsigned quantisers = a.x ? (a.k8 / 16 + 7) / 8 * ((a.m + 7) / 8) : 0;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)b.sorters + quantisers);
  return a.x_bf16 ? (int)launch_timed(mx4_prepare<true>, grid, dim3(kThreads), lds, s, b)
                  : (int)launch_timed(mx4_prepare<false>, grid, dim3(kThreads), lds, s, b);
}

}  // namespace hq
