// Kernel launch that honours the timing events armed for it (hq_time_next_launch):
// a launch with events goes through the extended launch, which records them
// at the dispatch's start and end on the device.
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>

#include "hq_internal.h"

namespace hq {

template <typename Kern, typename... Args>
inline hipError_t launch_timed(Kern kern, dim3 grid, dim3 block, size_t lds, hipStream_t s, Args... args) {
  const TimingEvents ev = take_timing();
  // a dispatch counts its work-items in 32 bits a dimension: a longer one would run in part
  if ((uint64_t)grid.x * block.x > UINT32_MAX || (uint64_t)grid.y * block.y > UINT32_MAX || (uint64_t)grid.z * block.z > UINT32_MAX)
    return hipErrorInvalidConfiguration;
  if (ev.start || ev.stop)
    hipExtLaunchKernelGGL(kern, grid, block, (uint32_t)lds, s, static_cast<hipEvent_t>(ev.start),
                          static_cast<hipEvent_t>(ev.stop), 0, args...);
  else
    hipLaunchKernelGGL(kern, grid, block, lds, s, args...);
  return hipGetLastError();
}

// The workgroups of a long input, whose work-items are more than a dimension of a dispatch
// counts: runs of kGridRun (of up to 1024 threads) along x, the runs along y.  The kernel takes
// grid_block() for its number and leaves at once past the last one.
constexpr unsigned kGridRun = 1u << 20;
inline dim3 grid_of(int64_t blocks) {
  return blocks <= kGridRun ? dim3((unsigned)blocks) : dim3(kGridRun, (unsigned)((blocks + kGridRun - 1) / kGridRun));
}
__device__ inline uint32_t grid_block() { return blockIdx.y * kGridRun + blockIdx.x; }

// `rows` of `threads` work-items each in as few launches as hold them, go(first, count) being
// one: for kernels whose grid is their rows, without a check in them.
template <typename Go>
inline hipError_t launch_rows(int64_t rows, int threads, Go&& go) {
  const int64_t most = UINT32_MAX / threads;
  const TimingEvents ev = take_timing();
  hipError_t e = hipSuccess;
  for (int64_t r = 0; r < rows && e == hipSuccess; r += most) {
    const int64_t n = std::min(most, rows - r);
    arm_timing({r ? nullptr : ev.start, r + n < rows ? nullptr : ev.stop});
    e = go(r, n);
  }
  return e;
}

// Raises a kernel's dynamic LDS limit to `bytes` on the current device, once
// per kernel and device (from any thread; setting it twice is harmless).
template <auto Kern>
inline hipError_t allow_lds(size_t bytes) {
  if (bytes <= 32 * 1024) return hipSuccess;
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(Kern), hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace hq
