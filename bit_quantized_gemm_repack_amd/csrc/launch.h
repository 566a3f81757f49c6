// Kernel launch that honours the timing events armed for it (hq_time_next_launch):
// a launch with events goes through the extended launch, which records them
// at the dispatch's start and end on the device.
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include <atomic>

#include "hq_internal.h"

namespace hq {

template <typename Kern, typename... Args>
inline hipError_t launch_timed(Kern kern, dim3 grid, dim3 block, size_t lds, hipStream_t s, Args... args) {
  const TimingEvents ev = take_timing();
  if (ev.start || ev.stop)
    hipExtLaunchKernelGGL(kern, grid, block, (uint32_t)lds, s, static_cast<hipEvent_t>(ev.start),
                          static_cast<hipEvent_t>(ev.stop), 0, args...);
  else
    hipLaunchKernelGGL(kern, grid, block, lds, s, args...);
  return hipGetLastError();
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
