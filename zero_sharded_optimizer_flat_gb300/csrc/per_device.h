// What has to be set up once on every device that a kernel is launched on.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace zopt {

// init() on the first call on the current device (a kernel's attributes hold for one device alone), and
// again after a failure; one record per call site (per lambda type, as once() has it). Two threads'
// first calls may both run init(), which has to bear that.
template <typename F>
cudaError_t once_per_device(F init) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;  // (beyond 64 devices: every time)
  if ((done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = init();
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace zopt
