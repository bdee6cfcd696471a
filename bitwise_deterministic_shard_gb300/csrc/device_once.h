// Set-up that a kernel needs once on each device of the process, such as the limit of its dynamic shared memory: that
// limit belongs to a device, so setting it on the first one alone leaves every launch on another refused.
#pragma once
#include <atomic>
#include <cstdint>

namespace detattn {

class DeviceOnce {
  std::atomic<uint64_t> done{0};

 public:
  // setup() == 0 the first time on that device, 0 after it; on a device past the 64 kept ones, or after a failure, again
  // each time.  Threads may meet in it: setup has to allow that, as a limit set twice does.
  template <typename F>
  auto operator()(int device, F setup) -> decltype(setup()) {
    using E = decltype(setup());
    const uint64_t bit = device >= 0 && device < 64 ? (uint64_t)1 << device : 0;
    if (done.load(std::memory_order_acquire) & bit) return (E)0;
    const E e = setup();
    if (e == (E)0) done.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

#if defined(__CUDACC__)
// Allows the kernel `bytes` of dynamic shared memory on the current device.
template <typename K>
cudaError_t allow_smem(DeviceOnce& once, K kernel, int bytes) {
  int device;
  const cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  return once(device, [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
}
#endif

}  // namespace detattn
