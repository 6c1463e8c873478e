// What belongs to a device and not to the process (its multiprocessors, a
// kernel's shared-memory attribute or occupancy), kept by device ordinal.
#pragma once
#include <cuda_runtime_api.h>

#include <atomic>

namespace dfl {

class PerDevice {
 public:
  static constexpr int kDevices = 64;
  // The current device's value, above 0: found by `find(device, &value)` at
  // its first call on the device and kept.  What fails, or finds nothing, is
  // not kept; devices past the table are asked every time.  Calls at the same
  // time may each find it.
  template <typename F>
  cudaError_t get(int* value, F find) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool held = dev >= 0 && dev < kDevices;
    int v = held ? v_[dev].load(std::memory_order_acquire) : 0;
    if (v <= 0) {
      e = find(dev, &v);
      if (e != cudaSuccess) return e;
      if (held && v > 0) v_[dev].store(v, std::memory_order_release);
    }
    *value = v;
    return cudaSuccess;
  }
  // `set()` once a device.
  template <typename F>
  cudaError_t once(F set) {
    int done;
    return get(&done, [&](int, int* v) {
      *v = 1;
      return set();
    });
  }

 private:
  std::atomic<int> v_[kDevices] = {};
};

}  // namespace dfl
