// Host-side pieces shared by the library's translation units: the calling
// thread's last error and launch count, device queries and the tensor-map
// encoder.  Defined in dsa_indexer.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>

namespace dsa_host {

// Records the message of a failing call and returns its code.
int fail(int code, const char* fmt, ...);
// DSA_OK, or DSA_ERR_CUDA with the pending launch error's message.
int check_launch(const char* what);
// SMs of the current device (0 without one).
int sm_count();

// Does something once for each device that is current at a call (again where it
// failed): a kernel's attributes belong to a device, not to the process.
class PerDevice {
 public:
  template <typename F>
  cudaError_t once(F set) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kDevices;
    if (known && done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = set();
    if (e == cudaSuccess && known) done_[dev].store(true, std::memory_order_release);
    return e;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<bool> done_[kDevices] = {};
};
// Allows `kernel` that many bytes of dynamic shared memory; `done` is the kernel's own.
int allow_smem(PerDevice& done, const void* kernel, int bytes);

// An integer from the environment, within [lo, hi]; `dflt` where it is not set.
int env_int(const char* name, int dflt, int lo, int hi);
// The driver's cuTensorMapEncodeTiled, or null.
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();
// The value dsa_last_launch_count() reports.
void set_last_launches(int n);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace dsa_host
