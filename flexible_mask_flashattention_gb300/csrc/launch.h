// Host helpers of calls that launch small kernels many times a second: what a device is asked for once, and launches.
#pragma once

#include <atomic>
#include <cuda_runtime.h>

namespace ffa {

constexpr int kDevices = 64;   // devices whose figures are kept; others are asked each time

// The current device and its SMs; false: a CUDA error.
inline bool current_device(int& device, int& sms) {
  static std::atomic<int> known[kDevices];
  if (cudaGetDevice(&device) != cudaSuccess) return false;
  sms = device < kDevices ? known[device].load(std::memory_order_relaxed) : 0;
  if (sms) return true;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return false;
  if (device < kDevices) known[device].store(sms, std::memory_order_relaxed);
  return true;
}

// Launch a kernel that wants more dynamic shared memory than the default 48 KB.  Its limit is raised before its first launch on a
// device (`raised`, per kernel), and again if a launch is refused: the limit belongs to the context's copy of the
// kernel, which a device reset replaces.
template <typename P>
cudaError_t launch_large(void (*kernel)(P), dim3 grid, unsigned block, int smem, int most, cudaStream_t stream, int device,
                         std::atomic<bool> (&raised)[kDevices], const P& params) {
  for (int attempt = 0;; ++attempt) {
    if (smem > 48 * 1024 && (attempt > 0 || device >= kDevices || !raised[device].load(std::memory_order_acquire))) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (e != cudaSuccess) return e;
      if (device < kDevices) raised[device].store(true, std::memory_order_release);
    }
    kernel<<<grid, block, smem, stream>>>(params);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaErrorInvalidValue || smem <= 48 * 1024 || attempt > 0) return e;
  }
}

// Launch a kernel that may start before the one ahead of it on the stream has ended (it calls wait_for_primary).
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned block, cudaStream_t stream, A... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace ffa
