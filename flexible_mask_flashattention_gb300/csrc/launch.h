// Host helpers of calls that launch small kernels many times a second: what a device is asked for once, launches, and the checks
// of alignment and that outputs overlap nothing.
#pragma once

#include <atomic>
#include <cstdint>
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

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Do the byte ranges [a, a + na) and [b, b + nb) meet?
inline bool meet(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

// A range of memory a call reads or writes, in bytes.
struct Span {
  const void* p;
  int64_t n;
};

// Does an output meet an input or another output?
inline bool any_meet(const Span* out, int n_out, const Span* in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (meet(out[i].p, out[i].n, in[j].p, in[j].n)) return true;
    for (int j = i + 1; j < n_out; ++j)
      if (meet(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
  }
  return false;
}

// Bytes from the first to the last value of a strided [tokens][heads][d] bf16 tensor.
inline int64_t span_bytes(int64_t tokens, int64_t stride, int64_t heads, int64_t d) {
  return tokens <= 0 ? 0 : 2 * ((tokens - 1) * stride + heads * d);
}

}  // namespace ffa
