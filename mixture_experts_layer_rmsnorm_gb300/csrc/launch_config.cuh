// launch_config.cuh -- host-side configuration of a kernel that is done once
// per device (function attributes, occupancy queries) and is safe to reach from
// several host threads: each launcher keeps a function-local PerDevice.
#pragma once

#include <cuda_runtime.h>

#include <mutex>

namespace moe {

constexpr int kMaxDevices = 64;

// The result of `make(value)` for the current device, computed on the first
// call for that device; `make` returns the configuration's status and may set
// an int (e.g. an occupancy figure), returned through `out`.
struct PerDevice {
  std::once_flag once[kMaxDevices];
  cudaError_t status[kMaxDevices] = {};
  int value[kMaxDevices] = {};

  template <typename F>
  cudaError_t get(F&& make, int* out = nullptr) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&] { status[dev] = make(value[dev]); });
    if (out) *out = value[dev];
    return status[dev];
  }
};

// Launch `kernel` (programmatic dependent launch) on `ctas` CTAs.  `config`: one per kernel.
template <typename Kernel, typename... Args>
cudaError_t launch_ctas(Kernel kernel, PerDevice& config, int ctas, int threads, size_t smem_bytes,
                        cudaStream_t stream, const Args&... args) {
  const cudaError_t e = config.get([&](int&) -> cudaError_t {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem_bytes));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem_bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr int kMaxPairs = 128;

// Launch `kernel` (programmatic dependent launch) on clusters of two CTAs, as
// many as fit on the device at once, kMaxPairs at most.  `config`: one per kernel.
template <typename Kernel, typename... Args>
cudaError_t launch_pairs(Kernel kernel, PerDevice& config, int threads, size_t smem_bytes, cudaStream_t stream,
                         const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem_bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  int fit = 0;
  const cudaError_t e = config.get(
      [&](int& pairs) -> cudaError_t {
        cudaError_t ce =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem_bytes));
        if (ce != cudaSuccess) return ce;
        cudaLaunchConfig_t q = cfg;
        q.gridDim = dim3(2 * kMaxPairs);
        q.attrs = attr + 1;
        q.numAttrs = 1;
        int n = 0;
        ce = cudaOccupancyMaxActiveClusters(&n, kernel, &q);
        if (ce != cudaSuccess) return ce;
        if (n <= 0) return cudaErrorInvalidConfiguration;
        pairs = n;
        return cudaSuccess;
      },
      &fit);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(2 * (fit < kMaxPairs ? fit : kMaxPairs));
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace moe
