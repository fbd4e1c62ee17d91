// saga_launch.cuh - launch helpers of the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdlib.h>

#include <atomic>
#include <utility>

namespace saga {

// Whether kernels are launched with programmatic stream serialization
// (SAGA_PDL=0 in the environment: plain stream order).
inline bool pdl_enabled() {
  static const bool on = [] {
    const char* e = getenv("SAGA_PDL");
    return !(e != nullptr && e[0] == '0');
  }();
  return on;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// cudaFuncSetAttribute holds per device.  Per kernel and device, once (device
// ordinals from 64 on: every time): the dynamic shared memory it may take, and
// the largest shared-memory carveout.  Every kernel of the library asks for the
// same carveout, so an SM running a small kernel (a combine) never has to drain
// and reconfigure before a split CTA of the next call can join it.
inline cudaError_t prepare_kernel(const void* fn, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool tracked = dev >= 0 && dev < 64;
  if (tracked && (done.load(std::memory_order_acquire) >> dev & 1ull)) return cudaSuccess;
  if (bytes > 0) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && tracked) done.fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

}  // namespace saga
