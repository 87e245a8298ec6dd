// Launches and device error words of the operators around the decode.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "mla_decode.h"

namespace mla {

// A programmatic dependent launch (the grid is scheduled while the previous
// kernel on the stream drains; the kernel waits for it at its first
// instruction), in clusters of `cluster` CTAs when that is above 1.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), int grid, int threads, size_t smem,
                             int cluster, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// SMs of the current device.
inline cudaError_t current_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  return e == cudaSuccess ? cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) : e;
}

// Status of a call whose kernels record their first error in the __device__
// word `symbol`: with check_status, waits for the stream, reads the word and
// clears it.
inline mla_status_t finish_call(cudaError_t e, const void* symbol, int check_status, cudaStream_t s) {
  int32_t err = 0;
  if (e == cudaSuccess && check_status) {
    e = cudaMemcpyFromSymbolAsync(&err, symbol, sizeof(err), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && err != 0) {
      const int32_t zero = 0;
      e = cudaMemcpyToSymbolAsync(symbol, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
      if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
  }
  if (e != cudaSuccess) {
    cudaGetLastError();   // clear a non-sticky error so later calls start clean
    return MLA_ERR_CUDA;
  }
  return static_cast<mla_status_t>(err);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace mla
