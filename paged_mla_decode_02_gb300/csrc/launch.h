// Launches and the device error word of the operators around the decode.
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

// The current device's error word, in which the kernels of mla_paging.h record
// the first error.
cudaError_t paging_error_word(int32_t** word);

// Status of a call that queued its kernels with result `e`; with check_status,
// waits for the stream and takes what the error word holds.
mla_status_t finish_call(cudaError_t e, int check_status, cudaStream_t s);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace mla
