// The device error word of the operators around the decode (mla_paging.h).
//
// One word for all of them: a step queues several and checks once, through
// any.  Each kernel gets its address as an argument, since a device variable
// belongs to one translation unit.  A check takes the word and clears it in one
// exchange, so an error that another stream's kernel records meanwhile is
// either in what the check returns or left for the next one.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "launch.h"

namespace mla {
namespace {

__device__ int32_t g_paging_err;   // first device error since the last check

constexpr unsigned kTaken = 256;   // checks that may be under way at once
__device__ int32_t g_taken[kTaken];

__global__ void take_error_kernel(unsigned place) { g_taken[place] = atomicExch(&g_paging_err, 0); }

}  // namespace

cudaError_t paging_error_word(int32_t** word) {
  constexpr int kDevices = 64;
  static std::atomic<int32_t*> known[kDevices];   // a device variable stays where its module was loaded
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kDevices && (*word = known[dev].load(std::memory_order_relaxed))) return cudaSuccess;
  void* p = nullptr;
  e = cudaGetSymbolAddress(&p, g_paging_err);
  if (e != cudaSuccess) return e;
  *word = static_cast<int32_t*>(p);
  if (dev < kDevices) known[dev].store(*word, std::memory_order_relaxed);
  return cudaSuccess;
}

mla_status_t finish_call(cudaError_t e, int check_status, cudaStream_t s) {
  int32_t err = 0;
  if (e == cudaSuccess && check_status) {
    static std::atomic<unsigned> turn;
    const unsigned place = turn.fetch_add(1, std::memory_order_relaxed) % kTaken;
    take_error_kernel<<<1, 1, 0, s>>>(place);
    e = cudaGetLastError();
    if (e == cudaSuccess)
      e = cudaMemcpyFromSymbolAsync(&err, g_taken, sizeof(err), place * sizeof(err), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();   // clear a non-sticky error so later calls start clean
    return MLA_ERR_CUDA;
  }
  return static_cast<mla_status_t>(err);
}

}  // namespace mla
