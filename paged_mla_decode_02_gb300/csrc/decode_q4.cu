// Paged MLA decode over a 4-bit cache.
//
// For request b, head h, over the rows k_t of the request's tokens:
//   S = sm_scale * (q_nope . k_t[0:512] + q_pe . k_t[512:576]),
//   out = softmax(S) . k[0:512],  lse = ln sum exp(S).
//
// Simple form: a CTA takes eight query rows of a work unit, a warp each, and
// walks the unit's tokens 32 at a time.  The rows are expanded to fp32 in shared
// memory; lane t makes the score of token t, then holds 16 of the output dims.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_utils.cuh"
#include "kernels.h"
#include "launch.h"
#include "q4.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = kThreads / 32;     // query rows of a CTA
constexpr int kTok = 32;                 // tokens at a time
constexpr int kPitch = kD + 1;           // words between rows: lanes of a column in different banks
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr size_t kSmem = (kTok * kPitch + kRows * kD) * sizeof(float);

template <bool kOutF32>
__global__ void __launch_bounds__(kThreads) decode_q4_kernel(const DecodeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ float sm[];
  float* keys = sm;
  float* query = sm + kTok * kPitch;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PlanDev prm = *a.params;
  const int H = a.num_heads, P = prm.page_size;
  const int groups = (H + kRows - 1) / kRows;
  const int worker = blockIdx.x / groups, h = (blockIdx.x % groups) * kRows + warp;
  const int u0 = worker < prm.n_workers ? a.worker_ptr[worker] : 0;
  const int u1 = worker < prm.n_workers ? a.worker_ptr[worker + 1] : 0;
  const int hide = prm.q_len > 1 && h < H ? prm.q_len - 1 - h / prm.heads_per_token : 0;
  const float c = prm.sm_scale * kLog2e;
  for (int ui = u0; ui < u1; ++ui) {
    const WorkUnit u = a.units[ui];
    __syncthreads();
    if (h < H) {
      const size_t row = static_cast<size_t>(u.req) * H + h;
      for (int d = lane; d < kD; d += 32)
        query[warp * kD + d] = __bfloat162float(d < kDCkv ? static_cast<const __nv_bfloat16*>(a.q_nope)[row * kDCkv + d]
                                                          : static_cast<const __nv_bfloat16*>(a.q_pe)[row * kDKpe + d - kDCkv]);
    }
    float o[kDCkv / 32] = {};
    float top = -INFINITY, sum = 0.f;
    const int end = min(u.tok_end, u.kv_len - hide);
    for (int t0 = u.tok_begin; t0 < u.tok_end; t0 += kTok) {
      __syncthreads();
      for (int i = threadIdx.x; i < kTok * kQ4Words; i += kThreads) {
        const int t = i / kQ4Words, w = i % kQ4Words;
        float x[8] = {};
        float unit = 0.f;
        if (t0 + t < u.tok_end) {
          const int page = a.kv_indices[u.page_base + (t0 + t) / P];
          if (page < 0 || page >= a.num_pages) {
            report_error(a.err, kErrBounds);
          } else {
            const uint8_t* row = static_cast<const uint8_t*>(a.ckv) + (static_cast<size_t>(page) * P + (t0 + t) % P) * kQ4Row;
            q4_expand(reinterpret_cast<const uint32_t*>(row)[w], x);
            unit = q4_unit(Q4Meta{*reinterpret_cast<const uint4*>(row + kQ4Meta)}, w / 4);
          }
        }
#pragma unroll
        for (int d = 0; d < 8; ++d) keys[t * kPitch + 8 * w + d] = x[d] * unit;
      }
      __syncthreads();
      float s = 0.f;
      for (int d = 0; d < kD; ++d) s = fmaf(query[warp * kD + d], keys[lane * kPitch + d], s);
      s = t0 + lane < end ? s * c : -INFINITY;
      float m = s;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, x));
      m = fmaxf(m, top);
      const float base = m == -INFINITY ? 0.f : m, alpha = exp2f(top - base);
      const float p = exp2f(s - base);
      sum = sum * alpha + p;
      top = m;
#pragma unroll
      for (int i = 0; i < kDCkv / 32; ++i) o[i] *= alpha;
      for (int t = 0; t < kTok; ++t) {
        const float w = __shfl_sync(~0u, p, t);
#pragma unroll
        for (int i = 0; i < kDCkv / 32; ++i) o[i] = fmaf(w, keys[t * kPitch + 32 * i + lane], o[i]);
      }
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(~0u, sum, x);
    if (h >= H) continue;
    const bool split = u.out_slot >= 0;
    const size_t row = static_cast<size_t>(u.req) * H + h;
    const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
    if (lane == 0) {
      const float lse = (top + log2f(sum)) * kLn2;
      if (split) a.lse_part[lse_part_offset(u.out_slot, 0, h, H)] = lse;
      else a.lse[row] = lse;
    }
#pragma unroll
    for (int i = 0; i < kDCkv / 32; ++i) {
      const int d = 32 * i + lane;
      if (split) a.o_part[part_offset(u.out_slot, h, d, H)] = o[i] * inv;
      else if (kOutF32) static_cast<float*>(a.out)[row * kDCkv + d] = o[i] * inv;
      else static_cast<__nv_bfloat16*>(a.out)[row * kDCkv + d] = __float2bfloat16(o[i] * inv);
    }
  }
}

}  // namespace

cudaError_t launch_decode_q4(const DecodeArgs& a, bool out_f32, cudaStream_t s) {
  auto kernel = out_f32 ? decode_q4_kernel<true> : decode_q4_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, a.n_workers * ((a.num_heads + kRows - 1) / kRows), kThreads, kSmem, 1, s, a);
}

}  // namespace mla
