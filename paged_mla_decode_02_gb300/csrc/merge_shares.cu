// The shares of split requests into one state each, after the 4-bit decode:
//   M = max_i lse_i,  w_i = exp(lse_i - M),
//   out = sum_i w_i O_i / sum_i w_i,   lse = M + ln sum_i w_i;
// a request without tokens gets out = 0, lse = -inf, and a NaN share makes both NaN.
//
// A block takes 8 dims of some query rows of a request at a time: 2 lanes a row
// (four dims each), and as many groups of threads as make it 256, which take the
// shares in turn and are joined in their order.  How many groups follows from the
// shares that a request has on average: many shares of few requests are read in
// parallel, few shares of many requests by as many rows.  4 requests of 38 shares,
// 64 rows: 11.4 us from a cold start, 18 MB, where a thread for all shares of a row
// took 19.5.  Bound by the latency of its reads, the plan's first (read while the
// decode ends) and then the shares, which L2 mostly holds.
#include <cuda_bf16.h>

#include "device_utils.cuh"
#include "kernels.h"
#include "launch.h"

namespace mla {
namespace {

constexpr int kThreads = 256;
// Registers for the reads of kAhead shares against rows in flight: of the whole decode of
// 4 requests of 38 shares and 64 rows, 47.7 us with 4 blocks an SM, 51.6 with 6, 51.4
// with 2; of 128 ragged requests of 128 rows 195.4, 197.5 and 203.3.
constexpr int kBlocksPerSm = 4;
constexpr int kAhead = 4;      // shares that a thread reads at once
constexpr int kMinRows = 16;   // of a block

template <bool kOutF32>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) merge_shares_kernel(const MergeArgs a) {
  __shared__ float4 s_sum[kThreads];
  __shared__ float2 s_mw[kThreads];
  // The plan's arrays were uploaded before the decode ahead began: read while it ends.
  // (of a plan of other rows, as a replay may meet, the decode leaves nothing to merge)
  const int H = a.num_heads, n_merge = a.params->num_heads == H ? a.params->n_merge : 0;
  // rows of a block: a power of two that leaves a group for every kAhead shares
  const int shares = n_merge > 0 ? (a.params->n_slots + n_merge - 1) / n_merge : 0;
  int rows = kThreads / 2;
  while (rows > kMinRows && (kThreads / 2 / rows * kAhead < shares || rows / 2 >= H)) rows /= 2;
  const int groups = kThreads / 2 / rows;
  const int row_blocks = (H + rows - 1) / rows;
  const int per_entry = row_blocks * (kDCkv / 8);
  const int half = threadIdx.x & 1, row = (threadIdx.x >> 1) % rows, group = (threadIdx.x >> 1) / rows;
  MergeEntry me{};
  if (static_cast<int>(blockIdx.x) < n_merge * per_entry) me = a.merge[blockIdx.x / per_entry];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int item = blockIdx.x; item < n_merge * per_entry; item += gridDim.x) {
    if (item != static_cast<int>(blockIdx.x)) me = a.merge[item / per_entry];
    const int h = item % per_entry / (kDCkv / 8) * rows + row, d = item % (kDCkv / 8) * 8 + 4 * half;
    float M = -INFINITY, W = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    // A state of weight w.  Not one without tokens (w = 0): m would not be a number above
    // -inf.  A NaN share leaves M as it was, maybe -inf, and makes W NaN.
    auto add = [&](float m, float w, const float4& o) {
      const float top = fmaxf(M, m);
      const float x = __expf(M - top), y = __expf(m - top);   // a NaN stays one in W and the sums
      sum = make_float4(sum.x * x + o.x * y, sum.y * x + o.y * y, sum.z * x + o.z * y, sum.w * x + o.w * y);
      W = W * x + w * y;
      M = top;
    };
    if (h < H) {
      for (int i0 = group; i0 < me.n_slots; i0 += groups * kAhead) {
        float4 o[kAhead];
        float l[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int i = i0 + groups * j;
          l[j] = -INFINITY;
          if (i < me.n_slots) {
            o[j] = *reinterpret_cast<const float4*>(a.o_part + part_offset(me.first_slot + i, h, d, H));
            l[j] = a.lse_part[lse_part_offset(me.first_slot + i, 0, h, H)];
          }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (l[j] != -INFINITY) add(l[j], 1.f, o[j]);
      }
    }
    if (groups > 1) {
      s_sum[threadIdx.x] = sum;
      s_mw[threadIdx.x] = make_float2(M, W);
      __syncthreads();
      if (group == 0)
        for (int g = 1; g < groups; ++g) {
          const float2 mw = s_mw[threadIdx.x + 2 * rows * g];
          const float4 o = s_sum[threadIdx.x + 2 * rows * g];
          if (mw.y != 0.f) add(mw.x, mw.y, o);
        }
      __syncthreads();
    }
    if (group == 0 && h < H && me.req < a.batch) {
      const float inv = W == 0.f ? 0.f : 1.f / W;
      const size_t at = (static_cast<size_t>(me.req) * H + h) * kDCkv + d;
      if (kOutF32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
      else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
            make_uint2(pack_bf16x2(sum.x * inv, sum.y * inv), pack_bf16x2(sum.z * inv, sum.w * inv));
      if (d == 0) a.lse[static_cast<size_t>(me.req) * H + h] = W == 0.f ? -INFINITY : M + logf(W);
    }
  }
}

}  // namespace

cudaError_t launch_merge_shares(const MergeArgs& a, bool out_f32, int num_sms, cudaStream_t s) {
  if (a.merge_cap <= 0) return cudaSuccess;
  const long long items = static_cast<long long>(a.merge_cap) * (kDCkv / 8) * ((a.num_heads + kMinRows - 1) / kMinRows);
  const int grid = static_cast<int>(items < kBlocksPerSm * num_sms ? items : kBlocksPerSm * num_sms);
  return launch_dependent(out_f32 ? merge_shares_kernel<true> : merge_shares_kernel<false>, grid, kThreads, 0, 1, s, a);
}

}  // namespace mla
