// The new tokens of a step into the paged cache: mla_rope_append (rotary
// embedding of queries and rope keys, RMS norm of the latent rows, write) and
// mla_summarize_pages (mean rows of the pages just completed).
//
// Rotation: pair i of a row turns by pos * f_i radians.  Far positions need
// that product modulo one turn to more bits than fp32 has, so the host turns
// f_i into a 64-bit fixed-point fraction of a turn, F_i = f_i / 2 pi * 2^64,
// and the kernel multiplies pos * F_i in wrapping 64-bit integers: the whole
// turns fall off the top exactly, and the product is off by at most |pos|
// units of 2^-64 turns.  Its upper 32 bits, signed, are the angle in
// [-1/2, 1/2) turns that sincospi takes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "device_utils.cuh"
#include "launch.h"
#include "mla_internal.h"
#include "mla_paging.h"

namespace mla {
namespace {

__device__ int32_t g_append_err;   // first device error of this file's kernels

constexpr int kPairs = kDKpe / 2;
constexpr int kMaxAxes = 8;
constexpr int kQThreads = 256;
constexpr int kKvWarps = 8;

struct RopeDev {
  uint64_t turn[kPairs];     // f_i / 2 pi as a fraction of 2^64
  uint8_t axis[kPairs];
  float scale;
};

struct AppendArgs {
  RopeDev rope;
  const int32_t* positions;
  int64_t axis_stride;
  const int64_t* slots;
  const __nv_bfloat16* q;
  int64_t q_token_stride, q_head_stride;
  __nv_bfloat16* q_out;
  const __nv_bfloat16* ckv;
  int64_t ckv_stride;
  const __nv_bfloat16* kpe;
  int64_t kpe_stride;
  const __nv_bfloat16* weight;
  float eps;
  void* ckv_cache;
  void* kpe_cache;
  float inv_scale;           // 1 / kv_scale (1 for a bf16 cache)
  int64_t cache_slots;       // num_pages * page_size
  int64_t tokens;
  int heads;
  int64_t q_blocks;
};

__device__ __forceinline__ float2 cos_sin(const AppendArgs& a, int pair, int64_t t) {
  const int pos = a.positions[a.rope.axis[pair] * a.axis_stride + t];
  const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * a.rope.turn[pair];
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, &s, &c);
  return make_float2(c * a.rope.scale, s * a.rope.scale);
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// Eight values rounded to the cache's type at element offset `at`.  e4m3
// saturates at +-448; NaN stays NaN.
template <bool kFp8>
__device__ __forceinline__ void store8(void* cache, int64_t at, const float (&x)[8]) {
  if (kFp8) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | hi << 16;
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + at) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(cache) + at) = pack8(x);
  }
}

// A quarter of a 64-wide row: the 16-byte chunks c and c + 4 (dims 8c.. and
// 32 + 8c..), which hold eight whole pairs in either layout.
template <bool kInterleaved>
__device__ __forceinline__ int pair_of(int part, int k) {
  return kInterleaved ? (k < 4 ? 4 * part + k : 16 + 4 * part + k - 4) : 8 * part + k;
}
template <bool kInterleaved>
__device__ __forceinline__ void rotate(float (&lo)[8], float (&hi)[8], const float2 (&cs)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float& x = kInterleaved ? (k < 4 ? lo[2 * k] : hi[2 * k - 8]) : lo[k];
    float& y = kInterleaved ? (k < 4 ? lo[2 * k + 1] : hi[2 * k - 7]) : hi[k];
    const float u = x * cs[k].x - y * cs[k].y, v = x * cs[k].y + y * cs[k].x;
    x = u;
    y = v;
  }
}

template <bool kInterleaved, bool kFp8>
__global__ void __launch_bounds__(kQThreads) append_kernel(const __grid_constant__ AppendArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x < a.q_blocks) {
    // queries: four threads per (token, head) row
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x;
    const int part = static_cast<int>(i & 3);
    const int64_t row = i >> 2, t = row / a.heads;
    if (t >= a.tokens) return;
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.cache_slots) return;
    const __nv_bfloat16* src = a.q + t * a.q_token_stride + (row - t * a.heads) * a.q_head_stride + 8 * part;
    float lo[8], hi[8];
    unpack8(*reinterpret_cast<const uint4*>(src), lo);
    unpack8(*reinterpret_cast<const uint4*>(src + 32), hi);
    float2 cs[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) cs[k] = cos_sin(a, pair_of<kInterleaved>(part, k), t);
    rotate<kInterleaved>(lo, hi, cs);
    __nv_bfloat16* dst = a.q_out + row * kDKpe + 8 * part;
    *reinterpret_cast<uint4*>(dst) = pack8(lo);
    *reinterpret_cast<uint4*>(dst + 32) = pack8(hi);
    return;
  }
  // keys: one warp per token
  const int64_t t = (blockIdx.x - a.q_blocks) * kKvWarps + warp;
  if (t >= a.tokens) return;
  const int64_t slot = a.slots[t];
  if (slot < 0) return;
  if (slot >= a.cache_slots) {
    if (lane == 0) report_error(&g_append_err, kErrBounds);
    return;
  }
  const __nv_bfloat16* src = a.ckv + t * a.ckv_stride;
  float x[2][8];
  float sq = 0.f;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    unpack8(*reinterpret_cast<const uint4*>(src + 256 * j + 8 * lane), x[j]);
#pragma unroll
    for (int k = 0; k < 8; ++k) sq += x[j][k] * x[j][k];
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sq += __shfl_xor_sync(~0u, sq, d);
  const float r = a.weight ? rsqrtf(sq * (1.f / kDCkv) + a.eps) : 1.f;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (a.weight) {
      float w[8];
      unpack8(*reinterpret_cast<const uint4*>(a.weight + 256 * j + 8 * lane), w);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[j][k] *= r * w[k];
    }
    if (kFp8) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[j][k] *= a.inv_scale;
    }
    store8<kFp8>(a.ckv_cache, slot * kDCkv + 256 * j + 8 * lane, x[j]);
  }
  if (lane < 4) {
    float lo[8], hi[8];
    const __nv_bfloat16* ks = a.kpe + t * a.kpe_stride + 8 * lane;
    unpack8(*reinterpret_cast<const uint4*>(ks), lo);
    unpack8(*reinterpret_cast<const uint4*>(ks + 32), hi);
    float2 cs[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      cs[k] = cos_sin(a, pair_of<kInterleaved>(lane, k), t);
      if (kFp8) {
        cs[k].x *= a.inv_scale;
        cs[k].y *= a.inv_scale;
      }
    }
    rotate<kInterleaved>(lo, hi, cs);
    store8<kFp8>(a.kpe_cache, slot * kDKpe + 8 * lane, lo);
    store8<kFp8>(a.kpe_cache, slot * kDKpe + 8 * lane + 32, hi);
  }
}

// ---------------------------------------------------------------------------
// Page summaries
// ---------------------------------------------------------------------------
constexpr int kSumThreads = 288;   // 72 eight-dim columns x 4 row groups

struct SummarizeArgs {
  const int64_t* slots;
  int64_t tokens;
  const void* ckv;
  const void* kpe;
  float scale;               // kv_scale / page_size
  int64_t cache_slots;
  int page_shift;
  __nv_bfloat16* summaries;
};

template <bool kFp8>
__device__ __forceinline__ void load8(const void* cache, int64_t at, float (&x)[8]) {
  if (kFp8) {
    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + at);
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b2 = e4m3x2_to_bf16x2(static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1))));
      x[2 * i] = __uint_as_float(b2 << 16);
      x[2 * i + 1] = __uint_as_float(b2 & 0xffff0000u);
    }
  } else {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(cache) + at), x);
  }
}

template <bool kFp8>
__global__ void __launch_bounds__(kSumThreads) summarize_kernel(const SummarizeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int P = 1 << a.page_shift;
  const int64_t slot = a.slots[blockIdx.x];
  if (slot < 0) return;
  if (slot >= a.cache_slots) {
    if (threadIdx.x == 0) report_error(&g_append_err, kErrBounds);
    return;
  }
  if ((slot & (P - 1)) != P - 1) return;
  __shared__ float part[3][kD];
  const int64_t first = slot - (P - 1);
  const int group = threadIdx.x / 72, col = (threadIdx.x % 72) * 8;
  float sum[8] = {};
  for (int r = group; r < P; r += 4) {
    float x[8];
    if (col < kDCkv) load8<kFp8>(a.ckv, (first + r) * kDCkv + col, x);
    else load8<kFp8>(a.kpe, (first + r) * kDKpe + col - kDCkv, x);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] += x[k];
  }
  if (group) {
#pragma unroll
    for (int k = 0; k < 8; ++k) part[group - 1][col + k] = sum[k];
  }
  __syncthreads();
  if (group) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) sum[k] = (sum[k] + part[0][col + k] + part[1][col + k] + part[2][col + k]) * a.scale;
  *reinterpret_cast<uint4*>(a.summaries + (slot >> a.page_shift) * kD + col) = pack8(sum);
}

bool cache_args(const void* ckv_cache, const void* kpe_cache, int kv_dtype, float kv_scale, int num_pages,
                int page_size, mla_status_t* st) {
  *st = MLA_ERR_INVALID_ARG;
  if (!ckv_cache || !kpe_cache || !aligned16(ckv_cache) || !aligned16(kpe_cache) || num_pages < 1 || page_size < 1)
    return false;
  if (!std::isfinite(kv_scale) || kv_scale <= 0.f || !std::isfinite(1.f / kv_scale)) return false;
  *st = MLA_ERR_UNSUPPORTED;
  if (kv_dtype != MLA_DTYPE_BF16 && kv_dtype != MLA_DTYPE_FP8_E4M3) return false;
  return page_size == 16 || page_size == 32 || page_size == 64;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status_t mla_rope_append(const mla_rope_t* rope, const int32_t* positions, int64_t axis_stride,
                                        const int64_t* slots, const void* q_pe, int64_t q_token_stride,
                                        int64_t q_head_stride, void* q_pe_out, const void* ckv, int64_t ckv_stride,
                                        const void* kpe, int64_t kpe_stride, const void* norm_weight, float eps,
                                        void* ckv_cache, void* kpe_cache, int kv_dtype, float kv_scale, int num_pages,
                                        int page_size, int64_t tokens, int num_heads, int check_status, void* stream) {
  mla_status_t st;
  if (!rope || rope->n_axes < 1 || rope->n_axes > kMaxAxes || !std::isfinite(rope->scale)) return MLA_ERR_INVALID_ARG;
  if (!cache_args(ckv_cache, kpe_cache, kv_dtype, kv_scale, num_pages, page_size, &st)) return st;
  if (tokens < 0 || num_heads < 0 || num_heads > 1024 || axis_stride < 0 || !std::isfinite(eps) || eps < 0.f)
    return MLA_ERR_INVALID_ARG;
  if (tokens > (1ll << 24)) return MLA_ERR_CAPACITY;   // keeps the grid inside its limit
  AppendArgs a{};
  for (int i = 0; i < kPairs; ++i) {
    if (rope->axis_of_pair[i] < 0 || rope->axis_of_pair[i] >= rope->n_axes || !std::isfinite(rope->inv_freq[i]))
      return MLA_ERR_INVALID_ARG;
    const double turns = rope->inv_freq[i] * 0.15915494309189533577;   // 1 / 2 pi
    double part = turns - std::floor(turns);                          // whole turns per position fall away
    if (part >= 1.0) part = 0.0;                                      // a tiny negative frequency rounds up to one
    a.rope.turn[i] = static_cast<uint64_t>(std::ldexp(part, 64));
    a.rope.axis[i] = static_cast<uint8_t>(rope->axis_of_pair[i]);
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (tokens > 0) {
    if (!positions || !slots || !ckv || !kpe || (num_heads > 0 && (!q_pe || !q_pe_out))) return MLA_ERR_INVALID_ARG;
    if (!aligned16(ckv) || !aligned16(kpe) || !aligned16(q_pe) || !aligned16(q_pe_out) || !aligned16(norm_weight) ||
        (ckv_stride | kpe_stride | q_token_stride | q_head_stride) & 7)
      return MLA_ERR_INVALID_ARG;
  }
  const bool fp8 = kv_dtype == MLA_DTYPE_FP8_E4M3;
  a.rope.scale = rope->scale;
  a.positions = positions;
  a.axis_stride = axis_stride;
  a.slots = slots;
  a.q = static_cast<const __nv_bfloat16*>(q_pe);
  a.q_token_stride = q_token_stride;
  a.q_head_stride = q_head_stride;
  a.q_out = static_cast<__nv_bfloat16*>(q_pe_out);
  a.ckv = static_cast<const __nv_bfloat16*>(ckv);
  a.ckv_stride = ckv_stride;
  a.kpe = static_cast<const __nv_bfloat16*>(kpe);
  a.kpe_stride = kpe_stride;
  a.weight = static_cast<const __nv_bfloat16*>(norm_weight);
  a.eps = eps;
  a.ckv_cache = ckv_cache;
  a.kpe_cache = kpe_cache;
  a.inv_scale = fp8 ? 1.f / kv_scale : 1.f;
  a.cache_slots = static_cast<int64_t>(num_pages) * page_size;
  a.tokens = tokens;
  a.heads = num_heads > 0 ? num_heads : 1;
  a.q_blocks = (tokens * num_heads * 4 + kQThreads - 1) / kQThreads;
  cudaError_t e = cudaSuccess;
  if (tokens > 0) {
    const int grid = static_cast<int>(a.q_blocks + (tokens + kKvWarps - 1) / kKvWarps);
    auto kernel = rope->interleaved ? (fp8 ? append_kernel<true, true> : append_kernel<true, false>)
                                    : (fp8 ? append_kernel<false, true> : append_kernel<false, false>);
    e = launch_dependent(kernel, grid, kQThreads, 0, 1, s, a);
  }
  return finish_call(e, &g_append_err, check_status, s);
}

extern "C" mla_status_t mla_summarize_pages(const int64_t* slots, int64_t tokens, const void* ckv_cache,
                                            const void* kpe_cache, int kv_dtype, float kv_scale, int num_pages,
                                            int page_size, void* summaries, int check_status, void* stream) {
  mla_status_t st;
  if (!cache_args(ckv_cache, kpe_cache, kv_dtype, kv_scale, num_pages, page_size, &st)) return st;
  if (tokens < 0 || !summaries || !aligned16(summaries) || (tokens > 0 && !slots)) return MLA_ERR_INVALID_ARG;
  if (tokens > (1ll << 24)) return MLA_ERR_CAPACITY;
  SummarizeArgs a{};
  a.slots = slots;
  a.tokens = tokens;
  a.ckv = ckv_cache;
  a.kpe = kpe_cache;
  a.scale = (kv_dtype == MLA_DTYPE_FP8_E4M3 ? kv_scale : 1.f) / static_cast<float>(page_size);
  a.cache_slots = static_cast<int64_t>(num_pages) * page_size;
  a.page_shift = page_size == 16 ? 4 : page_size == 32 ? 5 : 6;
  a.summaries = static_cast<__nv_bfloat16*>(summaries);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (tokens > 0)
    e = launch_dependent(kv_dtype == MLA_DTYPE_FP8_E4M3 ? summarize_kernel<true> : summarize_kernel<false>,
                         static_cast<int>(tokens), kSumThreads, 0, 1, s, a);
  return finish_call(e, &g_append_err, check_status, s);
}
