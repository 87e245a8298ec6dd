// The new tokens of a step into the paged cache: mla_rope_append (rotary
// embedding of queries and rope keys, RMS norm of the latent rows, write) and
// mla_summarize_pages (mean rows of the pages just completed).
//
// Rotation: pair i of a row turns by pos * f_i radians.  Far positions need
// that product modulo one turn to more bits than fp32 has, so the host turns
// f_i into a 64-bit fixed-point fraction of a turn, F_i = f_i / 2 pi * 2^64,
// good to two units for |f_i| up to 2^40 (fraction_of_turn), and the kernel
// multiplies pos * F_i in wrapping 64-bit integers: the whole turns fall off the
// top exactly, and the product is off by at most 2 |pos| units of 2^-64 turns,
// 2^-32 turns at the largest.  Its upper 32 bits, signed, are the angle in
// [-1/2, 1/2) turns that sincospi takes: off by less than 2^-31 turns with what
// lies below them, where fp32 itself, which holds 24 bits of it, is off by 2^-26.
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

constexpr int kPairs = kDKpe / 2;
constexpr int kMaxAxes = 8;
constexpr int kQThreads = 256;
constexpr int kKvWarps = kQThreads / 32;
constexpr int kRowsPerBlock = 256;  // query rows of a CTA, where there are plenty
constexpr int64_t kManyRows = 152 * 4 * kRowsPerBlock;   // a CTA for each place on the GPU
constexpr int kMostTokens = 32;     // tokens of a CTA's queries

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
  int32_t* err;
  int64_t cache_slots;       // num_pages * page_size
  int64_t tokens;
  int heads;
  int tokens_per_block;      // of a CTA's queries
  int64_t kv_blocks;
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

// Two values of a cached row at element offset `at` (even).
template <bool kFp8>
__device__ __forceinline__ void store2(void* cache, int64_t at, float x, float y) {
  if (kFp8)
    *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(cache) + at) =
        __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
  else
    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(cache) + at) = pack_bf16x2(x, y);
}
template <bool kFp8>
__device__ __forceinline__ void store1(void* cache, int64_t at, float x) {
  if (kFp8)
    static_cast<uint8_t*>(cache)[at] = __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
  else
    static_cast<__nv_bfloat16*>(cache)[at] = __float2bfloat16_rn(x);
}

// The first CTAs take the keys, a warp per token; the others the queries of a
// few tokens each.  A token's 32 angles are shared by all of its heads: a CTA
// makes them once, into shared memory, while its first reads are under way,
// and then is bound by reading and writing the rows (a thread turns a quarter
// of a row, 32 bytes each way): 8190 tokens x 128 heads, 283 MB in 48.0 us,
// 5.9 TB/s.
template <bool kInterleaved, bool kFp8>
__global__ void __launch_bounds__(kQThreads, 4) append_kernel(const __grid_constant__ AppendArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x >= a.kv_blocks) {
    // ---------------- queries ----------------
    __shared__ __align__(16) float2 turns[kMostTokens][kPairs];   // read two at a time
    __shared__ bool real[kMostTokens];
    const int64_t t0 = (blockIdx.x - a.kv_blocks) * a.tokens_per_block;
    const int n = static_cast<int>(a.tokens - t0 < a.tokens_per_block ? a.tokens - t0 : a.tokens_per_block);
    const int units = n * a.heads * 4, part = tid & 3;
    auto place = [&](int u, int& t, int& h) {   // quarter u: of token t0 + t, head h
      t = (u >> 2) / a.heads;
      h = (u >> 2) - t * a.heads;
    };
    auto src = [&](int t, int h) {
      return reinterpret_cast<const uint4*>(a.q + (t0 + t) * a.q_token_stride + h * a.q_head_stride + 8 * part);
    };
    constexpr int kAhead = kRowsPerBlock * 4 / kQThreads;   // units read before they are turned
    uint4 lo[kAhead], hi[kAhead];
    auto read = [&](int u0) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int u = u0 + k * kQThreads;
        int t, h;
        if (u < units) {
          place(u, t, h);
          lo[k] = src(t, h)[0];
          hi[k] = src(t, h)[4];
        }
      }
    };
    read(tid);
    for (int i = tid; i < n * kPairs; i += kQThreads) turns[i / kPairs][i % kPairs] = cos_sin(a, i % kPairs, t0 + i / kPairs);
    if (tid < n) {
      const int64_t slot = a.slots[t0 + tid];
      real[tid] = slot >= 0 && slot < a.cache_slots;   // (one past the cache is reported with its key)
    }
    __syncthreads();
    for (int u0 = tid; u0 < units; u0 += kAhead * kQThreads) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int u = u0 + k * kQThreads;
        if (u >= units) break;
        int t, h;
        place(u, t, h);
        float x[8], y[8];
        unpack8(lo[k], x);
        unpack8(hi[k], y);
        float2 cs[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float4 two = *reinterpret_cast<const float4*>(&turns[t][pair_of<kInterleaved>(part, j)]);
          cs[j] = make_float2(two.x, two.y);
          cs[j + 1] = make_float2(two.z, two.w);
        }
        rotate<kInterleaved>(x, y, cs);
        if (real[t]) {
          uint4* dst = reinterpret_cast<uint4*>(a.q_out + ((t0 + t) * a.heads + h) * kDKpe + 8 * part);
          dst[0] = pack8(x);
          dst[4] = pack8(y);
        }
      }
      read(u0 + kAhead * kQThreads);
    }
    return;
  }
  // ---------------- keys ----------------
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kKvWarps + warp;
  if (t >= a.tokens) return;
  const int64_t slot = a.slots[t];
  const __nv_bfloat16* src = a.ckv + t * a.ckv_stride;
  float x[2][8];
#pragma unroll
  for (int j = 0; j < 2; ++j) unpack8(*reinterpret_cast<const uint4*>(src + 256 * j + 8 * lane), x[j]);
  const __nv_bfloat16* ks = a.kpe + t * a.kpe_stride;
  const int e0 = kInterleaved ? 2 * lane : lane, e1 = kInterleaved ? e0 + 1 : lane + 32;   // this lane's pair
  const float k0 = __bfloat162float(ks[e0]), k1 = __bfloat162float(ks[e1]);
  const float2 cs = cos_sin(a, lane, t);
  if (slot < 0) return;
  if (slot >= a.cache_slots) {
    if (lane == 0) report_error(a.err, kErrBounds);
    return;
  }
  float r = 1.f;
  if (a.weight) {
    auto mean_square = [&]() {
      float sq = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) sq += x[j][k] * x[j][k];
#pragma unroll
      for (int d = 16; d; d >>= 1) sq += __shfl_xor_sync(~0u, sq, d);
      return sq * (1.f / kDCkv);
    };
    float eps = a.eps, of = mean_square() + eps;
    if (of < 0x1p-100f || of == INFINITY) {   // squares that fp32 does not hold: of the row times a power of two
      const float up = of < 1.f ? 0x1p100f : 0x1p-100f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) x[j][k] *= up;
      eps = eps * up * up;
      of = mean_square() + eps;
    }
    r = rsqrtf(of);
  }
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
  const float c = cs.x * a.inv_scale, s = cs.y * a.inv_scale;
  const float u = k0 * c - k1 * s, v = k0 * s + k1 * c;
  if (kInterleaved) {
    store2<kFp8>(a.kpe_cache, slot * kDKpe + e0, u, v);
  } else {
    store1<kFp8>(a.kpe_cache, slot * kDKpe + e0, u);
    store1<kFp8>(a.kpe_cache, slot * kDKpe + e1, v);
  }
}

// ---------------------------------------------------------------------------
// Page summaries
// ---------------------------------------------------------------------------
constexpr int kSumThreads = 32 * (kD / 64);   // a warp for each 64 dims of a row
// CTAs of an SM, all resident: one wave, no CTA waits for another's end (65500
// tokens in bf16: 14.3 us with four, 16.5 with three; 131000 in e4m3, whose
// threads sum more dims: 15.2 with three, 15.8 with four)
__host__ __device__ constexpr int sum_blocks(bool fp8) { return fp8 ? 3 : 4; }

struct SummarizeArgs {
  const int64_t* slots;
  int64_t tokens;
  const void* ckv;
  const void* kpe;
  float scale;               // kv_scale / page_size
  int64_t cache_slots;
  int page_shift;
  __nv_bfloat16* summaries;
  int32_t* err;
  int per_block;             // tokens a CTA looks at
};

// sum + v in fp32, v the bits of an fp16 or bf16 value: one instruction, where
// a conversion and an addition are two (131000 tokens, e4m3: 15.7 us with those).
template <bool kHalf>
__device__ __forceinline__ void add_wide(float& sum, unsigned short v) {
  if (kHalf) asm("add.rn.f32.f16 %0, %1, %0;" : "+f"(sum) : "h"(v));
  else asm("add.rn.f32.bf16 %0, %1, %0;" : "+f"(sum) : "h"(v));
}

// Sixteen bytes of a cached row added in fp32: 8 bf16 or 16 e4m3 values.
template <bool kFp8, int N>
__device__ __forceinline__ void add_values(float (&sum)[N], const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (kFp8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
      add_wide<true>(sum[2 * i], h.x);
      add_wide<true>(sum[2 * i + 1], h.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      add_wide<false>(sum[2 * i], w[i] & 0xffffu);
      add_wide<false>(sum[2 * i + 1], w[i] >> 16);
    }
  }
}

// A CTA looks at a run of tokens; for each that completes a page, warp w sums
// dims 64 w .. 64 w + 63 of the page's rows: 16 bytes of a row to a lane, so 4
// (bf16) or 8 (e4m3) rows to a load.  The rows' partial sums meet in the warp
// by halves: at each step a lane passes on half of its dims and adds what it
// gets to the other half, down to two.  The warps of a CTA read the same rows
// at about the same time, and each has the next four loads under way while it
// adds the last; two pages share them where one has rows for two only (kPair:
// e4m3, 16 tokens).  Bound by HBM for long prompts (131000 tokens, e4m3,
// 32-token pages: 81 MB in 15.2 us, 5.3 TB/s; 16-token pages 15.8, a page at a
// time 20.7).
template <bool kFp8, bool kPair>
__global__ void __launch_bounds__(kSumThreads, sum_blocks(kFp8)) summarize_kernel(const SummarizeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kDims = kFp8 ? 16 : 8, kLanes = 64 / kDims, kRows = 32 / kLanes, kLoads = 4;
  constexpr int kOfPage = kPair ? kLoads / 2 : kLoads;   // loads of a page at a time
  __shared__ int pages[kSumThreads], n;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = 1 << a.page_shift, row0 = lane / kLanes, col = (lane % kLanes) * kDims;
  // the pages that this run of tokens completes, in any order
  if (threadIdx.x == 0) n = 0;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * a.per_block + threadIdx.x;
  const int64_t slot = static_cast<int>(threadIdx.x) < a.per_block && t < a.tokens ? a.slots[t] : -1;
  __syncthreads();
  if (slot >= a.cache_slots) report_error(a.err, kErrBounds);
  else if (slot >= 0 && (slot & (P - 1)) == P - 1) pages[atomicAdd(&n, 1)] = static_cast<int>(slot >> a.page_shift);
  __syncthreads();
  // their rows, kLoads loads of kRows at a time
  const bool pe = warp == kSumThreads / 32 - 1;
  const int width = (pe ? kDKpe : kDCkv) * (kFp8 ? 1 : 2);   // bytes of a row
  const char* rows = static_cast<const char*>(pe ? a.kpe : a.ckv) + ((pe ? 0 : 64 * warp) + col) * (kFp8 ? 1 : 2);
  const int batches = P / (kRows * kOfPage);   // of a page
  uint4 next[kLoads];
  auto read = [&](int i, int batch) {
#pragma unroll
    for (int k0 = 0; k0 < kLoads; k0 += kOfPage) {
      if (kPair && i + k0 / kOfPage >= n) break;
      const char* src = rows + ((static_cast<int64_t>(pages[i + k0 / kOfPage]) << a.page_shift) + row0) * width;
#pragma unroll
      for (int k = 0; k < kOfPage; ++k)
        next[k0 + k] = *reinterpret_cast<const uint4*>(src + (batch * kOfPage + k) * kRows * width);
    }
  };
  float sum[kDims] = {};
  auto finish = [&](int page) {   // the sums of its rows are done
    int at = col;   // the first of this lane's dims
#pragma unroll
    for (int half = kDims / 2, d = kLanes; half > 1; half >>= 1, d <<= 1) {
      const bool upper = lane & d;
#pragma unroll
      for (int j = 0; j < half; ++j) {
        const float keep = upper ? sum[half + j] : sum[j], pass = upper ? sum[j] : sum[half + j];
        sum[j] = keep + __shfl_xor_sync(~0u, pass, d);
      }
      if (upper) at += half;
    }
    *reinterpret_cast<uint32_t*>(a.summaries + static_cast<int64_t>(page) * kD + 64 * warp + at) =
        pack_bf16x2(sum[0] * a.scale, sum[1] * a.scale);
#pragma unroll
    for (int j = 0; j < kDims; ++j) sum[j] = 0.f;
  };
  if (n > 0) read(0, 0);
  for (int i = 0, batch = 0; i < n;) {
    uint4 v[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) v[k] = next[k];
    const int now = i;
    if (kPair) {
      i += 2;
    } else if (++batch == batches) {
      batch = 0;
      ++i;
    }
    if (i < n) read(i, batch);
#pragma unroll
    for (int k = 0; k < kOfPage; ++k) add_values<kFp8>(sum, v[k]);
    if (!kPair && batch) continue;
    finish(pages[now]);
    if (kPair && now + 1 < n) {
#pragma unroll
      for (int k = kOfPage; k < kLoads; ++k) add_values<kFp8>(sum, v[k]);
      finish(pages[now + 1]);
    }
  }
}

// frequency / 2 pi, a fraction of a turn in units of 2^-64.  1 / 2 pi is taken
// as the double next to it and the double next to what that leaves (together
// within 2^-110), the first product with the rounding that fma recovers, and
// each of the three terms is rounded once, after its whole turns are off.
uint64_t fraction_of_turn(double frequency) {
  constexpr double kHigh = 0x1.45f306dc9c883p-3, kLow = -0x1.6b01ec5417056p-57;
  const double turns = frequency * kHigh;
  const double terms[3] = {turns, std::fma(frequency, kHigh, -turns), frequency * kLow};
  uint64_t sum = 0;
  for (const double t : terms) {
    const double units = std::nearbyint((t - std::nearbyint(t)) * 0x1p64);   // at most 2^63 either way
    sum += units < 0 ? uint64_t{0} - static_cast<uint64_t>(-units) : static_cast<uint64_t>(units);
  }
  return sum;
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
    a.rope.turn[i] = fraction_of_turn(rope->inv_freq[i]);
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
  // Query rows of a CTA: four quarters to a thread keep 128 KB an SM in flight
  // (8190 tokens x 128 heads: 48.0 us, with two 54.6), but a short step is over
  // sooner on more SMs (64 x 128: 2.5 us with two, 3.5 with four).
  const int rows = tokens * num_heads >= kManyRows ? kRowsPerBlock : kRowsPerBlock / 2;
  a.tokens_per_block = num_heads == 0 || num_heads >= rows ? 1 : rows / num_heads < kMostTokens ? rows / num_heads : kMostTokens;
  a.kv_blocks = (tokens + kKvWarps - 1) / kKvWarps;
  cudaError_t e = cudaSuccess;
  if (tokens > 0 && (e = paging_error_word(&a.err)) == cudaSuccess) {
    const int64_t q_blocks = num_heads > 0 ? (tokens + a.tokens_per_block - 1) / a.tokens_per_block : 0;
    const int grid = static_cast<int>(a.kv_blocks + q_blocks);
    auto kernel = rope->interleaved ? (fp8 ? append_kernel<true, true> : append_kernel<true, false>)
                                    : (fp8 ? append_kernel<false, true> : append_kernel<false, false>);
    e = launch_dependent(kernel, grid, kQThreads, 0, 1, s, a);
  }
  return finish_call(e, check_status, s);
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
  int sms = 0;
  cudaError_t e = cudaSuccess;
  if (tokens > 0 && (e = current_sms(&sms)) == cudaSuccess && (e = paging_error_word(&a.err)) == cudaSuccess) {
    // one wave of CTAs with equal runs of tokens (fewer CTAs for a short run are no
    // better: 8192 tokens of a prompt 2.9 us against 3.4 with one an SM, but 4096
    // single ones 5.2 against 4.4, and 88 against 48 where each completes a page)
    const bool fp8 = kv_dtype == MLA_DTYPE_FP8_E4M3;
    const int64_t blocks = static_cast<int64_t>(sms) * sum_blocks(fp8), run = (tokens + blocks - 1) / blocks;
    a.per_block = static_cast<int>(run < kSumThreads ? run : kSumThreads);
    auto kernel = !fp8              ? summarize_kernel<false, false>
                  : page_size == 16 ? summarize_kernel<true, true>
                                    : summarize_kernel<true, false>;
    e = launch_dependent(kernel, static_cast<int>((tokens + a.per_block - 1) / a.per_block), kSumThreads, 0, 1, s, a);
  }
  return finish_call(e, check_status, s);
}
