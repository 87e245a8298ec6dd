// Rows into a 4-bit cache (mla_quantize_append) and rows out of a paged cache
// of any type (mla_read_cache).
//
// Both move rows and little else, so both are bound by HBM and laid out alike:
// eight lanes to a row, four rows to a warp, lane j taking the 8-dim chunks j,
// j + 8, .. of the 72 (64 of ckv, 8 of kpe).  A chunk is 16 bytes of a 16-bit
// row and one word of codes, so a row's eight lanes read and write runs of 128
// and 32 bytes, and the four chunks of a group (32 dims, one shift) lie in four
// neighbouring lanes.  Every load of a row is under way before the first is used.
//
// Measured from a graph, cold L2: 131000 fp32 rows written in 55.5 us, 6.2 TB/s,
// 91 % of the copy rate; 100000 4-bit rows read to bf16 in 27.0 us, 5.4 TB/s, to fp16 in
// 28.2 and to fp32 in 63.8, 4.1 TB/s; as many rows of a bf16 cache to bf16 in 36.8 us,
// 6.3 TB/s; 92000 e4m3 rows to fp16 in 26.9 us, 5.9 TB/s.  8190 rows written take 9.0 us
// and 64 take 6.7, 1600 read 8.6: the launch and a chain of dependent reads (slots, or
// offsets, page list and page, then the row).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "device_utils.cuh"
#include "launch.h"
#include "mla_paging.h"
#include "q4.cuh"

namespace mla {
namespace {

constexpr int kThreads = 128;
constexpr int kLanes = 8;                        // of a row
constexpr int kChunks = kQ4Words / kLanes;       // of a lane: 8 of ckv, 1 of kpe
constexpr int kRowsPerBlock = kThreads / kLanes;
static_assert(kChunks == 9, "chunks of a lane");

// Chunk i of a lane as it lies in memory: 8 values of 2 or 4 bytes.
template <typename T>
struct Chunk {
  uint32_t w[2 * sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void load_chunk(Chunk<T>& c, const T* src) {
#pragma unroll
  for (int h = 0; h < static_cast<int>(sizeof(T)) / 2; ++h) {
    const uint4 v = reinterpret_cast<const uint4*>(src)[h];
    c.w[4 * h] = v.x, c.w[4 * h + 1] = v.y, c.w[4 * h + 2] = v.z, c.w[4 * h + 3] = v.w;
  }
}

// The fp32 bits of the chunk's largest magnitude; compared as integers, in which
// NaN is above infinity.
template <typename T>
__device__ __forceinline__ uint32_t top_bits(const Chunk<T>& c) {
  if constexpr (sizeof(T) == 4) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, c.w[i] & 0x7fffffffu);
    return m;
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, c.w[i] & 0x7fff7fffu);
    m = max(m >> 16, m & 0xffffu);
    if constexpr (std::is_same<T, __half>::value)
      return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
    return m << 16;
  }
}
template <typename T>
__device__ __forceinline__ float2 pair_of(const Chunk<T>& c, int i) {   // dims 2i, 2i + 1
  if constexpr (sizeof(T) == 4)
    return make_float2(__uint_as_float(c.w[2 * i]), __uint_as_float(c.w[2 * i + 1]));
  else if constexpr (std::is_same<T, __half>::value)
    return __half22float2(*reinterpret_cast<const __half2*>(&c.w[i]));
  else
    return make_float2(__uint_as_float(c.w[i] << 16), __uint_as_float(c.w[i] & 0xffff0000u));
}
// The bytes with the signs of dims 4h .. 4h + 3.
template <typename T>
__device__ __forceinline__ uint32_t sign_bytes(const Chunk<T>& c, int h) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t lo = __byte_perm(c.w[4 * h], c.w[4 * h + 1], 0x0073);
    const uint32_t hi = __byte_perm(c.w[4 * h + 2], c.w[4 * h + 3], 0x0073);
    return __byte_perm(lo, hi, 0x5410);
  } else {
    return __byte_perm(c.w[2 * h], c.w[2 * h + 1], 0x7531);
  }
}
// 8 values times f as a word of codes.  The products are exact (f is a power of
// two) but for those far below the least magnitude; the conversion rounds to
// nearest even and saturates.
template <typename T>
__device__ __forceinline__ uint32_t codes_of(const Chunk<T>& c, float f) {
  uint32_t mags = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = pair_of(c, i);
    mags |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(x.x * f, x.y * f), __NV_E2M1, cudaRoundNearest)) << (8 * i);
  }
  return (mags & 0x77777777u) | (sign_bytes(c, 0) & 0x80808080u) | ((sign_bytes(c, 1) >> 4) & 0x08080808u);
}

struct QuantizeArgs {
  const void* ckv;
  int64_t ckv_stride;
  const void* kpe;
  int64_t kpe_stride;
  const int64_t* slots;
  uint8_t* cache;
  int64_t cache_slots;
  int64_t tokens;
  int32_t* err;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantizeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int j = threadIdx.x % kLanes;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + threadIdx.x / kLanes;
  int64_t slot = t < a.tokens ? a.slots[t] : -1;
  if (slot >= a.cache_slots) {
    if (j == 0) report_error(a.err, kErrBounds);
    slot = -1;
  }
  // a lane without a row takes part in the shuffles with zeros
  Chunk<T> c[kChunks] = {};
  if (slot >= 0) {
    const T* ckv = static_cast<const T*>(a.ckv) + t * a.ckv_stride + 8 * j;
#pragma unroll
    for (int i = 0; i < kChunks - 1; ++i) load_chunk(c[i], ckv + 8 * kLanes * i);
    load_chunk(c[kChunks - 1], static_cast<const T*>(a.kpe) + t * a.kpe_stride + 8 * j);
  }
  // e_g of this lane's nine groups (2i + j / 4), and the row's
  uint32_t row_top = 0;
  int e[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    uint32_t top = top_bits(c[i]);
    top = max(top, __shfl_xor_sync(~0u, top, 1));
    top = max(top, __shfl_xor_sync(~0u, top, 2));
    row_top = max(row_top, top);
    // top = m 2^x with m in [1, 2); 6 * 2^e = 1.5 * 2^(e + 2)
    e[i] = static_cast<int>(top >> 23) - 127 - 2 + ((top & 0x7fffffu) > 0x400000u);
  }
  row_top = max(row_top, __shfl_xor_sync(~0u, row_top, 4));
  const bool nan = row_top > 0x7f800000u;
  const int row_e = min(max(static_cast<int>(row_top >> 23) - 127 - 2 + ((row_top & 0x7fffffu) > 0x400000u), kQ4MinExp), kQ4MaxExp);
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.cache + slot * kQ4Row);
  uint64_t shifts = 0;   // of this lane's groups 2i (or 2i + 1), i < 8, a byte each
  uint32_t last = 0;     // of its group in kpe
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int k = nan ? 0 : min(max(row_e - e[i], 0), kQ4MaxShift);
    const uint32_t w = nan ? 0u : codes_of(c[i], pow2(k - row_e));
    if (i < kChunks - 1) shifts |= static_cast<uint64_t>(k) << (8 * i);
    else last = k;
    if (slot >= 0) dst[kLanes * i + j] = w;
  }
  // lane 0 has the even groups' shifts, lane 4 the odd ones'
  shifts |= __shfl_xor_sync(~0u, shifts, 4) << 4;
  last |= __shfl_xor_sync(~0u, last, 4) << 4;
  if (slot >= 0 && j == 0) {
    const uint32_t exponent = nan ? kQ4NanExp : row_e + 127;
    *reinterpret_cast<uint4*>(dst + kQ4Words) = make_uint4(static_cast<uint32_t>(shifts), static_cast<uint32_t>(shifts >> 32), last | exponent << 8, 0u);
  }
}

struct ReadArgs {
  const void* cache;
  const void* kpe_cache;
  float kv_scale;
  int num_pages;
  int page_shift;
  const int32_t* kv_indptr;
  const int32_t* kv_indices;
  int64_t n_indices;
  const int32_t* starts;
  const int32_t* row_indptr;
  int batch;
  void* ckv_out;
  int64_t ckv_stride;
  void* kpe_out;
  int64_t kpe_stride;
  int64_t max_rows;
  int32_t* err;
};

template <typename T>
__device__ __forceinline__ void store_chunk(T* dst, const float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
      }
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// code * scale for a conversion that rounds it to 16 bits as if it were exact.  A code
// has 4 bits and the scale 24, fp32 holds 24 of the product's 28: a product rounded to
// fp32 first may land in the middle between two numbers of the type and then on the
// wrong one.  So it is truncated, and its last bit set if that lost anything (8 or 11
// of the 24 bits are the type's, so the last one only breaks ties).
__device__ __forceinline__ float truncated_product(float code, float scale) {
  const float lo = __fmul_rd(fabsf(code), scale), hi = __fmul_ru(fabsf(code), scale);
  return __uint_as_float(__float_as_uint(lo) | (lo != hi ? 1u : 0u) | (__float_as_uint(code) & 0x80000000u));
}
// A scale of 20 bits (a power of two first of all) whose products fp32 has without that,
// none of them subnormal: 26.9 us for 29.9, 92000 rows to fp16.
__device__ __forceinline__ bool short_scale(float scale) { return (__float_as_uint(scale) & 15u) == 0 && scale >= 0x1p-100f; }

// The request of row r: how many of row_indptr[1 ..] are at or below it, found
// by a row's eight lanes together, eight probes a step.
__device__ __forceinline__ int request_of(const int32_t* row_indptr, int batch, int64_t r) {
  const int j = threadIdx.x % kLanes;
  const int shift = (threadIdx.x & 31) & ~(kLanes - 1);
  int lo = 0, n = batch;   // the answer is in lo .. lo + n
  while (__any_sync(~0u, n > 0)) {
    const int step = (n + kLanes) / (kLanes + 1);
    const int64_t probe = lo + static_cast<int64_t>(j + 1) * step;
    const bool below = n > 0 && probe <= lo + n && row_indptr[probe] <= r;
    const int count = __popc((__ballot_sync(~0u, below) >> shift) & 0xffu);
    lo += count * step;
    n = n <= 0 ? 0 : count == kLanes ? n - count * step : min(step - 1, n - count * step);
  }
  return lo;
}

enum class Kind { kBf16, kFp8, kQ4 };

template <Kind kKind, typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(ReadArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int j = threadIdx.x % kLanes;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + threadIdx.x / kLanes;
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.row_indptr[a.batch] > a.max_rows) report_error(a.err, kErrBounds);
  const int b = request_of(a.row_indptr, a.batch, r);
  if (b >= a.batch || r >= a.max_rows) return;
  const int first = a.row_indptr[b];
  if (r < first) return;   // before the first request's rows
  const int64_t start = a.starts[b], token = start + (r - first);
  const int64_t list = a.kv_indptr[b], entry = list + (token >> a.page_shift);
  int page = -1;
  if (start >= 0 && list >= 0 && entry < a.kv_indptr[b + 1] && entry < a.n_indices) page = a.kv_indices[entry];
  if (page < 0 || page >= a.num_pages) {
    if (j == 0) report_error(a.err, kErrBounds);
    return;
  }
  const int64_t slot = (static_cast<int64_t>(page) << a.page_shift) + (token & ((1 << a.page_shift) - 1));
  T* ckv = static_cast<T*>(a.ckv_out) + r * a.ckv_stride + 8 * j;
  T* kpe = static_cast<T*>(a.kpe_out) + r * a.kpe_stride + 8 * j;
  auto put = [&](int i, const float (&x)[8]) { store_chunk(i < kChunks - 1 ? ckv + 8 * kLanes * i : kpe, x); };
  if constexpr (kKind == Kind::kQ4) {
    const uint8_t* row = static_cast<const uint8_t*>(a.cache) + slot * kQ4Row;
    uint32_t w[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) w[i] = reinterpret_cast<const uint32_t*>(row)[kLanes * i + j];
    const Q4Meta m{*reinterpret_cast<const uint4*>(row + kQ4Meta)};
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int group = 2 * i + (j >> 2);
      if constexpr (std::is_same<T, __half>::value) {   // whose range the values may leave
        float x[8];
        q4_expand(w[i], x);
        const float unit = q4_unit(m, group);
#pragma unroll
        for (int d = 0; d < 8; ++d) x[d] *= unit;
        put(i, x);
      } else {
        const uint4 v = q4_bf16x8(q4_table(m, group), w[i]);
        uint4* dst = reinterpret_cast<uint4*>(i < kChunks - 1 ? ckv + 8 * kLanes * i : kpe);
        if constexpr (sizeof(T) == 2) {
          *dst = v;
        } else {
          dst[0] = make_uint4(v.x << 16, v.x & 0xffff0000u, v.y << 16, v.y & 0xffff0000u);
          dst[1] = make_uint4(v.z << 16, v.z & 0xffff0000u, v.w << 16, v.w & 0xffff0000u);
        }
      }
    }
  } else if constexpr (kKind == Kind::kFp8) {
    uint2 w[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const uint8_t* src = i < kChunks - 1 ? static_cast<const uint8_t*>(a.cache) + slot * kDCkv + 8 * kLanes * i
                                           : static_cast<const uint8_t*>(a.kpe_cache) + slot * kDKpe;
      w[i] = *reinterpret_cast<const uint2*>(src + 8 * j);
    }
    auto expand = [&](auto product) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        float x[8];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const uint32_t half = (d < 2 ? w[i].x : w[i].y) >> (16 * (d & 1));
          const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(half), __NV_E4M3);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
          x[2 * d] = product(f.x);
          x[2 * d + 1] = product(f.y);
        }
        put(i, x);
      }
    };
    if (sizeof(T) == 4 || short_scale(a.kv_scale)) expand([&](float f) { return f * a.kv_scale; });
    else expand([&](float f) { return truncated_product(f, a.kv_scale); });
  } else {
    Chunk<__nv_bfloat16> c[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      load_chunk(c[i], i < kChunks - 1 ? static_cast<const __nv_bfloat16*>(a.cache) + slot * kDCkv + 8 * (kLanes * i + j)
                                       : static_cast<const __nv_bfloat16*>(a.kpe_cache) + slot * kDKpe + 8 * j);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      float x[8];
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const float2 f = pair_of(c[i], d);
        x[2 * d] = f.x;
        x[2 * d + 1] = f.y;
      }
      put(i, x);
    }
  }
}

using ReadKernel = void (*)(ReadArgs);
template <Kind kKind>
ReadKernel read_kernel_for(int out_dtype) {
  return out_dtype == MLA_DTYPE_BF16   ? read_kernel<kKind, __nv_bfloat16>
         : out_dtype == MLA_DTYPE_FP16 ? read_kernel<kKind, __half>
                                       : read_kernel<kKind, float>;
}

// Bytes of an element of plain rows; 0 for a type that rows do not have.
int row_element(int dtype) {
  return dtype == MLA_DTYPE_BF16 || dtype == MLA_DTYPE_FP16 ? 2 : dtype == MLA_DTYPE_FP32 ? 4 : 0;
}
bool page_size_ok(int page_size) { return page_size == 16 || page_size == 32 || page_size == 64; }

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status_t mla_quantize_append(const void* ckv, int64_t ckv_stride, const void* kpe, int64_t kpe_stride,
                                            int row_dtype, const int64_t* slots, void* cache, int num_pages,
                                            int page_size, int64_t tokens, int check_status, void* stream) {
  if (!cache || !aligned16(cache) || num_pages < 1 || page_size < 1 || tokens < 0) return MLA_ERR_INVALID_ARG;
  const int elt = row_element(row_dtype);
  if (elt == 0 || !page_size_ok(page_size)) return MLA_ERR_UNSUPPORTED;
  if (tokens > (1ll << 24)) return MLA_ERR_CAPACITY;   // keeps the grid inside its limit
  if (tokens > 0) {
    if (!ckv || !kpe || !slots) return MLA_ERR_INVALID_ARG;
    if (!aligned16(ckv) || !aligned16(kpe) || ((ckv_stride | kpe_stride) & (16 / elt - 1))) return MLA_ERR_INVALID_ARG;
  }
  QuantizeArgs a{};
  a.ckv = ckv;
  a.ckv_stride = ckv_stride;
  a.kpe = kpe;
  a.kpe_stride = kpe_stride;
  a.slots = slots;
  a.cache = static_cast<uint8_t*>(cache);
  a.cache_slots = static_cast<int64_t>(num_pages) * page_size;
  a.tokens = tokens;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (tokens > 0 && (e = paging_error_word(&a.err)) == cudaSuccess) {
    const int grid = static_cast<int>((tokens + kRowsPerBlock - 1) / kRowsPerBlock);
    auto kernel = row_dtype == MLA_DTYPE_BF16   ? quantize_kernel<__nv_bfloat16>
                  : row_dtype == MLA_DTYPE_FP16 ? quantize_kernel<__half>
                                                : quantize_kernel<float>;
    e = launch_dependent(kernel, grid, kThreads, 0, 1, s, a);
  }
  return finish_call(e, check_status, s);
}

extern "C" mla_status_t mla_read_cache(const void* cache, const void* kpe_cache, int kv_dtype, float kv_scale,
                                       int num_pages, int page_size, const int32_t* kv_indptr,
                                       const int32_t* kv_indices, int64_t n_indices, const int32_t* starts,
                                       const int32_t* row_indptr, int batch, void* ckv_out, int64_t ckv_stride,
                                       void* kpe_out, int64_t kpe_stride, int out_dtype, int64_t max_rows,
                                       int check_status, void* stream) {
  if (!cache || !aligned16(cache) || num_pages < 1 || page_size < 1 || batch < 0 || max_rows < 0 || n_indices < 0)
    return MLA_ERR_INVALID_ARG;
  const int elt = row_element(out_dtype);
  const bool q4 = kv_dtype == MLA_DTYPE_Q4, fp8 = kv_dtype == MLA_DTYPE_FP8_E4M3;
  if (elt == 0 || !page_size_ok(page_size) || (!q4 && !fp8 && kv_dtype != MLA_DTYPE_BF16)) return MLA_ERR_UNSUPPORTED;
  if (q4 ? kpe_cache != nullptr : (!kpe_cache || !aligned16(kpe_cache))) return MLA_ERR_INVALID_ARG;
  if (fp8 && (!std::isfinite(kv_scale) || kv_scale <= 0.f)) return MLA_ERR_INVALID_ARG;
  if (batch > 4096 || max_rows > INT32_MAX) return MLA_ERR_CAPACITY;
  if (batch > 0 && max_rows > 0) {
    if (!kv_indptr || !starts || !row_indptr || !ckv_out || !kpe_out || (n_indices > 0 && !kv_indices))
      return MLA_ERR_INVALID_ARG;
    if (!aligned16(ckv_out) || !aligned16(kpe_out) || ((ckv_stride | kpe_stride) & (16 / elt - 1)) || ckv_stride < kDCkv ||
        kpe_stride < kDKpe)   // rows of the outputs must not overlap
      return MLA_ERR_INVALID_ARG;
  }
  ReadArgs a{};
  a.cache = cache;
  a.kpe_cache = kpe_cache;
  a.kv_scale = kv_scale;
  a.num_pages = num_pages;
  a.page_shift = page_size == 16 ? 4 : page_size == 32 ? 5 : 6;
  a.kv_indptr = kv_indptr;
  a.kv_indices = kv_indices;
  a.n_indices = n_indices;
  a.starts = starts;
  a.row_indptr = row_indptr;
  a.batch = batch;
  a.ckv_out = ckv_out;
  a.ckv_stride = ckv_stride;
  a.kpe_out = kpe_out;
  a.kpe_stride = kpe_stride;
  a.max_rows = max_rows;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  // outputs of no rows: a block that looks at what row_indptr places
  if (batch > 0 && row_indptr && (e = paging_error_word(&a.err)) == cudaSuccess) {
    const int grid = max_rows > 0 ? static_cast<int>((max_rows + kRowsPerBlock - 1) / kRowsPerBlock) : 1;
    auto kernel = q4    ? read_kernel_for<Kind::kQ4>(out_dtype)
                  : fp8 ? read_kernel_for<Kind::kFp8>(out_dtype)
                        : read_kernel_for<Kind::kBf16>(out_dtype);
    e = launch_dependent(kernel, grid, kThreads, 0, 1, s, a);
  }
  return finish_call(e, check_status, s);
}
