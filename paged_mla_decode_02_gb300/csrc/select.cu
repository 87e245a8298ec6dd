// The choice of the pages that a sparse decode reads: mla_page_scores (a
// page's best score over the heads of a query, against the page's mean row)
// and mla_select_pages (the best scoring pages of each row as a page list).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "device_utils.cuh"
#include "launch.h"
#include "mla_internal.h"
#include "mla_paging.h"

namespace mla {
namespace {

constexpr int kMaxRows = 4096;
__device__ int32_t g_select_err;   // first device error of this file's kernels

// Row r's page list: its first entry and length, or nothing (reported) when
// it leaves kv_indices or is longer than `longest`.
struct Lists {
  const int32_t* indptr;
  const int32_t* indices;
  int64_t n_indices;
  int64_t longest;
};
__device__ __forceinline__ int list_of(const Lists& l, int r, int* first) {
  const int b = l.indptr[r], e = l.indptr[r + 1];
  *first = b;
  if (b >= 0 && e >= b && e <= l.n_indices && e - b <= l.longest) return e - b;
  report_error(&g_select_err, kErrBounds);
  return 0;
}

// ---------------------------------------------------------------------------
// Scores
// ---------------------------------------------------------------------------
struct ScoreArgs {
  const __nv_bfloat16* q_nope;
  const __nv_bfloat16* q_pe;
  const __nv_bfloat16* summaries;
  int num_pages;
  Lists lists;
  int rows, heads;
  float* scores;
  int64_t stride;
};

constexpr int kScoreWarps = 8;

// One warp per page of a row, 18 of its 576 dims in each lane.
__global__ void __launch_bounds__(32 * kScoreWarps) scores_kernel(const ScoreArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.y;
  int first;
  const int n = list_of(a.lists, r, &first);
  for (int p = blockIdx.x * kScoreWarps + warp; p < n; p += gridDim.x * kScoreWarps) {
    const int page = a.lists.indices[first + p];
    float best = -INFINITY;
    if (page < 0 || page >= a.num_pages) {
      report_error(&g_select_err, kErrBounds);
    } else {
      float x[18];
      for (int k = 0; k < 18; ++k) x[k] = __bfloat162float(a.summaries[static_cast<int64_t>(page) * kD + 32 * k + lane]);
      for (int h = 0; h < a.heads; ++h) {
        const int64_t row = static_cast<int64_t>(r) * a.heads + h;
        float s = 0.f;
        for (int k = 0; k < 16; ++k) s += x[k] * __bfloat162float(a.q_nope[row * kDCkv + 32 * k + lane]);
        for (int k = 0; k < 2; ++k) s += x[16 + k] * __bfloat162float(a.q_pe[row * kDKpe + 32 * k + lane]);
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
        best = fmaxf(best, s);   // a NaN loses
      }
    }
    if (lane == 0) a.scores[r * a.stride + p] = best;
  }
}

// ---------------------------------------------------------------------------
// Selection
// ---------------------------------------------------------------------------
struct SelectArgs {
  const float* scores;
  int64_t stride;
  Lists lists;
  int rows, top_k, keep_first, keep_last;
  int32_t* sel_indptr;
  int32_t* sel_indices;
};

constexpr int kSelThreads = 1024;

// Scores as unsigned keys in the same order: NaN as -inf, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float s) {
  if (s != s) s = -INFINITY;
  const uint32_t u = __float_as_uint(s + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int block_sum(int v, int* sm) {
  v = __reduce_add_sync(~0u, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(~0u, sm[threadIdx.x & 31]);
}

// Exclusive prefix sum over the block's threads; *total receives the sum.
__device__ __forceinline__ int block_scan(int v, int* sm, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(~0u, incl, d);
    if (lane >= d) incl += o;
  }
  __syncthreads();
  if (lane == 31) sm[warp] = incl;
  __syncthreads();
  int w = sm[lane];
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(~0u, w, d);
    if (lane >= d) w += o;
  }
  *total = __shfl_sync(~0u, w, 31);
  const int before = __shfl_sync(~0u, w, warp ? warp - 1 : 0);
  return (warp ? before : 0) + incl - v;
}

// One CTA per row.  The k-th highest key of the middle pages is found bit by
// bit: the largest threshold with at least k keys at or above it.  Pages
// above it are kept, and the first of those equal to it as far as k reaches.
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int sm[32];
  const int tid = threadIdx.x, r = blockIdx.x;
  // the pages that the rows before this one keep
  int before = 0, first;
  for (int i = tid; i < r; i += kSelThreads) before += min(a.top_k, list_of(a.lists, i, &first));
  before = block_sum(before, sm);
  const int n = list_of(a.lists, r, &first);
  const int keep = min(a.top_k, n);
  if (tid == 0) {
    if (r == 0) a.sel_indptr[0] = 0;
    a.sel_indptr[r + 1] = before + keep;
  }
  const float* s = a.scores + r * a.stride;
  const int32_t* pages = a.lists.indices + first;
  int32_t* out = a.sel_indices + before;
  if (n <= a.top_k) {
    for (int p = tid; p < n; p += kSelThreads) out[p] = pages[p];
    return;
  }
  const int lo = a.keep_first, hi = n - a.keep_last;
  const int want = keep - a.keep_first - a.keep_last;
  uint32_t cut = 0;
  if (want > 0) {
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t t = cut | 1u << bit;
      int c = 0;
      for (int p = lo + tid; p < hi; p += kSelThreads) c += key_of(s[p]) >= t;
      if (block_sum(c, sm) >= want) cut = t;
    }
  } else {
    cut = 0xffffffffu;
  }
  int above = 0;
  for (int p = lo + tid; p < hi; p += kSelThreads) above += key_of(s[p]) > cut;
  int ties = want - block_sum(above, sm);   // how many of those equal to the cut are kept
  int at = 0;
  for (int p0 = 0; p0 < n; p0 += kSelThreads) {
    const int p = p0 + tid;
    const bool middle = p >= lo && p < hi;
    const uint32_t k = middle ? key_of(s[p]) : 0;
    int total;
    const int tie = block_scan(middle && k == cut, sm, &total);
    const bool kept = p < n && (!middle || k > cut || (k == cut && tie < ties));
    ties -= total;
    const int place = block_scan(kept, sm, &total);
    if (kept) out[at + place] = pages[p];
    at += total;
  }
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status_t mla_page_scores(const void* q_nope, const void* q_pe, const void* summaries, int num_pages,
                                        const int32_t* kv_indptr, const int32_t* kv_indices, int64_t n_indices,
                                        int rows, int num_heads, float* scores, int64_t score_stride,
                                        int check_status, void* stream) {
  if (rows < 0 || num_heads < 1 || num_heads > kMaxHeads || num_pages < 1 || n_indices < 0 || score_stride < 0)
    return MLA_ERR_INVALID_ARG;
  if (rows > kMaxRows) return MLA_ERR_CAPACITY;
  if (rows > 0 && (!q_nope || !q_pe || !summaries || !kv_indptr || (n_indices > 0 && !kv_indices) ||
                   (score_stride > 0 && !scores)))
    return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_nope) || !aligned16(q_pe) || !aligned16(summaries)) return MLA_ERR_INVALID_ARG;
  ScoreArgs a{};
  a.q_nope = static_cast<const __nv_bfloat16*>(q_nope);
  a.q_pe = static_cast<const __nv_bfloat16*>(q_pe);
  a.summaries = static_cast<const __nv_bfloat16*>(summaries);
  a.num_pages = num_pages;
  a.lists = {kv_indptr, kv_indices, n_indices, score_stride};
  a.rows = rows;
  a.heads = num_heads;
  a.scores = scores;
  a.stride = score_stride;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (rows > 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(32, rows);
    cfg.blockDim = dim3(32 * kScoreWarps);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, scores_kernel, a);
  }
  return finish_call(e, &g_select_err, check_status, s);
}

extern "C" mla_status_t mla_select_pages(const float* scores, int64_t score_stride, const int32_t* kv_indptr,
                                         const int32_t* kv_indices, int64_t n_indices, int rows, int top_k,
                                         int keep_first, int keep_last, int32_t* sel_indptr, int32_t* sel_indices,
                                         int64_t sel_cap, int check_status, void* stream) {
  if (rows < 0 || n_indices < 0 || score_stride < 0 || sel_cap < 0) return MLA_ERR_INVALID_ARG;
  if (top_k < 1 || keep_first < 0 || keep_last < 1 || static_cast<int64_t>(keep_first) + keep_last > top_k)
    return MLA_ERR_INVALID_ARG;
  if (rows > kMaxRows || static_cast<int64_t>(rows) * top_k > INT32_MAX ||
      static_cast<int64_t>(rows) * top_k > sel_cap)
    return MLA_ERR_CAPACITY;
  if (!sel_indptr || (rows > 0 && (!kv_indptr || !sel_indices || (n_indices > 0 && !kv_indices) ||
                                   (score_stride > 0 && !scores))))
    return MLA_ERR_INVALID_ARG;
  SelectArgs a{};
  a.scores = scores;
  a.stride = score_stride;
  a.lists = {kv_indptr, kv_indices, n_indices, score_stride};
  a.rows = rows;
  a.top_k = top_k;
  a.keep_first = keep_first;
  a.keep_last = keep_last;
  a.sel_indptr = sel_indptr;
  a.sel_indices = sel_indices;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = rows > 0 ? launch_dependent(select_kernel, rows, kSelThreads, 0, 1, s, a)
                           : cudaMemsetAsync(sel_indptr, 0, sizeof(int32_t), s);
  return finish_call(e, &g_select_err, check_status, s);
}
