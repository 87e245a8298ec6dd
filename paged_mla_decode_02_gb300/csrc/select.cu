// The choice of the pages that a sparse decode reads: mla_page_scores (a
// page's best score over the heads of a query, against the page's mean row)
// and mla_select_pages (the best scoring pages of each row as a page list).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "device_utils.cuh"
#include "launch.h"
#include "mla_internal.h"
#include "mla_paging.h"
#include "tc_utils.cuh"
#include "tmap.h"

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
//
// A row's scores are the row maxima of S = summaries[pages] . q^T, a product
// of M = pages, N = heads, K = 576 that reads 1152 bytes per page: bound by
// HBM.  The pages of all rows in a line (the page lists laid end to end) are
// cut into one even run for each SM; a CTA takes its run in tiles of up to
// 128 pages of one row.
// - One warp copies, in nine chunks of 64 dims through a ring in shared
//   memory, the pages' rows (tile::gather4, each lane the four pages it
//   holds the ids of) and the row's queries (from L2: reading them again for
//   every tile costs less than keeping 144 KB of them resident would leave
//   for pages in flight).
// - One thread issues the tcgen05 MMAs into one of two TMEM accumulators.
// - Four warps read the other: a TMEM lane holds one page's products with
//   all heads, so a thread takes its page's maximum without any exchange.
struct ScoreArgs {
  const char* summaries;
  int num_pages;
  Lists lists;
  int rows, heads;
  float* scores;
  int64_t stride;
};

constexpr int kScoreThreads = 320;      // warp 0 queries, warp 1 MMAs, warps 2..5 maxima, 6..9 pages
constexpr int kCopyWarps = 4;
constexpr int kCopiesAhead = 4;         // chunks of pages a copying thread has in flight
constexpr int kTilePages = 128;         // the MMA's M
constexpr int kChunks = kD / 64;        // copies of 64 dims
constexpr int kScoreStages = 6;
constexpr int kPanelBytes = kTilePages * 128;
constexpr int kStageBytes = 2 * kPanelBytes;   // pages, then queries (up to 128 heads)
constexpr int kMinRun = 32;             // pages of a CTA's run, at least
enum { kFull = 0, kEmpty = kScoreStages, kTFull = 2 * kScoreStages, kTEmpty = kTFull + 2, kFinal = kTEmpty + 2,
       kNumBar };

__host__ __device__ constexpr int scores_smem(int rows) {
  return kScoreStages * kStageBytes + 8 * kNumBar + 16 + 4 * (rows + 1) + 1024;
}

struct Tile {
  int row, page0, pages;   // pages page0 .. page0 + pages - 1 of the row's list
};

__global__ void __launch_bounds__(kScoreThreads, 1)
    scores_kernel(const __grid_constant__ CUtensorMap map_qn, const __grid_constant__ CUtensorMap map_qp,
                  const ScoreArgs a) {
  using namespace tc;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t base = smem_u32(sm);
  const uint32_t bars = base + kScoreStages * kStageBytes;
  auto bar = [&](int i) { return bars + 8 * i; };
  unsigned char* after = sm + kScoreStages * kStageBytes + 8 * kNumBar;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(after);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(after + 4);
  int* at = reinterpret_cast<int*>(after + 16);          // [rows + 1]: pages before each row
  __shared__ long long warp_sum[kScoreThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kNumBar; ++i)
      mbar_init(bar(i), i < kEmpty ? 1 + kCopyWarps : i == kTEmpty || i == kTEmpty + 1 ? 4 : 1);
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(smem_u32(tmem_slot), 2 * kMaxHeads);
  // pages before each row, over the rows' lists as far as they are sound
  long long all;
  {
    const int per = (a.rows + kScoreThreads - 1) / kScoreThreads;
    long long sum = 0;
    int first;
    for (int i = 0; i < per; ++i) {
      const int r = tid * per + i;
      if (r < a.rows) sum += list_of(a.lists, r, &first);
      if (r < a.rows) at[r + 1] = static_cast<int>(sum);
    }
    long long incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(~0u, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    long long before = incl - sum;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    for (int i = 0; i < per; ++i)
      if (tid * per + i < a.rows) at[tid * per + i + 1] += static_cast<int>(before);
    if (tid == 0) at[0] = 0;
    all = 0;
    for (int w = 0; w < kScoreThreads / 32; ++w) all += warp_sum[w];
    // more than kv_indices can hold: lists that overlap (kv_indptr goes back)
    if (all > INT32_MAX && tid == 0) report_error(&g_select_err, kErrBounds);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  // this CTA's run of the line of pages
  const int total = all > INT32_MAX ? 0 : static_cast<int>(all);
  const int even = (total + gridDim.x - 1) / gridDim.x;
  const int run = even > kMinRun ? even : kMinRun;
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * run;
  int pos = static_cast<int>(lo < total ? lo : total);
  const int end = static_cast<int>(lo + run < total ? lo + run : total);
  int row = 0;
  if (pos < end) {   // the row that holds page pos
    int hi = a.rows;
    while (hi - row > 1) {
      const int mid = (row + hi) >> 1;
      if (at[mid] <= pos) row = mid; else hi = mid;
    }
  }
  // the tiles of the run, in order (every role walks the same ones)
  auto next = [&](Tile& t) {
    if (pos >= end) return false;
    while (at[row + 1] <= pos) ++row;
    int n = at[row + 1] < end ? at[row + 1] - pos : end - pos;
    n = n < kTilePages ? n : kTilePages;
    t = {row, pos - at[row], n};
    pos += n;
    return true;
  };
  const int heads16 = (a.heads + 15) & ~15;
  bool ok = true;
  Tile t;

  if (warp == 0) {
    // ---------------- queries ----------------
    int st = 0;
    while (ok && next(t)) {
      for (int c = 0; c < kChunks; ++c, ++st) {
        const int slot = st % kScoreStages;
        if (!(ok = mbar_wait_warp(bar(kEmpty + slot), ((st / kScoreStages) & 1) ^ 1, abort_flag))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(kFull + slot), a.heads * 128);
          tma_load_2d(base + slot * kStageBytes + kPanelBytes, c < kChunks - 1 ? &map_qn : &map_qp,
                      c < kChunks - 1 ? 64 * c : 0, t.row * a.heads, bar(kFull + slot));
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) report_error(&g_select_err, kErrTimeout);
    if (lane == 0)   // every copy issued has landed before the CTA leaves
      for (int k = 1; k <= kScoreStages && k <= st; ++k)
        mbar_wait_drain(bar(kFull + (st - k) % kScoreStages), ((st - k) / kScoreStages) & 1);
    __syncwarp();
  } else if (warp >= 6) {
    // ---------------- pages ----------------
    // thread i copies 16-byte column i % 8 of rows i / 8 + 16 j
    const int i = tid - 6 * 32, col = i & 7, row0 = i >> 3;
    const uint32_t dst = base + row0 * 128 + ((col ^ (row0 & 7)) << 4);
    int st = 0, done = 0;
    auto land = [&]() {   // the oldest chunk's copies of this warp are in place
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kFull + done % kScoreStages));
      ++done;
    };
    while (ok && next(t)) {
      const int32_t* ids = a.lists.indices + a.lists.indptr[t.row] + t.page0;
      const char* src[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int p = row0 + 16 * j;
        int id = p < t.pages ? ids[p] : -1;
        if (id < 0 || id >= a.num_pages) id = -1;   // not read; scored -inf below
        src[j] = id < 0 ? nullptr : a.summaries + static_cast<int64_t>(id) * (2 * kD) + 16 * col;
      }
      for (int c = 0; c < kChunks; ++c, ++st) {
        const int slot = st % kScoreStages;
        if (!(ok = mbar_wait_warp(bar(kEmpty + slot), ((st / kScoreStages) & 1) ^ 1, abort_flag))) break;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (src[j]) cp_async_16(dst + slot * kStageBytes + j * 2048, src[j] + 128 * c, 16);
        cp_async_commit();
        if (st - done >= kCopiesAhead) {
          cp_async_wait<kCopiesAhead>();
          land();
        }
      }
    }
    cp_async_wait<0>();
    while (ok && done < st) land();
    if (!ok && lane == 0) report_error(&g_select_err, kErrTimeout);
  } else if (warp == 1) {
    // ---------------- MMAs ----------------
    const uint32_t idesc = idesc_bf16_f32(kTilePages, heads16, false, false);
    int st = 0, n = 0;
    for (; ok && next(t); ++n) {
      const int acc = n & 1;
      if (!(ok = mbar_wait_warp(bar(kTEmpty + acc), ((n >> 1) & 1) ^ 1, abort_flag))) break;
      tc_fence_after();
      for (int c = 0; c < kChunks; ++c, ++st) {
        const int slot = st % kScoreStages;
        if (!(ok = mbar_wait_warp(bar(kFull + slot), (st / kScoreStages) & 1, abort_flag))) break;
        tc_fence_after();
        const uint32_t sa = base + slot * kStageBytes;
        const uint64_t da = smem_desc(sa, 16, 1024, kSw128);
        const uint64_t dq = smem_desc(sa + kPanelBytes, 16, 1024, kSw128);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ss(tmem + acc * kMaxHeads, da + 2 * kk, dq + 2 * kk, idesc, (c | kk) != 0, lane == 0);
        mma_commit(bar(kEmpty + slot), lane == 0);
      }
      if (!ok) break;
      mma_commit(bar(kTFull + acc), lane == 0);
    }
    if (!ok && lane == 0) report_error(&g_select_err, kErrTimeout);
    mma_commit(bar(kFinal), lane == 0);   // every MMA issued completes before TMEM is freed
    if (lane == 0) mbar_wait_drain(bar(kFinal), 0);
    __syncwarp();
  } else {
    // ---------------- maxima: page 32 quad + lane of the tile ----------------
    const int quad = warp & 3;
    for (int n = 0; ok && next(t); ++n) {
      const int acc = n & 1, p = 32 * quad + lane;
      int id = -1;
      if (p < t.pages) id = a.lists.indices[a.lists.indptr[t.row] + t.page0 + p];
      if (!(ok = mbar_wait_warp(bar(kTFull + acc), (n >> 1) & 1, abort_flag))) break;
      tc_fence_after();
      float best = -INFINITY;
      if (32 * quad < t.pages) {
#pragma unroll 1
        for (int c = 0; c < heads16; c += 32) {
          uint32_t v[32];
          tmem_ld32(tmem + (static_cast<uint32_t>(32 * quad) << 16) + acc * kMaxHeads + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (c + k < a.heads) best = fmaxf(best, __uint_as_float(v[k]));   // a NaN loses
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kTEmpty + acc));
      if (p < t.pages) {
        if (id < 0 || id >= a.num_pages) {
          report_error(&g_select_err, kErrBounds);
          best = -INFINITY;
        }
        a.scores[t.row * a.stride + t.page0 + p] = best;
      }
    }
    if (!ok && lane == 0) report_error(&g_select_err, kErrTimeout);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kMaxHeads);
  }
}

// Row-major [rows, cols] bf16, box box_rows x 64 elements, 128-byte swizzle.
bool encode_rows(CUtensorMap* m, const void* base, int64_t rows, int cols, int box_rows) {
  EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
  a.summaries = static_cast<const char*>(summaries);
  a.num_pages = num_pages;
  a.lists = {kv_indptr, kv_indices, n_indices, score_stride};
  a.rows = rows;
  a.heads = num_heads;
  a.scores = scores;
  a.stride = score_stride;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (rows > 0) {
    CUtensorMap mn, mp;
    const int64_t q_rows = static_cast<int64_t>(rows) * num_heads;
    if (!encode_rows(&mn, q_nope, q_rows, kDCkv, num_heads) ||
        !encode_rows(&mp, q_pe, q_rows, kDKpe, num_heads))
      return MLA_ERR_CUDA;
    int sms = 0;
    e = current_sms(&sms);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(scores_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, scores_smem(kMaxRows));
    // no more CTAs than the lists have runs of the least length
    const int64_t runs = (n_indices + kMinRun - 1) / kMinRun;
    const int grid = static_cast<int>(runs < 1 ? 1 : runs < sms ? runs : sms);
    if (e == cudaSuccess)
      e = launch_dependent(scores_kernel, grid, kScoreThreads, scores_smem(rows), 1, s, mn, mp, a);
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
