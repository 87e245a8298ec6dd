// Page tables of a step on the device (mla_build_tables): the lengths of the
// requests after the step, pages taken from and returned to a stack of free
// pages, and from them the page lists (CSR), the cache slots and the
// positions of the new tokens.
//
// All of it follows from four prefix sums over the batch -- pages held, pages
// newly taken, pages returned, new tokens -- which every CTA of the kernel
// makes for itself in shared memory.  Each output element is then found on
// its own: a warp copies a run of the flat page list, a thread makes a
// token's slot, with a binary search of its request in a prefix sum.  The
// j-th page taken is known from j alone (the stack's top first, the returned
// pages on top in request order), so no thread waits for another's page.
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "mla_internal.h"
#include "mla_paging.h"
#include "tc_utils.cuh"

namespace mla {
namespace {

constexpr int kThreads = 1024;
constexpr int kMaxBatch = 4096;
constexpr int kPerThread = kMaxBatch / kThreads;   // requests a thread scans
// One cluster: its barrier lets all CTAs read the lengths before any writes
// them in place.  16 CTAs are the most a cluster can have (512 requests, 262144
// list entries: 14.9 us with 8, 23 with 4, 71 with one; a decode step of 64
// requests hardly differs).
constexpr int kCtas = 16;

struct TablesArgs {
  const int32_t* kv_len;
  const int32_t* new_len;
  int32_t* kv_len_out;
  int32_t* block_table;
  int64_t table_stride;
  int max_pages;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* free_count_out;
  int num_pages;
  int batch;
  int page_shift;
  int32_t* kv_indptr;
  int32_t* kv_indices;
  int64_t indices_cap;
  int32_t* q_indptr;
  int64_t* slots;
  int32_t* positions;
  int64_t max_tokens;
  int32_t* status;
};

struct Sums {
  int pages, fresh, freed;   // bounded by batch * max_pages < 2^31
  long long tokens;
  __device__ Sums operator+(const Sums& o) const {
    return {pages + o.pages, fresh + o.fresh, freed + o.freed, tokens + o.tokens};
  }
};

__device__ __forceinline__ Sums shfl_up(const Sums& s, int d) {
  return {__shfl_up_sync(~0u, s.pages, d), __shfl_up_sync(~0u, s.fresh, d), __shfl_up_sync(~0u, s.freed, d),
          __shfl_up_sync(~0u, s.tokens, d)};
}

// The last b in [0, n) with at[b] <= x; at[0] = 0 <= x, ascending.
__device__ __forceinline__ int owner(const int* at, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads, 1) tables_kernel(const TablesArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ int sm[];
  __shared__ Sums warp_sums[32];
  __shared__ int refusal;   // 1: invalid, 2: over a capacity
  const int B = a.batch, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* page_at = sm;                 // [B + 1] each: prefix sums
  int* fresh_at = page_at + B + 1;
  int* freed_at = fresh_at + B + 1;
  int* token_at = freed_at + B + 1;
  int* len = token_at + B + 1;       // [B]: the lengths before the step
  const int rank = tc::cluster_ctarank();
  const int P = 1 << a.page_shift;
  const int fc = *a.free_count;
  if (tid == 0) refusal = 0;

  // thread t scans requests [t * per, (t + 1) * per)
  const int per = (B + kThreads - 1) / kThreads;
  Sums mine[kPerThread], sum = {};
  bool invalid = fc < 0 || fc > a.num_pages, over = false;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * per + i;
    Sums s = {};
    if (i < per && b < B) {
      const int L = a.kv_len[b], n = a.new_len[b];
      len[b] = L;
      const long long old = (static_cast<long long>(L) + P - 1) >> a.page_shift;
      if (L < 0 || n < -1 || old > a.max_pages) {
        invalid = true;
      } else if (n < 0) {
        s.freed = static_cast<int>(old);
      } else {
        const long long after = static_cast<long long>(L) + n;
        const long long pages = (after + P - 1) >> a.page_shift;
        if (after > INT32_MAX || pages > a.max_pages) {
          over = true;
        } else {
          s = {static_cast<int>(pages), static_cast<int>(pages - old), 0, n};
        }
      }
    }
    mine[i] = s;
    sum = sum + s;
  }
  // (warps past the batch take no part, and leave the others the SM)
  const int warps = (B + 32 * per - 1) / max(32 * per, 1);
  Sums incl = sum;
  if (warp < warps) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sums o = shfl_up(incl, d);
      if (lane >= d) incl = incl + o;
    }
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    Sums w = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sums o = shfl_up(w, d);
      if (lane >= d) w = w + o;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  const Sums total = warp_sums[31];
  Sums at = {};
  if (warp) at = warp_sums[warp - 1];
  at = at + incl;
  at = {at.pages - sum.pages, at.fresh - sum.fresh, at.freed - sum.freed, at.tokens - sum.tokens};
  // (a token count past INT32_MAX is past max_tokens: the step is refused)
  if (tid == 0) page_at[0] = fresh_at[0] = freed_at[0] = token_at[0] = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * per + i;
    at = at + mine[i];
    if (i < per && b < B) {
      page_at[b + 1] = at.pages;
      fresh_at[b + 1] = at.fresh;
      freed_at[b + 1] = at.freed;
      token_at[b + 1] = static_cast<int>(at.tokens);
    }
  }
  const long long top = static_cast<long long>(fc) + total.freed;   // the stack's height before pages are taken
  invalid = invalid || top > a.num_pages;
  over = over || total.fresh > top || total.pages > a.indices_cap || total.tokens > a.max_tokens;
  if (invalid) atomicOr(&refusal, 1);
  if (over) atomicOr(&refusal, 2);
  __syncthreads();                                  // also publishes the sums
  const int refused = refusal;
  if (rank == 0 && tid == 0)
    *a.status = refused & 1 ? MLA_ERR_INVALID_ARG : refused ? MLA_ERR_CAPACITY : MLA_OK;
  // Once every CTA has arrived here, all have read the lengths and the count:
  // they may be written in place, and the status by a thread that finds a bad
  // page id.
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  auto all_have_read = [] { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); };

  // warps in turn over the CTAs, so that few elements use all of them
  const int gwarp = warp * kCtas + rank;
  const long long gid = 32ll * gwarp + lane;
  constexpr int kAll = kCtas * kThreads;
  if (refused) {
    for (long long t = gid; t < a.max_tokens; t += kAll) {
      a.slots[t] = -1;
      a.positions[t] = 0;
    }
    all_have_read();
    for (long long b = gid; b < B; b += kAll) a.kv_len_out[b] = len[b];
    if (gid == 0) *a.free_count_out = fc;
    return;
  }

  // the r-th page returned, and the j-th page taken
  auto returned = [&](int r) {
    const int b = owner(freed_at, B, r);
    return a.block_table[b * a.table_stride + (r - freed_at[b])];
  };
  auto taken = [&](int j) {
    const int v = static_cast<int>(top) - 1 - j;
    return v < fc ? a.free_pages[v] : returned(v - fc);
  };
  bool bad = false;

  // page lists: each warp a run of whole 32-entry rows of the flat list (a list
  // may end so near 2^31 entries that a step past its end does not fit an int)
  {
    constexpr int kWarps = kAll / 32;
    const long long run = ((total.pages + kWarps - 1ll) / kWarps + 31) / 32 * 32;
    const long long lo = gwarp * run;
    const int e1 = static_cast<int>(lo + run < total.pages ? lo + run : total.pages);
    int e = static_cast<int>(lo < total.pages ? lo : total.pages);
    if (e < e1) {
      for (int b = owner(page_at, B, e); e < e1; ++b) {
        const int base = page_at[b], end = page_at[b + 1] < e1 ? page_at[b + 1] : e1;
        const int old = page_at[b + 1] - base - (fresh_at[b + 1] - fresh_at[b]);
        int32_t* row = a.block_table + b * a.table_stride;
        unsigned i = static_cast<unsigned>(e) + lane;
        const unsigned known = min(end, base + old);
        for (; i - lane + 128 <= known; i += 128) {   // four reads in flight
          int page[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) page[k] = row[i - base + 32 * k];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            bad |= page[k] < 0 || page[k] >= a.num_pages;
            a.kv_indices[i + 32 * k] = page[k];
          }
        }
        for (; i < static_cast<unsigned>(end); i += 32) {
          const int col = i - base;
          int page;
          if (col < old) {
            page = row[col];
          } else {
            page = taken(fresh_at[b] + col - old);
            row[col] = page;
          }
          bad |= page < 0 || page >= a.num_pages;
          a.kv_indices[i] = page;
        }
        e = end;
      }
    }
  }

  // the pages returned beyond those taken stay on the stack
  const int kept = total.freed - total.fresh;
  for (long long r = gid; r < kept; r += kAll) a.free_pages[fc + r] = returned(static_cast<int>(r));

  // slots and positions of the new tokens
  for (long long t = gid; t < a.max_tokens; t += kAll) {
    int64_t slot = -1;
    int pos = 0;
    if (t < total.tokens) {
      const int b = owner(token_at, B, static_cast<int>(t));
      pos = len[b] + (static_cast<int>(t) - token_at[b]);
      const int col = pos >> a.page_shift;
      const int old = page_at[b + 1] - page_at[b] - (fresh_at[b + 1] - fresh_at[b]);
      const int page = col < old ? a.block_table[b * a.table_stride + col] : taken(fresh_at[b] + col - old);
      if (page >= 0 && page < a.num_pages) slot = (static_cast<int64_t>(page) << a.page_shift) + (pos & (P - 1));
      else bad = true;
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }

  all_have_read();
  for (long long b = gid; b <= B; b += kAll) {
    a.kv_indptr[b] = page_at[b];
    a.q_indptr[b] = token_at[b];
    if (b < B) a.kv_len_out[b] = freed_at[b + 1] > freed_at[b] ? 0 : len[b] + (token_at[b + 1] - token_at[b]);
  }
  if (gid == 0) *a.free_count_out = static_cast<int>(top) - total.fresh;
  if (bad) *a.status = MLA_ERR_DEVICE_BOUNDS;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status_t mla_build_tables(const int32_t* kv_len, const int32_t* new_len, int32_t* kv_len_out,
                                         int32_t* block_table, int64_t table_stride, int max_pages,
                                         int32_t* free_pages, const int32_t* free_count, int32_t* free_count_out,
                                         int num_pages, int batch, int page_size, int32_t* kv_indptr,
                                         int32_t* kv_indices, int64_t indices_cap, int32_t* q_indptr, int64_t* slots,
                                         int32_t* positions, int64_t max_tokens, int32_t* status, void* stream) {
  if (num_pages < 1 || max_pages < 1 || page_size < 1 || batch < 0 || table_stride < max_pages || indices_cap < 0 ||
      max_tokens < 0)
    return MLA_ERR_INVALID_ARG;
  if (page_size != 16 && page_size != 32 && page_size != 64) return MLA_ERR_UNSUPPORTED;
  if (batch > kMaxBatch || static_cast<int64_t>(batch) * max_pages > INT32_MAX || max_tokens > INT32_MAX)
    return MLA_ERR_CAPACITY;
  if (!free_pages || !free_count || !free_count_out || !kv_indptr || !q_indptr || !status ||
      (batch > 0 && (!kv_len || !new_len || !kv_len_out || !block_table)) || (indices_cap > 0 && !kv_indices) ||
      (max_tokens > 0 && (!slots || !positions)))
    return MLA_ERR_INVALID_ARG;
  TablesArgs a{};
  a.kv_len = kv_len;
  a.new_len = new_len;
  a.kv_len_out = kv_len_out;
  a.block_table = block_table;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.free_count_out = free_count_out;
  a.num_pages = num_pages;
  a.batch = batch;
  a.page_shift = page_size == 16 ? 4 : page_size == 32 ? 5 : 6;
  a.kv_indptr = kv_indptr;
  a.kv_indices = kv_indices;
  a.indices_cap = indices_cap;
  a.q_indptr = q_indptr;
  a.slots = slots;
  a.positions = positions;
  a.max_tokens = max_tokens;
  a.status = status;
  const size_t smem = sizeof(int) * (5 * static_cast<size_t>(batch) + 4);
  // (the same limits in every call: calls may run at once on several threads)
  cudaError_t e = cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && smem > 32 * 1024)
    e = cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(int)) * (5 * kMaxBatch + 4));
  if (e == cudaSuccess)
    e = launch_dependent(tables_kernel, kCtas, kThreads, smem, kCtas, static_cast<cudaStream_t>(stream), a);
  return finish_call(e, 0, nullptr);
}
