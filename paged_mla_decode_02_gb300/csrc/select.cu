// The choice of the pages that a sparse decode reads: mla_page_scores (a
// page's best score over the heads of a query, against the page's mean row)
// and mla_select_pages (the best scoring pages of each row as a page list).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "device_utils.cuh"
#include "issue.cuh"
#include "launch.h"
#include "mla_internal.h"
#include "mla_paging.h"
#include "tc_utils.cuh"
#include "tmap.h"

namespace mla {
namespace {

constexpr int kMaxRows = 4096;
constexpr int64_t kMaxList = 1 << 30;   // pages of a list

// Row r's page list: its first entry and length, or nothing (reported) when
// it leaves kv_indices or is longer than `longest`.
struct Lists {
  const int32_t* indptr;
  const int32_t* indices;
  int64_t n_indices;
  int64_t longest;
  int32_t* err;
};
__device__ __forceinline__ int list_of(const Lists& l, int r, int* first) {
  const int b = l.indptr[r], e = l.indptr[r + 1];
  *first = b;
  if (b >= 0 && e >= b && e <= l.n_indices && e - b <= l.longest) return e - b;
  report_error(l.err, kErrBounds);
  return 0;
}

// ---------------------------------------------------------------------------
// Scores
// ---------------------------------------------------------------------------
//
// A row's scores are the row maxima of S = summaries[pages] . q^T, a product
// of M = pages, N = heads, K = 576 that reads 1152 bytes per page: bound by
// HBM, and next by what passes from L2 to the SMs.  The rows' lists are cut
// into tiles of up to 128 pages, and the CTAs take whole tiles in order, some one
// more than others.  (Few or short lists make smaller tiles, so that all SMs take
// part: the size, of four, with the least estimated time of the fullest CTA.)
// - One warp copies a row's queries into shared memory by TMA, in nine panels
//   of 64 dims that stay for all tiles of the row (and make way, four by four,
//   for the next row's).
// - Two sets of four warps copy the pages' rows, a 64-dim chunk at a time,
//   through a ring of panels with cp.async.  (As tile::gather4 copies the TMA
//   took 90 cycles for four 128-byte rows, half the speed.)
// - One warp issues the tcgen05 MMAs into one of two TMEM accumulators.
// - Four warps read the other: a TMEM lane holds one page's products with
//   all heads, so a thread takes its page's maximum without any exchange.
// With more than 48 heads the queries would leave room for four panels of the
// nine of a tile, too few to cover the latency of memory, so a share is taken
// by a CTA pair (kPair, cta_group::2): tiles have up to 256 pages, halved
// between the two CTAs, as are the heads of the queries that each holds, and
// the even CTA issues MMAs of M = 256 that read both.
// Measured: 64 rows x 1024 pages x 128 heads, 85 MB, 17.7 us (4.8 TB/s, of
// which about 5 us until the first tile has arrived; then the rate of HBM, at
// which 28 of the 76 pairs take four tiles and the others three: 19 % above the
// mean); with 16 heads, 77 MB, 16.4 us (152 CTAs, four tiles of 128 for 56 of
// them); 4 rows x 100 pages x 16 heads 5.7 us.
struct ScoreArgs {
  const char* summaries;
  int num_pages;
  Lists lists;
  int rows, heads;
  float* scores;
  int64_t stride;
};

constexpr int kScoreThreads = 448;      // warp 0 queries, warp 1 MMAs, warps 2..5 maxima, 6..13 pages
constexpr int kCopyWarps = 4;           // of each of two sets that take turns
constexpr int kTilePages = 128;         // the MMA's M
constexpr int kChunks = kD / 64;        // panels of 64 dims
constexpr int kPanelBytes = kTilePages * 128;
constexpr int kQPanels = 4, kQGroups = (kChunks + kQPanels - 1) / kQPanels;   // panels of queries copied at once
constexpr int kSizes = 4;               // tile sizes to choose from: quarters of the largest
constexpr unsigned kMostTiles = (1u << 26) + 1024;   // 2^31 pages of kv_indices in tiles of 32, and a part for each row
constexpr int kTileCost = 48;           // what a tile costs beyond its pages, in pages
constexpr int kFewHeads = 48;           // as many as one CTA serves
constexpr int kScoreRows = 640;         // rows of a launch: their lists' places are in shared memory
template <bool kPair>
struct ScoreForm {
  static constexpr int kCtas = kPair ? 2 : 1, kStages = kChunks;   // panels of the ring: a tile's
  // full (pages, queries) and accumulator-free barriers count in the even CTA
  enum { kFull = 0, kEmpty = kStages, kQFull = 2 * kStages, kQEmpty = kQFull + kQGroups, kTFull = kQEmpty + kQGroups,
         kTEmpty = kTFull + 2, kFinal = kTEmpty + 2, kBars };
  // heads that a CTA holds (the MMA's N over the CTAs, each a multiple of 16)
  __host__ __device__ static constexpr int heads_held(int heads) {
    return (heads + 16 * kCtas - 1) / (16 * kCtas) * 16;
  }
  __host__ __device__ static constexpr int smem(int heads, int rows) {
    return kStages * kPanelBytes + kChunks * heads_held(heads) * 128 + 8 * kBars + 16 + 4 * (3 * rows + 1) + 1024;
  }
};

struct Tile {
  int row, page0, pages;   // pages page0 .. page0 + pages - 1 of the row's list
  bool enters, leaves;     // the first, the last tile of the row in this share
};

#ifdef MLA_STALL_TEST
// Test build only: when nonzero, one CTA (the first, or the second if negative)
// leaves out the signal of its n-th chunk of pages (n = 1 ..), or, from
// kStallQueries up, its copy of group n - kStallQueries of its first row's
// queries: the waits for them run out.
__device__ int g_scores_stall;
constexpr int kStallQueries = 1000;
#endif

// 16 bytes into shared memory, the 256 around them into L2: the next chunk of
// the row follows.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <bool kPair>
__global__ void __launch_bounds__(kScoreThreads, 1)
    scores_kernel(const __grid_constant__ CUtensorMap map_qn, const __grid_constant__ CUtensorMap map_qp,
                  const ScoreArgs a) {
  using namespace tc;
  using F = ScoreForm<kPair>;
  constexpr int kStages = F::kStages;
  constexpr int kCopiesAhead = kStages / 2 - 1;   // chunks of pages a copying thread leaves in flight
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int held = F::heads_held(a.heads);               // heads whose queries this CTA holds
  const int q_panel = held * 128;                        // bytes of a panel of them
  const int used = kStages * kPanelBytes + kChunks * q_panel;
  const uint32_t base = smem_u32(sm), q_base = base + kStages * kPanelBytes;
  const uint32_t bars = base + used;
  auto bar = [&](int i) { return bars + 8 * i; };
  unsigned char* after = sm + used + 8 * F::kBars;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(after);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(after + 4);
  int* at = reinterpret_cast<int*>(after + 16);          // [rows + 1]: tiles before each row
  int* first_of = at + a.rows + 1;                       // [rows]: where its list begins, and its pages
  int* len_of = first_of + a.rows;
  __shared__ int warp_sum[kScoreThreads / 32], dealt[2];
  __shared__ unsigned size_sum[kSizes][kScoreThreads / 32];
  const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
  const int rank = kPair ? static_cast<int>(cluster_ctarank()) : 0;
  auto wait = [&](int i, int parity) {
    return kPair ? mbar_wait_cl_warp(bar(i), parity, abort_flag) : mbar_wait_warp(bar(i), parity, abort_flag);
  };
  auto spin = [&](int i, int parity) { return mbar_spin<kPair>(bar(i), parity, abort_flag); };
  // A role whose wait ran out issues nothing more that another CTA or a later
  // wait would have to see land; it reports that, and tells the pair's other CTA.
  auto give_up = [&]() {
    if (lane == 0) {
      report_error(a.lists.err, kErrTimeout);
      *abort_flag = 1;
      if (kPair) st_cluster_u32(map_to_rank(smem_u32(const_cast<const int*>(abort_flag)), rank ^ 1), 1);
    }
  };
#ifdef MLA_STALL_TEST
  const int stall = static_cast<int>(blockIdx.x) == (g_scores_stall < 0) ? abs(g_scores_stall) : 0;
#else
  constexpr int stall = 0, kStallQueries = 0;
#endif
  auto arrive_even = [&](int i) {   // at the even CTA's barrier
    if (kPair) mbar_arrive_remote(map_to_rank(bar(i), 0)); else mbar_arrive(bar(i));
  };
  auto commit = [&](int i, int ctas = 3) {   // at the CTAs' barriers (a bit for each)
    if (kPair) commit_pair_elect(bar(i), ctas); else mma_commit_elect(bar(i));
  };
  if (tid == 0) *abort_flag = 0;
  if (tid < F::kBars) {
    mbar_init(bar(tid), tid < F::kEmpty                                ? kCopyWarps * F::kCtas
                        : tid == F::kTEmpty || tid == F::kTEmpty + 1 ? 4 * F::kCtas
                                                                     : 1);
    fence_barrier_init();
  }
  __syncwarp();
  if (kPair) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // the barriers are there
  // (what came before touches no memory of the previous kernel's)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int unit = blockIdx.x / F::kCtas, units = gridDim.x / F::kCtas;
  int total = 0, tile = kTilePages * F::kCtas;
  if (warp >= 2 && warp < 6) {
    // Tensor memory is taken before the next kernel may be scheduled and after
    // the previous one is done: a CTA that shares the SM with one of theirs
    // can neither hold what that one waits for nor wait for it.
    if (warp == 5) {
      if (kPair) tmem_alloc_pair(smem_u32(tmem_slot), 2 * kMaxHeads);
      else tmem_alloc(smem_u32(tmem_slot), 2 * kMaxHeads);
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    // Meanwhile the rows of the first tile start on their way to L2, if the
    // lists lie end to end and are tiles of full size; where that is a little
    // off, another CTA reads what comes.
    const int64_t base0 = a.lists.indptr[0], line = a.lists.indptr[a.rows] - base0;
    if (base0 >= 0 && line >= units * (tile / 2)) {
      const int tiles = static_cast<int>((line + tile - 1) / tile), each = tiles / units;
      const int64_t p = static_cast<int64_t>(unit * each + min(unit, tiles % units)) * tile + rank * kTilePages + tid - 64;
      if (p < line && base0 + p < a.lists.n_indices) {
        const int id = a.lists.indices[base0 + p];
        if (id >= 0 && id < a.num_pages) {
          const char* row = a.summaries + static_cast<int64_t>(id) * (2 * kD);
#pragma unroll
          for (int k = 0; k < kChunks; ++k) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + 128 * k));
        }
      }
    }
  } else {
    // The other warps: how many tiles of each size the lists make (32 bits
    // hold a warp's), the size to take, and the tiles before each row.
    constexpr int kWarps = kScoreThreads / 32 - 4, kPer = kScoreRows / (32 * kWarps);   // kPer: rows of a thread
    static_assert(kPer * 32 * kWarps == kScoreRows, "every row has a thread");
    constexpr int kQuarter = kTilePages * F::kCtas / kSizes;
    const int w = warp < 2 ? warp : warp - 4, r0 = (32 * w + lane) * kPer;
    unsigned len[kPer], sum[kSizes] = {};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = r0 + i;
      int first = 0;
      len[i] = r < a.rows ? list_of(a.lists, r, &first) : 0;
      if (r < a.rows) {
        first_of[r] = first;
        len_of[r] = len[i];
      }
#pragma unroll
      for (int k = 0; k < kSizes; ++k) sum[k] += (len[i] + (k + 1) * kQuarter - 1) / ((k + 1) * kQuarter);
    }
#pragma unroll
    for (int k = 0; k < kSizes; ++k) {
      sum[k] = __reduce_add_sync(~0u, sum[k]);
      if (lane == 0) size_sum[k][w] = sum[k];
    }
    named_bar_sync(1, 32 * kWarps);
    int quarters = kSizes, all = 0;
    float least = 0.f;
    bool sound = true;
#pragma unroll
    for (int k = kSizes; k > 0; --k) {
      const unsigned some = lane < kWarps ? size_sum[k - 1][lane] : 0;
      // a warp's rows make no more tiles than kv_indices can hold, or their
      // lists overlap (kv_indptr goes back)
      sound &= !__any_sync(~0u, some > kMostTiles);
      const int n = __reduce_add_sync(~0u, some);
      const float cost = ceilf(static_cast<float>(n) / units) * (k * kQuarter + kTileCost);
      if (k == kSizes || cost < least) {
        quarters = k;
        least = cost;
        all = n;
      }
    }
    auto tiles_of = [&](unsigned pages) -> int {   // of a list
      const unsigned t = (pages + kQuarter - 1) / kQuarter;
      return quarters == 1 ? t : quarters == 2 ? (t + 1) >> 1 : quarters == 3 ? (t + 2) / 3 : (t + 3) >> 2;
    };
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mine += tiles_of(len[i]);
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(~0u, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) warp_sum[w] = incl;
    named_bar_sync(1, 32 * kWarps);
    int before = incl - mine + __reduce_add_sync(~0u, lane < w ? warp_sum[lane] : 0);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      before += tiles_of(len[i]);
      if (r0 + i < a.rows) at[r0 + i + 1] = before;
    }
    if (w == 0 && lane == 0) {
      at[0] = 0;
      dealt[0] = sound ? all : 0;
      dealt[1] = quarters * kQuarter;
      if (!sound) report_error(a.lists.err, kErrBounds);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (kPair) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  total = dealt[0];   // tiles, and their size in pages
  tile = dealt[1];
  // this CTA's (pair's) share of them
  const int each = total / units, more = total % units;
  const int begin = unit * each + min(unit, more), end = begin + each + (unit < more);
  int pos = begin, row = 0;
  if (pos < end) {   // the row that holds tile pos
    int hi = a.rows;
    while (hi - row > 1) {
      const int mid = (row + hi) >> 1;
      if (at[mid] <= pos) row = mid; else hi = mid;
    }
  }
  // the tiles of the share, in order (every role walks the same ones)
  auto next = [&](Tile& t) {
    if (pos >= end) return false;
    while (at[row + 1] <= pos) ++row;
    const int page0 = (pos - at[row]) * tile, n = min(tile, len_of[row] - page0);
    t = {row, page0, n, pos == at[row] || pos == begin, pos + 1 == at[row + 1] || pos + 1 == end};
    if (kPair) {   // this CTA's half (of a single page: none)
      const int half = (n + 1) >> 1;
      t.pages = rank ? n - half : half;
      if (rank && t.pages) t.page0 += half;
    }
    ++pos;
    return true;
  };
  bool ok = true;
  Tile t;

  if (warp == 0) {
    // ---------------- queries ----------------
    // (here and below, votes make the loops' conditions uniform to the compiler)
    int visit = 0;   // rows entered
    while (ok && __any_sync(~0u, next(t))) {
      if (!__any_sync(~0u, t.enters)) continue;
#pragma unroll
      for (int g = 0; g < kQGroups; ++g) {
        // (armed again while its last copy was still expected, a barrier would count wrongly)
        ok = ok && __all_sync(~0u, spin(F::kQEmpty + g, (visit & 1) ^ 1));
        if (!ok) continue;
        const int y = t.row * a.heads + rank * held, full = F::kQFull + g;
        const int bytes = (g < kQGroups - 1 ? kQPanels : 1) * q_panel * F::kCtas;
        const void* map = g < kQGroups - 1 ? &map_qn : &map_qp;
        if (rank == 0 && lane == 0) mbar_arrive_expect_tx(bar(full), bytes);
        __syncwarp();
        const uint32_t dst = q_base + g * kQPanels * q_panel;
        const int z = g < kQGroups - 1 ? g * kQPanels : 0;
        if (stall && visit == 0 && stall == kStallQueries + g) continue;
        if (kPair) tma_load_3d_pair_elect(dst, map, 0, y, z, map_to_rank(bar(full), 0));
        else tma_load_3d_elect(dst, map, 0, y, z, bar(full));
      }
      ++visit;
    }
    if (!ok) give_up();
    if (ok && rank == 0 && lane == 0) {   // every copy issued has landed before the CTA leaves
#pragma unroll 1
      for (int g = 0; g < kQGroups && visit > 0; ++g) {
        const uint32_t b = bar(F::kQFull + g), parity = (visit - 1) & 1;
        if (kPair) mbar_wait_cl_drain(b, parity); else mbar_wait_drain(b, parity);
      }
    }
    __syncwarp();
  } else if (warp >= 6) {
    // ---------------- pages ----------------
    // Two sets of four warps take turns, a chunk each.  Thread i of a set
    // copies 16-byte column i % 8 of rows i / 8 + 16 j.
    const int set = (warp - 6) / kCopyWarps, i = (tid - 6 * 32) % (32 * kCopyWarps), col = i & 7, row0 = i >> 3;
    const uint32_t dst = base + row0 * 128 + ((col ^ (row0 & 7)) << 4);
    // the ids of a tile's pages that this thread copies (a wrong one reads page
    // 0; scored -inf below)
    int ids[8];
    auto read_ids = [&](const Tile& x) {
      const int32_t* list = a.lists.indices + first_of[x.row] + x.page0;
#pragma unroll
      for (int j = 0; j < 8; ++j) ids[j] = list[max(0, min(row0 + 16 * j, x.pages - 1))];
    };
    int turn = set, slot = set % kStages, phase = 1;        // the set's next chunk: its number, slot and phase
    int landing = set % kStages, pending = 0, first = 0;    // first: number of the tile's first chunk
    int landed = set - 1;                                   // chunks landed, of both sets
    auto land = [&]() {   // the set's oldest chunk in flight is in place
      fence_proxy_async_smem();
      __syncwarp();
      landed += 2;
      if (lane == 0 && !(stall && stall == landed)) arrive_even(F::kFull + landing);
      landing += 2;
      if (landing >= kStages) landing -= kStages;
      --pending;
    };
    bool more = next(t);
    if (more) read_ids(t);
    while (ok && more) {
      const char* src[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t id = ids[j] < 0 || ids[j] >= a.num_pages ? 0 : ids[j];
        src[j] = a.summaries + id * (2 * kD) + 16 * col + 128 * (turn - first);
      }
      const int rows16 = (t.pages + 15) >> 4;
      if ((more = next(t))) read_ids(t);   // the next tile's are on their way meanwhile
#pragma unroll 1
      for (; turn < first + kChunks; turn += 2) {
        if (!(ok = wait(F::kEmpty + slot, phase))) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j < rows16) copy16(dst + slot * kPanelBytes + j * 2048, src[j]);
          src[j] += 256;
        }
        cp_async_commit();
        slot += 2;
        if (slot >= kStages) {
          slot -= kStages;
          phase ^= 1;
        }
        if (++pending > kCopiesAhead) {
          cp_async_wait<kCopiesAhead>();
          land();
        }
      }
      first += kChunks;
    }
    cp_async_wait<0>();
    while (ok && pending > 0) land();
    if (!ok) give_up();
  } else if (warp == 1) {
    // ---------------- MMAs (a pair: in its even CTA) ----------------
    const uint32_t idesc = idesc_bf16_f32(kTilePages * F::kCtas, held * F::kCtas, false, false);
    int n = 0, visit = -1;   // tiles, and rows entered, before this one
    for (; rank == 0 && ok && __any_sync(~0u, next(t)); ++n) {
      const int acc = n & 1;
      const bool enters = __any_sync(~0u, t.enters), leaves = __any_sync(~0u, t.leaves);
      visit += enters;
      ok &= spin(F::kTEmpty + acc, ((n >> 1) & 1) ^ 1);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {   // panel c of the ring holds chunk c of every tile
        if (enters && c % kQPanels == 0) ok &= spin(F::kQFull + c / kQPanels, visit & 1);
        ok &= spin(F::kFull + c, n & 1);
        tc_fence_after();
        const uint64_t da = smem_desc(base + c * kPanelBytes, 16, 1024, kSw128);
        const uint64_t dq = smem_desc(q_base + c * q_panel, 16, 1024, kSw128);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kPair) mma_pair_elect(tmem + acc * kMaxHeads, da + 2 * kk, dq + 2 * kk, idesc, (c | kk) != 0);
          else mma_ss_elect(tmem + acc * kMaxHeads, da + 2 * kk, dq + 2 * kk, idesc, (c | kk) != 0);
        }
        commit(F::kEmpty + c);
        if (leaves && (c % kQPanels == kQPanels - 1 || c == kChunks - 1)) {
          // (not where the issuing lane's wait ran out: their copy may still be expected)
          const uint32_t empty = bar(F::kQEmpty + c / kQPanels);
          if (kPair) commit_pair_elect_if(empty, 3, ok); else mma_commit_elect_if(empty, ok);
        }
      }
      commit(F::kTFull + acc);
      ok = __all_sync(~0u, ok);
    }
    if (!ok) give_up();
    if (rank == 0) {
      commit(F::kFinal, 1);   // every MMA issued completes before TMEM is freed
      if (lane == 0) {
        if (kPair) mbar_wait_cl_drain(bar(F::kFinal), 0); else mbar_wait_drain(bar(F::kFinal), 0);
      }
    }
    __syncwarp();
  } else {
    // ---------------- maxima: page 32 quad + lane of the tile ----------------
    const int quad = warp & 3;
    for (int n = 0; ok && next(t); ++n) {
      const int acc = n & 1, p = 32 * quad + lane;
      int id = -1;
      if (p < t.pages) id = a.lists.indices[first_of[t.row] + t.page0 + p];
      if (!(ok = wait(F::kTFull + acc, (n >> 1) & 1))) break;
      tc_fence_after();
      float best = -INFINITY;
      if (32 * quad < t.pages) {
#pragma unroll 1
        for (int c = 0; c < a.heads; c += 32) {
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
      if (lane == 0) arrive_even(F::kTEmpty + acc);
      if (p < t.pages) {
        if (id < 0 || id >= a.num_pages) {
          report_error(a.lists.err, kErrBounds);
          best = -INFINITY;
        }
        a.scores[t.row * a.stride + t.page0 + p] = best;
      }
    }
    if (!ok) give_up();
  }
  tc_fence_before();
  if (kPair) cluster_sync_all(); else __syncthreads();   // (a pair: neither reads the other's memory any more)
  if (warp == 5) {
    tc_fence_after();
    if (kPair) tmem_dealloc_pair(tmem, 2 * kMaxHeads);
    else tmem_dealloc(tmem, 2 * kMaxHeads);
  } else if (warp == 0 && *abort_flag) {
    // Where a wait ran out, here or in the pair's other CTA, copies of queries
    // may be on their way whose barrier nobody waited for: no more are issued
    // now, and the shared memory is held until they must have landed.
    pause_ns(kDrainLimitNs);
  }
}

// Row-major [rows, 64 panels] bf16 as (dim of a panel, row, panel): a box of
// some rows and panels lands panel by panel, each in rows of 128 bytes with the
// 128-byte swizzle.
bool encode_panels(CUtensorMap* m, const void* base, int64_t rows, int panels, int box_rows, int box_panels) {
  EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(panels)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(panels) * 128, 128};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(box_panels)};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
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

// Scores as unsigned keys in the same order: NaN as -inf, -0 as 0.  Never 0.
__device__ __forceinline__ uint32_t key_of(float s) {
  if (s != s) s = -INFINITY;
  const uint32_t u = __float_as_uint(s + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Rows of scores up to this long take a CTA of 256 threads, longer ones of 1024
// (256 rows of 1024 pages: 5.5 us against 6.6; 64 rows of 2048: 6.8 against 5.5).
constexpr int64_t kNarrow = 1024;
constexpr int kFewLeft = 128;            // pages ranked against each other
constexpr int kStagedPages = 49152;      // keys that fit a CTA's shared memory

// One CTA per row.  The middle pages are ordered by key, then by position:
// the composite of a page is its key above its distance from the row's end, so
// no two are equal and the want-th highest composite, the cut, parts kept from
// left.  It is found by digits of eight bits, from the first bit in which the
// keys differ down: a histogram of the digit over the pages that agree with
// the digits found so far (in shared memory, in integers: their order does not
// show), and the digit in which the want-th falls.  That ends when all pages
// of the digit are wanted, or when few are left, which are then ranked against
// each other.  Each warp holds a run of the row's pages in order, so counts
// of the warps before it place what it keeps.
// The keys stay in shared memory (kStaged) or, for longer rows, are read again
// from L2 in each pass.  What bounds the kernel is latency -- three dependent
// reads of memory, two barriers a pass -- and its code: loops stay rolled, as
// most of their lines run once or twice.
template <int kThreads, bool kStaged>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kWarps = kThreads / 32, kUnroll = kStaged ? 2 : 8;
  extern __shared__ uint32_t staged[];
  __shared__ __align__(16) int hist[2][256];             // read four at a time
  __shared__ int sums[kWarps], places[kWarps], digit_of, need_of, left_of, few;
  __shared__ uint32_t ors[kWarps], ands[kWarps];
  __shared__ unsigned long long rest[kFewLeft], cut_of;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = blockIdx.x;
  for (int i = tid; i < 512; i += kThreads) hist[0][i] = 0;
  if (tid == 0) few = 0;
  int first;
  const int n = list_of(a.lists, r, &first);
  const float* s = a.scores + r * a.stride;
  const int32_t* pages = a.lists.indices + first;
  const int lo = a.keep_first, hi = n - a.keep_last;   // the middle: [lo, hi)
  const bool all = n <= a.top_k;

  // this warp's run: `steps` times 32 pages from `base`; keys of the middle
  // pages, 0 for the others
  const int steps = (n + kThreads - 1) / kThreads;
  const int base = warp * steps * 32 + lane;
  auto read_key = [&](int p) { return p >= lo && p < hi ? key_of(s[p]) : 0u; };
  auto key_at = [&](int p) { return kStaged ? staged[p] : read_key(p); };
  uint32_t any = 0, every = ~0u;
  if (!all) {
#pragma unroll 8
    for (int e = 0; e < steps; ++e) {
      const uint32_t k = read_key(base + 32 * e);
      if (kStaged) staged[base + 32 * e] = k;
      any |= k;
      every &= k ? k : ~0u;
    }
  }
  // what the rows before this one keep, and the bits in which keys differ
  int before = 0, unused;
  for (int i = tid; i < r; i += kThreads) before += min(a.top_k, list_of(a.lists, i, &unused));
  before = __reduce_add_sync(~0u, before);
  any = __reduce_or_sync(~0u, any);
  every = __reduce_and_sync(~0u, every);
  if (lane == 0) {
    sums[warp] = before;
    ors[warp] = any;
    ands[warp] = every;
  }
  __syncthreads();
  before = __reduce_add_sync(~0u, lane < kWarps ? sums[lane] : 0);
  if (tid == 0) {
    if (r == 0) a.sel_indptr[0] = 0;
    a.sel_indptr[r + 1] = before + min(a.top_k, n);
  }
  int32_t* out = a.sel_indices + before;
  if (all) {
    for (int p = tid; p < n; p += kThreads) out[p] = pages[p];
    return;
  }
  any = __reduce_or_sync(~0u, lane < kWarps ? ors[lane] : 0u);
  every = __reduce_and_sync(~0u, lane < kWarps ? ands[lane] : ~0u);

  auto composite = [&](uint32_t k, int p) {
    return static_cast<unsigned long long>(k) << 32 | static_cast<uint32_t>(n - 1 - p);
  };
  unsigned long long cut = ~0ull;   // above every composite: none of the middle
  int need = a.top_k - a.keep_first - a.keep_last;
  if (need > 0) {
    const int tail = 31 - __clz(n);                         // the highest bit of a distance, or above it
    int top = any != every ? 63 - __clz(any ^ every) : tail;
    cut = composite(every, n - 1);                          // with what the keys have in common alone
    if (any != every) cut = top == 63 ? 0 : cut >> (top + 1) << (top + 1);
    for (int side = 0;; side ^= 1) {
      const int shift = max(top - 7, top >= 32 ? 32 : 0);   // a digit lies within the key or the distance
      const uint32_t digits = (2u << (top - shift)) - 1;
      if (shift >= 32) {   // a digit of the key: 32 bits are enough
        const uint32_t have = static_cast<uint32_t>(cut >> 32);
#pragma unroll kUnroll
        for (int e = 0; e < steps; ++e) {
          const uint32_t k = key_at(base + 32 * e);
          if (k && ((k ^ have) >> (top - 32)) < 2) atomicAdd(&hist[side][(k >> (shift - 32)) & digits], 1);
        }
      } else {
#pragma unroll kUnroll
        for (int e = 0; e < steps; ++e) {
          const int p = base + 32 * e;
          const uint32_t k = key_at(p);
          const unsigned long long c = composite(k, p);
          if (k && ((c ^ cut) >> top) < 2) atomicAdd(&hist[side][static_cast<uint32_t>(c >> shift) & digits], 1);
        }
      }
      __syncthreads();
      if (warp == 0) {
        // lane l holds the digits 8 (31 - l) .. + 7: the highest come first
        const int4* h = reinterpret_cast<const int4*>(hist[side] + 8 * (31 - lane));
        const int4 u = h[0], v = h[1];
        const int sum = u.x + u.y + u.z + u.w + v.x + v.y + v.z + v.w;
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(~0u, incl, d);
          if (lane >= d) incl += o;
        }
        // the lane that the need-th falls to, and its digits one to a lane
        const uint32_t reach = __ballot_sync(~0u, incl >= need);
        const int owner = __ffs(reach) - 1, above = __shfl_sync(~0u, incl - sum, owner);
        const int digit = 8 * (31 - owner) + 7 - (lane & 7), mine = hist[side][digit];
        incl = mine;
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) {
          const int o = __shfl_up_sync(~0u, incl, d);
          if ((lane & 7) >= d) incl += o;
        }
        incl += above;
        if (lane < 8 && incl >= need && incl - mine < need) {
          digit_of = digit;
          need_of = need - (incl - mine);
          left_of = mine;
        }
      } else {
        for (int i = tid - 32; i < 256; i += kThreads - 32) hist[side ^ 1][i] = 0;
      }
      __syncthreads();
      cut |= static_cast<unsigned long long>(digit_of) << shift;
      need = need_of;
      if (need == left_of) break;                           // all from the cut up
      top = shift == 32 ? tail : shift - 1;
      if (left_of <= kFewLeft) {
        const int stays = shift;
#pragma unroll kUnroll
        for (int e = 0; e < steps; ++e) {
          const int p = base + 32 * e;
          const uint32_t k = key_at(p);
          const unsigned long long c = composite(k, p);
          if (k && (c ^ cut) >> stays == 0) rest[atomicAdd(&few, 1)] = c;
        }
        __syncthreads();
        if (tid < few) {
          const unsigned long long mine = rest[tid];
          int rank = 0;
          for (int j = 0; j < few; ++j) rank += rest[j] > mine;
          if (rank == need - 1) cut_of = mine;
        }
        __syncthreads();
        cut = cut_of;
        break;
      }
    }
  }

  // kept pages of this warp's run, and of the warps before it
  auto keeps = [&](int p) { return p < lo || (p >= hi && p < n) || (p < hi && composite(key_at(p), p) >= cut); };
  int c = 0;
#pragma unroll kUnroll
  for (int e = 0; e < steps; ++e) c += keeps(base + 32 * e);
  c = __reduce_add_sync(~0u, c);
  if (lane == 0) places[warp] = c;
  __syncthreads();
  int place = __reduce_add_sync(~0u, lane < warp ? places[lane] : 0);
  if (c == 0) return;
  constexpr int kBatch = 4;   // page ids read before any is written
  for (int e0 = 0; e0 < steps; e0 += kBatch) {
    int id[kBatch];
    uint32_t kept = 0;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int p = base + 32 * (e0 + j);
      if (e0 + j < steps && keeps(p)) {
        kept |= 1u << j;
        id[j] = pages[p];
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const uint32_t who = __ballot_sync(~0u, kept >> j & 1);
      if (kept >> j & 1) out[place + __popc(who & ((1u << lane) - 1))] = id[j];
      place += __popc(who);
    }
  }
}

}  // namespace
}  // namespace mla

using namespace mla;

#ifdef MLA_STALL_TEST
// Test build only: the signal or copy that a CTA of scores_kernel leaves out (0: none).
extern "C" int mla_test_set_scores_stall(int n) {
  return static_cast<int>(cudaMemcpyToSymbol(g_scores_stall, &n, sizeof(n)));
}
#endif

extern "C" mla_status_t mla_page_scores(const void* q_nope, const void* q_pe, const void* summaries, int num_pages,
                                        const int32_t* kv_indptr, const int32_t* kv_indices, int64_t n_indices,
                                        int rows, int num_heads, float* scores, int64_t score_stride,
                                        int64_t max_pages, int check_status, void* stream) {
  if (rows < 0 || num_heads < 1 || num_heads > kMaxHeads || num_pages < 1 || n_indices < 0 || max_pages < 0 ||
      score_stride < max_pages)
    return MLA_ERR_INVALID_ARG;
  if (rows > kMaxRows) return MLA_ERR_CAPACITY;
  if (rows > 0 && (!q_nope || !q_pe || !summaries || !kv_indptr || (n_indices > 0 && !kv_indices) ||
                   (max_pages > 0 && !scores)))
    return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_nope) || !aligned16(q_pe) || !aligned16(summaries)) return MLA_ERR_INVALID_ARG;
  ScoreArgs a{};
  a.summaries = static_cast<const char*>(summaries);
  a.num_pages = num_pages;
  a.lists = {kv_indptr, kv_indices, n_indices, max_pages < kMaxList ? max_pages : kMaxList, nullptr};
  a.rows = rows;
  a.heads = num_heads;
  a.scores = scores;
  a.stride = score_stride;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // one CTA to a run of pages with few heads, else a pair
  const bool pair = num_heads > kFewHeads;
  const int ctas = pair ? 2 : 1;
  const int held = pair ? ScoreForm<true>::heads_held(num_heads) : ScoreForm<false>::heads_held(num_heads);
  static_assert(ScoreForm<false>::smem(kFewHeads, kScoreRows) <= 227 * 1024 - 128 &&
                ScoreForm<true>::smem(kMaxHeads, kScoreRows) <= 227 * 1024 - 128, "shared memory of a CTA");
  auto kernel = pair ? scores_kernel<true> : scores_kernel<false>;
  int sms = 0;
  cudaError_t e = rows > 0 ? current_sms(&sms) : cudaSuccess;
  if (rows > 0 && e == cudaSuccess) e = paging_error_word(&a.lists.err);
  // (the same limit in every call: calls may run at once on several threads)
  if (rows > 0 && e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             pair ? ScoreForm<true>::smem(kMaxHeads, kScoreRows) : ScoreForm<false>::smem(kFewHeads, kScoreRows));
  for (int r0 = 0; r0 < rows && e == cudaSuccess; r0 += kScoreRows) {
    a.rows = rows - r0 < kScoreRows ? rows - r0 : kScoreRows;
    a.lists.indptr = kv_indptr + r0;
    a.scores = scores + r0 * score_stride;
    const int64_t first = static_cast<int64_t>(r0) * num_heads, q_rows = static_cast<int64_t>(a.rows) * num_heads;
    CUtensorMap mn, mp;
    if (!encode_panels(&mn, static_cast<const char*>(q_nope) + first * kDCkv * 2, q_rows, kDCkv / 64, held, kQPanels) ||
        !encode_panels(&mp, static_cast<const char*>(q_pe) + first * kDKpe * 2, q_rows, 1, held, 1))
      return MLA_ERR_CUDA;
    const int smem = pair ? ScoreForm<true>::smem(num_heads, a.rows) : ScoreForm<false>::smem(num_heads, a.rows);
    // no more CTAs than the lists can have tiles of the smallest size
    const int64_t tiles = n_indices / (kTilePages * ctas / kSizes) + a.rows, most = sms / ctas;
    const int grid = ctas * static_cast<int>(tiles < most ? tiles : most);
    e = launch_dependent(kernel, grid, kScoreThreads, smem, ctas, s, mn, mp, a);
  }
  return finish_call(e, check_status, s);
}

extern "C" mla_status_t mla_select_pages(const float* scores, int64_t score_stride, int64_t max_pages,
                                         const int32_t* kv_indptr, const int32_t* kv_indices, int64_t n_indices,
                                         int rows, int top_k, int keep_first, int keep_last, int32_t* sel_indptr,
                                         int32_t* sel_indices, int64_t sel_cap, int check_status, void* stream) {
  if (rows < 0 || n_indices < 0 || max_pages < 0 || score_stride < max_pages || sel_cap < 0) return MLA_ERR_INVALID_ARG;
  if (top_k < 1 || keep_first < 0 || keep_last < 1 || static_cast<int64_t>(keep_first) + keep_last > top_k)
    return MLA_ERR_INVALID_ARG;
  if (rows > kMaxRows || static_cast<int64_t>(rows) * top_k > INT32_MAX ||
      static_cast<int64_t>(rows) * top_k > sel_cap)
    return MLA_ERR_CAPACITY;
  if (!sel_indptr || (rows > 0 && (!kv_indptr || !sel_indices || (n_indices > 0 && !kv_indices) ||
                                   (max_pages > 0 && !scores))))
    return MLA_ERR_INVALID_ARG;
  SelectArgs a{};
  a.scores = scores;
  a.stride = score_stride;
  a.lists = {kv_indptr, kv_indices, n_indices, max_pages < kMaxList ? max_pages : kMaxList, nullptr};
  a.rows = rows;
  a.top_k = top_k;
  a.keep_first = keep_first;
  a.keep_last = keep_last;
  a.sel_indptr = sel_indptr;
  a.sel_indices = sel_indices;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // (a list is no longer than max_pages; a run of 32 pages to a warp)
  const int few = 256, many = 1024;
  const bool wide = max_pages > kNarrow, staged = max_pages <= kStagedPages;
  const int threads = wide ? many : few;
  const size_t smem = staged ? (max_pages + threads - 1) / threads * threads * sizeof(uint32_t) : 0;
  cudaError_t e = cudaSuccess;
  auto kernel = !wide ? select_kernel<few, true> : staged ? select_kernel<many, true> : select_kernel<many, false>;
  // (the same limit in every call: calls may run at once on several threads)
  if (rows > 0) e = paging_error_word(&a.lists.err);
  if (e == cudaSuccess && smem > 32 * 1024)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kStagedPages * static_cast<int>(sizeof(uint32_t)));
  if (e == cudaSuccess)
    e = rows == 0 ? cudaMemsetAsync(sel_indptr, 0, sizeof(int32_t), s)
                  : launch_dependent(kernel, rows, threads, smem, 1, s, a);
  return finish_call(e, check_status, s);
}
