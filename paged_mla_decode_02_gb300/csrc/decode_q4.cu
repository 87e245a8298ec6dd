// Paged MLA decode over a 4-bit cache.
//
// For request b, query row h, over the rows k_t of the request's tokens:
//   S = sm_scale * (q_nope . k_t[0:512] + q_pe . k_t[512:576]),
//   out = softmax(S) . k[0:512],  lse = ln sum exp(S).
//
// A row's values are e2m1 numbers times 2^(E - k), k <= 14 the shift of a group
// of 32 dims.  Over 2^(E - 6) each is an e4m3 number exactly (6 * 2^6 = 384 at
// most, 0.5 * 2^-8 = 2^-9 at least), so a tile of rows becomes a tile of e4m3
// codes by table lookup, and both products are tcgen05 MMAs of kind::f8f6f4 with
// the rows as A, read from shared memory in either direction:
//   S^T [128 tokens x rows]    = K [128 tokens x 576] . Q^T       (K-major)
//   O^T [512 dims x rows]     += V^T [512 dims x 128 tokens] . P^T (MN-major)
// One expanded tile serves both, and a CTA needs M = 128 of tokens and of dims
// only, so N is as small as the number of query rows: 16, 32 or 64 to a CTA (two
// CTAs share a request of 65 to 128 rows).
//
// The other operand of each product is split into terms of 8 bits:
// - the query row, under a power of two that brings its largest magnitude into
//   [2^7, 2^8), into hi = e4m3(x) and lo = e4m3(2^5 (x - hi)).  Both are rows of the
//   same B: S^T has a column for each, and hi's + 2^-5 lo's is the score.  The rest is
//   2^3 at most, so that lo fits under the largest e4m3 number, 448; held as it is it
//   would be off by 2^-10 for elements below 2^-2, a hundredth of the largest and less,
//   which a row with one large dim has many of (scores off by 6e-3 where it is 300
//   times the others).  So hi + 2^-5 lo is the bf16 query exactly down to 2^-7, and
//   within 2^-15 below.
// - P.  With the row's unit 2^(E_t - 6) moved into it, p = 2^(s_t + E_t - ref)
//   can span many powers of two that add up over a long context, so the terms'
//   range matters as much as their bits.  Up to 32 query rows, three e5m2 terms
//   side by side in B (the columns of O^T are added in the epilogue): nine bits,
//   from 2^15 down to 2^-17.  64 rows (O^T's three terms would not fit into
//   tensor memory): two terms, two MMAs into the same columns.  hi = e5m2(p), and
//   lo, of p - hi, in one of two forms that a unit's scores choose: e4m3, eight bits
//   of p from 2^12 down to 2^-3 and ever fewer below, or e5m2, seven bits from 2^15
//   down to 2^-11.  The first suits weights of which some are of like size.  Where a
//   row has but a few large ones (tokens that all attend to, whose own values may say
//   nothing), the sum of many small ones may be the result: 64 rows with such a one
//   among them take the second for the rest of the unit.  Off by 2^-8 or 2^-7 of
//   a weight at most, 0.1 or 0.2 % of a result whose values add up like a random walk;
//   with the first form alone 0.4 % where a token stands 6 natural units above the
//   rest, 4 % at 9.
//
// The softmax's state is kept per query row: a reference that moves (and O with
// it) when a score passes it by more than kSlack, and two sums in fp32 per
// thread: of the exact p, for the lse, and of what the terms leave of it, for the
// output is divided by the sum of the p that P stands for.  A weight is p / 2^E_t,
// one more factor a token.  A p too small for all its bits counts as it is in
// both: the row of a small E_t may weigh much and hold little, so that its p is
// rounded coarsely, or away.
//
// Roles, with registers dealt out to each: 8 or 16 warps expand tiles into two or
// three buffers, with the raw rows of the next tile on their way into registers; a
// warp for each 32 tokens and 8 or 16 query rows makes P; one warp issues the MMAs of
// the scores, one those of P . V; one looks up where the rows are, four tiles ahead,
// and asks for them into L2.  Waits are bounded (2 s): a warp that gives up says so, and
// goes on without waiting, so that the named barriers and commits of the others
// still come; the results are void and MLA_ERR_DEVICE_TIMEOUT is recorded.
//
// What bounds it (device time from a graph, cold L2): the way of a tile through its
// buffer, among 28 warps that take 54 to 57 % of the issue slots.
// - 16 query rows: 4 requests of 131072 tokens take 60 us, 2.7 TB/s, 27 tiles a CTA at
//   1.5 us each and a unit's start and end.  A buffer is held for the expansion (about
//   3700 cycles of a warp), the scores (1250), P (1700) and P . V (1700); shared memory
//   has room for three.  Loads or stores left out gain 2 us, the arithmetic of P nothing.
// - 64 rows: 64 requests of 4096 tokens and 128 heads take 93 us, 0.79 PFLOP/s, 2.5 us
//   a tile.  Expansion 2250, scores 2000 (500 after it), P 3300 and P . V 2500 cycles
//   (before lo had two forms), over two buffers.  Both products read the tile and their
//   other operand through shared memory, 2700 cycles of 128 bytes a tile.  Of 105 us, all
//   MMAs left out made 82, half of the expansion left out 95.
// A unit costs 3.2 us (16 rows) to 7.2 us (64) beyond its tiles: its query and first rows,
// its last P . V, the sums, the output; the first one of a launch more, for its code is
// fetched then.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <climits>
#include <type_traits>

#include "device_utils.cuh"
#include "issue.cuh"
#include "kernels.h"
#include "launch.h"
#include "q4.cuh"

namespace mla {
namespace {

using namespace tc;

#ifdef MLA_STALL_TEST
// Test build only: when nonzero, CTA 0's first worker warp leaves out its
// g_q4_stall-th signal of an expanded tile (1-based).
__device__ int g_q4_stall;
#endif

constexpr int kT = kTileTc;                   // 128 tokens to a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// An expanding warp's rows of a tile in one word: the address of the first and,
// in the bits that no address has, how many.
__device__ __forceinline__ uint64_t pack_rows(const uint8_t* src, int n) {
  return reinterpret_cast<uint64_t>(src) | static_cast<uint64_t>(n) << 59;
}
struct Rows {
  const uint8_t* src;
  int n;
  __device__ __forceinline__ explicit Rows(uint64_t w) : src(reinterpret_cast<const uint8_t*>(w & ((1ull << 59) - 1))), n(static_cast<int>(w >> 59)) {}
};

template <int kRows>
struct Shape {
  static constexpr int kNS = 2 * kRows;                    // columns of S^T
  static constexpr bool kSide = kRows < 64;                // P's terms side by side
  static constexpr int kPN = kSide ? 3 * kRows : kRows;    // N of P . V
  static constexpr int kPRow = kRows == 32 ? 128 : 64;     // bytes of a token's row of P
  static constexpr int kPPanel = kT * kPRow;
  static constexpr SmemSwizzle kPSwizzle = kRows == 32 ? kSw128 : kSw64;
  // warps: softmax (a lane quadrant and kJ query rows each), expanding, issue (a whole
  // warpgroup, for the registers)
  static constexpr int kJ = kRows == 16 ? 8 : 16;
  static constexpr int kSoftmaxWarps = 4 * kRows / kJ;
  static constexpr int kExpandWarps = kRows == 64 ? 8 : 16;
  static constexpr int kIssueWarp = kSoftmaxWarps + kExpandWarps;
  static constexpr int kThreads = 32 * (kIssueWarp + 4);
  // With three tiles in flight the expanding warps are two groups, for the even and the
  // odd tiles: what a tile costs a warp besides its rows counts half.
  static constexpr int kGroups = kRows == 16 ? 2 : 1;
  static constexpr int kTileWarps = kExpandWarps / kGroups;
  static constexpr int kTokWarp = kT / kTileWarps;         // rows that a warp expands, of one page
  // The scores' MMAs follow the expansion in kStages steps of 4 / kStages panels.  With 64
  // rows they take 2000 cycles, of which three quarters lie beside the expansion then (96.4
  // us for 100.8, 64 requests of 4096 tokens and 128 heads; later two steps 94.7 where four
  // made 92.7).  Fewer rows have fewer to hide, and the loads, 64 bytes of a row at a time
  // instead of 256, cost more (63.9 us for 60.2, 4 requests of 131072 tokens, 16 heads; 32
  // rows the same either way).
  static constexpr int kStages = kRows == 64 ? 4 : 1;
  // registers a thread at launch, then by role
  static constexpr int kRegs = 65536 / kThreads / 8 * 8;
  static constexpr int kRegsSoftmax = kRows == 32 ? 96 : 80, kRegsExpand = kRows == 32 ? 72 : 80;
  static constexpr int kRegsIssue = 24;
  static_assert(32 * (kSoftmaxWarps * kRegsSoftmax + kExpandWarps * kRegsExpand + 4 * kRegsIssue) <= kThreads * kRegs, "registers");
  // p reaches 2^kTop: the reference is set to leave kSlack of that, and moves when it is used up
  static constexpr float kTop = kSide ? 15.f : 12.f, kSlack = kSide ? 8.f : 7.f;
  // p from here on has all its bits (the last term's least unit is 2^-16, 2^-9)
  static constexpr float kFull = kSide ? 0x1p-8f : 0x1p-2f;
  // the same with lo in e5m2, of least unit 2^-16: the largest at 2^7 leaves seven bits of
  // weights 2^-18 of it.  (A slack too small is paid for in moves, which cost a good part of a
  // tile's time.)
  static constexpr float kTopWide = 15.f, kSlackWide = 8.f, kFullWide = 0x1p-9f;
  // That suits a row with no more large weights (2^-6 of the largest) in a tile than these:
  // the others may be the result then.  Errors of e4m3's last unit, 2^-10 / sqrt(3) of up to
  // 128 weights, are 0.3 % of 17 weights of 1/2, so with more of them it does as well.
  static constexpr int kFewLarge = 16;
  // a row found to need it in the middle of a unit has two tiles to go until all rows take
  // it, and its largest p up here
  static constexpr float kSlackFew = 1.f;
  // tensor memory columns
  static constexpr int kOBlock = kRows == 16 ? 64 : kPN;   // of 128 dims
  static constexpr int kColS = 4 * kOBlock;
  static_assert(kColS + 2 * kNS <= 512, "tensor memory");
  static constexpr int kBufs = kRows == 16 ? 3 : 2;        // expanded tiles
  static constexpr int kPeBufs = kRows == 32 ? 2 : 1;      // of the rope part
  static constexpr int kRowsAhead = 4;                     // tiles whose rows are known ahead
  // barriers
  static constexpr int kKFull0 = 0;                        // [kBufs][kStages] panels of the tile expanded (a signal of each of its warps)
  static constexpr int kSFull0 = kKFull0 + kBufs * kStages;   // [2] scores made
  static constexpr int kSFree0 = kSFull0 + 2;              // [2] scores read (a signal of every softmax warp)
  static constexpr int kPReady0 = kSFree0 + 2;             // [4] P of 32 tokens written (a signal for every kJ query rows)
  // [kBufs][4] P . V over 32 tokens made: their rows of K and P may be written again (by
  // buffer: the next tile's may be made before an expanding warp looks)
  static constexpr int kPvDone0 = kPReady0 + 4;
  static constexpr int kRowsFull0 = kPvDone0 + 4 * kBufs;  // [kRowsAhead] where the expanding warps find a tile's rows
  static constexpr int kRowsFree0 = kRowsFull0 + kRowsAhead;   // that place read (a signal of each)
  static constexpr int kQReady = kRowsFree0 + kRowsAhead;  // the unit's query in place (a signal of every softmax warp)
  static constexpr int kFinal0 = kQReady + 1;              // [2] every MMA of an issuing warp made
  static constexpr int kNumBars = kFinal0 + 2;
  // shared memory
  static constexpr int kOffQ = 0;
  static constexpr int kQPanel = kNS * 128;                // 128 dims of every term
  static constexpr int kOffQPe = 4 * kQPanel;
  static constexpr int kOffP = kOffQPe + kNS * 64;
  static constexpr int kOffK = kOffP + (kSide ? 1 : 2) * kPPanel;
  static constexpr int kPanel = kT * 128;                  // 128 tokens x 128 dims
  static constexpr int kOffKPe = kOffK + kBufs * 4 * kPanel;
  // exponent bytes by buffer and token: with 16 query rows in what their row of P leaves
  static constexpr bool kExpInP = kRows == 16;
  static constexpr int kOffExp = kOffKPe + kPeBufs * kT * 64;
  static __device__ __forceinline__ int exp_at(int buf, int tok) {
    return kExpInP ? kOffP + tok * kPRow + ((3 ^ ((tok >> 1) & 3)) << 4) + buf : kOffExp + buf * kT + tok;
  }
  static constexpr int kOffScale = kOffExp + (kExpInP ? 0 : kBufs * kT);   // [2][rows] 1 / query scale, by unit parity
  static constexpr int kOffRef = kOffScale + 2 * kRows * 4;   // [rows] kTop - kSlack, less the reference
  static constexpr int kOffTable = kOffRef + kRows * 4;    // [4] e4m3 codes of the magnitudes, for shifts 12 ..
  static constexpr int kOffRed = kOffTable + 4 * 8;        // [softmax warps][kJ] floats
  static constexpr int kOffRows = kOffRed + kSoftmaxWarps * kJ * 4;   // [kRowsAhead][warps of a tile] packed rows
  static constexpr int kOffWide = kOffRows + kRowsAhead * kTileWarps * 8;   // [4] of 32 tokens: lo in e5m2
  static constexpr int kOffSmall = kOffWide + (kSide ? 0 : 16);   // [softmax warps] count_small
  static constexpr int kOffForm = kOffSmall + (kSide ? 0 : 16 * kSoftmaxWarps);   // [kRows / kJ] lo in e5m2 where a reference moves
  static constexpr int kOffWant = kOffForm + (kSide ? 0 : 4 * (kRows / kJ));   // [2] by unit parity, the tile from which lo is e5m2
  static constexpr int kOffBar = kOffWant + (kSide ? 0 : 8);
  static_assert(kOffSmall % 16 == 0, "read as uint4");
  static_assert(kOffP % 1024 == 0 && kOffK % 1024 == 0 && kOffKPe % 1024 == 0, "swizzle atoms");
};

template <int kRows>
constexpr int smem_bytes() {
  return Shape<kRows>::kOffBar + 8 * Shape<kRows>::kNumBars + 8;   // tensor memory's address, abort flag
}
static_assert(smem_bytes<16>() <= 232448 && smem_bytes<32>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory budget");

// A and B of kind::f8f6f4: format 0 e4m3, 1 e5m2; D f32.
constexpr uint32_t idesc_f8(int N, int b_format, bool mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_format) << 10) | (static_cast<uint32_t>(mn) << 15) |
         (static_cast<uint32_t>(mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_f8_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A warp's 32 lanes x N consecutive columns of tensor memory.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t& r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, uint32_t r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r) : "memory");
}

// A warpgroup's registers a thread, from those at launch.  Each direction has its
// own instruction; one that goes the other way is an illegal instruction.
template <int kFrom, int kTo>
__device__ __forceinline__ void set_registers() {
  static_assert(kTo % 8 == 0 && kTo >= 24 && kTo <= 256, "register count");
  if constexpr (kTo > kFrom) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTo));
  else if constexpr (kTo < kFrom) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTo));
}

// A barrier of `threads` threads that also tells whether any of them says so.
__device__ __forceinline__ bool bar_any(int id, int threads, bool yes) {
  uint32_t any;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %3, 0;\nbar.red.or.pred q, %1, %2, p;\nselp.u32 %0, 1, 0, q;\n}"
      : "=r"(any)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(yes))
      : "memory");
  return any != 0;
}

// Two numbers in fp16 -> two 8-bit codes (the first in the low byte; nearest
// even, saturating) and back.
template <__nv_fp8_interpretation_t kType>
__device__ __forceinline__ uint32_t to_fp8x2(__half2 x) {
  return __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&x), __NV_SATFINITE, kType);
}
template <__nv_fp8_interpretation_t kType>
__device__ __forceinline__ __half2 from_fp8x2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), kType);
  return *reinterpret_cast<const __half2*>(&h);
}
// Two floats -> hi and lo in e4m3, x = hi + lo / kLoScale (x - hi is exact).
constexpr float kLoScale = 32.f;
__device__ __forceinline__ void split_query(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
  const float2 h = __half22float2(from_fp8x2<__NV_E4M3>(hi));
  lo = __nv_cvt_float2_to_fp8x2(make_float2((x0 - h.x) * kLoScale, (x1 - h.y) * kLoScale), __NV_SATFINITE, __NV_E4M3);
}

// Four codes to four e4m3 numbers: the magnitudes' indices select bytes of the
// table, the signs (in place already) go on top.
__device__ __forceinline__ uint32_t expand4(uint2 table, uint32_t select, uint32_t signs) {
  uint32_t d;   // of select's low 16 bits; __byte_perm would mask them once more
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(table.x), "r"(table.y), "r"(select));
  return d | (signs & 0x80808080u);
}
__device__ __forceinline__ uint4 expand16(uint2 table, uint32_t w0, uint32_t w1) {
  const uint32_t a = w0 & 0x77777777u, b = w1 & 0x77777777u;
  return make_uint4(expand4(table, a, w0), expand4(table, a >> 16, w0 << 4), expand4(table, b, w1), expand4(table, b >> 16, w1 << 4));
}
// e4m3 codes of magnitude * 2^(6 - shift): up to a shift of 11 all are normal
// numbers, whose exponent field starts at bit 3.
__device__ __forceinline__ uint2 normal_table(uint32_t shift) {
  return make_uint2(0x6c686000u - shift * 0x08080800u, 0x7c787470u - shift * 0x08080808u);
}

// max or sum over a warp's lanes of each of N values, each step handing half of
// them on: lane l ends with value l >> (5 - log2 N).
template <bool kMax, int N>
__device__ __forceinline__ float warp_reduce(const float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  float x[N];
#pragma unroll
  for (int j = 0; j < N; ++j) x[j] = v[j];
  int d = 16;
#pragma unroll
  for (int half = N / 2; half > 0; half >>= 1, d >>= 1) {
    const bool upper = lane & d;
#pragma unroll
    for (int j = 0; j < half; ++j) {
      const float keep = upper ? x[half + j] : x[j], got = __shfl_xor_sync(~0u, upper ? x[j] : x[half + j], d);
      x[j] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
#pragma unroll
  for (; d > 0; d >>= 1) {
    const float got = __shfl_xor_sync(~0u, x[0], d);
    x[0] = kMax ? fmaxf(x[0], got) : x[0] + got;
  }
  return x[0];
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nadd.rn.f32x2 d, a, b;\nmov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmul.rn.f32x2 d, a, b;\nmov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n.reg .b64 a, b, c, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\nfma.rn.f32x2 d, a, b, c;\n"
      "mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// How many of a warp's tokens have a weight p = 2^z below 1/2 (those that a row does
// not see among them): of 16 rows, a byte each, row j in byte j % 4 of word j / 4.
__device__ __forceinline__ uint4 count_small(const float (&z)[16]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // the signs of four rows' z + 1, summed over the lanes
    auto bits = [&](int i) { return __float_as_uint(z[4 * j + i] + 1.f); };
    const uint32_t signs = __byte_perm(__byte_perm(bits(0), bits(1), 0x0073), __byte_perm(bits(2), bits(3), 0x0073), 0x5410);
    w[j] = __reduce_add_sync(~0u, (signs >> 7) & 0x01010101u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// A bit for each row with no more than `most` (up to 127) of its 128 tokens' weights at
// 1/2 or above, from the sums of its four warps' counts.
__device__ __forceinline__ uint32_t few_large(const uint4& small, uint32_t most) {
  auto four = [&](uint32_t w) {
    const uint32_t enough = ((w + most * 0x01010101u) >> 7) & 0x01010101u;   // 128 - most at least
    return (enough | enough >> 7 | enough >> 14 | enough >> 21) & 15u;
  };
  return four(small.x) | four(small.y) << 4 | four(small.z) << 8 | four(small.w) << 12;
}

// Where the walk over a worker's tiles stands.
struct Cursor {
  int ui, tile, tiles;      // unit, tile of the unit
  int tok_begin, tok_end, page_base;
  __device__ __forceinline__ void set(const WorkUnit& u) {
    tok_begin = u.tok_begin;
    tok_end = u.tok_end;
    page_base = u.page_base;
    tile = 0;
    tiles = (tok_end - tok_begin + kT - 1) / kT;
  }
  __device__ __forceinline__ int tok0() const { return tok_begin + tile * kT; }
  // To the next tile; false past the last one.
  __device__ __forceinline__ bool next(const WorkUnit* units, int end) {
    if (++tile < tiles) return true;
    if (++ui >= end) return false;
    set(units[ui]);
    return true;
  }
};

template <int kRows, bool kOutF32>
__global__ void __launch_bounds__(Shape<kRows>::kThreads, 1) decode_q4_kernel(const DecodeArgs a) {
  using S = Shape<kRows>;
  constexpr int kJ = S::kJ, kSoftmaxWarps = S::kSoftmaxWarps, kTileWarps = S::kTileWarps, kIssueWarp = S::kIssueWarp, kTokWarp = S::kTokWarp;
  constexpr int kBufs = S::kBufs;
  extern __shared__ __align__(1024) unsigned char sm[];
  const uint32_t base = smem_u32(sm);
  auto bar = [&](int i) { return base + S::kOffBar + 8 * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + S::kOffBar + 8 * S::kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  // The plan's arrays were uploaded before the kernel ahead on the stream began, so
  // they may be read while that one ends; everything else is read after the wait.
  const int H = a.num_heads;
  const int groups = (H + 63) / 64;                 // CTAs to a worker (1 below kRows = 64)
  const int worker = blockIdx.x / groups, row0 = 64 * (blockIdx.x % groups);
  int u0 = a.worker_ptr[worker], u1 = a.worker_ptr[worker + 1];   // of a.n_workers + 1 entries
  const PlanDev prm = *a.params;
  // A replay may meet another plan than its call did: one of other rows to a request is
  // refused, and of a larger batch the requests behind the call's are neither read nor written.
  if (worker >= prm.n_workers || prm.num_heads != H) u0 = u1 = 0;
  WorkUnit unit0{};
  if (u0 < u1) unit0 = a.units[u0];
  const int page_shift = 31 - __clz(prm.page_size);

  if (threadIdx.x < S::kNumBars) {
    if (threadIdx.x == 0) *abort_flag = 0;
    if (threadIdx.x == 0 && blockIdx.x == 0 && prm.num_heads != H) report_error(a.err, kErrBounds);
    const int i = threadIdx.x;
    mbar_init(bar(i), i < S::kSFull0 || (i >= S::kRowsFree0 && i < S::kQReady) ? kTileWarps
                        : (i >= S::kSFree0 && i < S::kPReady0) || i == S::kQReady ? kSoftmaxWarps
                        : i >= S::kPReady0 && i < S::kPvDone0                     ? kSoftmaxWarps / 4
                                                                                  : 1);
    fence_barrier_init();
  }
  if (threadIdx.x < 4) {
    // e4m3 codes of magnitude * 2^(6 - shift), subnormal numbers among them (a shift
    // of 15, which no row has, as 14)
    uint32_t t[2] = {0, 0};
    const int shift = min(12 + static_cast<int>(threadIdx.x), kQ4MaxShift);
    for (int m = 1; m < 8; ++m) {
      // magnitude m = (2 + m % 2) 2^(m / 2) / 4 from index 2 on, m / 2 below
      const float v = (m < 2 ? 0.5f * m : (2 + (m & 1)) * pow2((m >> 1) - 2)) * pow2(6 - shift);
      t[m >> 2] |= static_cast<uint32_t>(__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3)) << (8 * (m & 3));
    }
    reinterpret_cast<uint2*>(sm + S::kOffTable)[threadIdx.x] = make_uint2(t[0], t[1]);
  }
  if (threadIdx.x < kRows) reinterpret_cast<float*>(sm + S::kOffRef)[threadIdx.x] = 0.f;
  if (!S::kSide && threadIdx.x < 2) reinterpret_cast<int*>(sm + S::kOffWant)[threadIdx.x] = INT_MAX;
  if (!S::kSide && threadIdx.x < 4) reinterpret_cast<uint32_t*>(sm + S::kOffWide)[threadIdx.x] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == kIssueWarp) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  bool ok = true;
  auto wait = [&](int i, int phase) { ok &= mbar_spin<false>(bar(i), phase & 1, abort_flag); };

  if (warp >= kIssueWarp) {
    set_registers<S::kRegs, S::kRegsIssue>();
    if (warp == kIssueWarp + 2 && u0 < u1) {
      // ================= the warp that finds the rows =================
      // Lane e: where expanding warp e has its rows of each tile, S::kRowsAhead tiles ahead,
      // and the request for them into L2 (without it 4 requests of 131072 tokens take 64
      // us for 60).  Behind the last tile, one without rows for each group.
      const uint8_t* cache = static_cast<const uint8_t*>(a.ckv);
      Cursor at;
      at.ui = u0;
      at.set(unit0);
      bool more = true;
      int behind = 0;
      for (int g = 0;; ++g) {
        const int t = at.tok0() + kTokWarp * lane;
        uint64_t r = 0;
        if (more && lane < kTileWarps && t < at.tok_end) {
          const int page = a.kv_indices[at.page_base + (t >> page_shift)];
          if (page < 0 || page >= a.num_pages) {   // its rows count as zeros
            report_error(a.err, kErrBounds);
          } else {
            const int n = min(kTokWarp, at.tok_end - t);
            const uint8_t* src = cache + ((static_cast<size_t>(page) << page_shift) + (t & ((1 << page_shift) - 1))) * kQ4Row;
            r = pack_rows(src, n);
            bulk_prefetch_l2(src, n * kQ4Row);
          }
        }
        if (g >= S::kRowsAhead) wait(S::kRowsFree0 + g % S::kRowsAhead, (g - S::kRowsAhead) / S::kRowsAhead);
        if (lane < kTileWarps) reinterpret_cast<uint64_t*>(sm + S::kOffRows)[g % S::kRowsAhead * kTileWarps + lane] = r;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::kRowsFull0 + g % S::kRowsAhead));
        if (more) {
          const int ui = at.ui;
          more = at.next(a.units, u1);
          // Another unit's: its query will be wanted too.  Of 64 rows (72 KB; 0.5 to 1 % of
          // batches of several units a worker), fewer come as fast by themselves, and their
          // tiles are found too quickly for a warp with more to do (2 us of 48).
          if (kRows == 64 && more && at.ui != ui) {
            const int req = a.units[at.ui].req;
            const size_t row = static_cast<size_t>(req) * H + row0;
            const int n = req < a.batch ? min(kRows, H - row0) : 0;
            for (int i = lane; i < n; i += 32) bulk_prefetch_l2(static_cast<const __nv_bfloat16*>(a.q_nope) + (row + i) * kDCkv, 2 * kDCkv);
            if (lane == 0 && n > 0) bulk_prefetch_l2(static_cast<const __nv_bfloat16*>(a.q_pe) + row * kDKpe, 2 * kDKpe * n);
          }
        } else if (++behind == S::kGroups) {
          break;
        }
      }
      if (!ok && lane == 0) report_error(a.err, kErrTimeout);
    } else if (warp <= kIssueWarp + 1) {
      // ================= the issuing warps =================
      const uint64_t k_desc = smem_desc(base + S::kOffK, 16, 1024, kSw128);
      const uint64_t kpe_desc = smem_desc(base + S::kOffKPe, 16, 512, kSw64);
      const uint64_t q_desc = smem_desc(base + S::kOffQ, 16, 1024, kSw128);
      const uint64_t qpe_desc = smem_desc(base + S::kOffQPe, 16, 512, kSw64);
      const uint64_t p_desc = smem_desc(base + S::kOffP, 16, 8 * S::kPRow, S::kPSwizzle);
      constexpr uint32_t id_s = idesc_f8(S::kNS, 0, false), id_hi = idesc_f8(S::kPN, 1, true);
      auto scores = [&](int g) {
        if (g > 1) wait(S::kSFree0 + (g & 1), (g - 2) >> 1);
        const uint32_t d = tmem + S::kColS + (g & 1) * S::kNS;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          if (p % (4 / S::kStages) == 0) {
            wait(S::kKFull0 + g % kBufs * S::kStages + p / (4 / S::kStages), g / kBufs);
            tc_fence_after();
          }
          const uint64_t ka = k_desc + static_cast<uint64_t>(((g % kBufs * 4 + p) * S::kPanel) >> 4);
          const uint64_t qb = q_desc + static_cast<uint64_t>((p * S::kQPanel) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_f8_elect(d, ka + 2 * kk, qb + 2 * kk, id_s, (p | kk) != 0);
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
          mma_f8_elect(d, kpe_desc + static_cast<uint64_t>(((S::kPeBufs == 2 ? (g & 1) * kT * 64 : 0) >> 4) + 2 * kk), qpe_desc + 2 * kk, id_s, 1);
        mma_commit_elect(bar(S::kSFull0 + (g & 1)));
      };
      auto values = [&](int g, bool first) {
        // 32 tokens at a time, rolled up: with less code for 28 warps to fetch 4 requests of
        // 131072 tokens and 16 heads take 59.8 us for 61.2 (the scores rolled up too: no more)
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          wait(S::kPReady0 + j, g);
          tc_fence_after();
          uint32_t id_lo = idesc_f8(S::kPN, 0, true);
          if constexpr (!S::kSide)   // e4m3 or e5m2; through a shuffle, for the MMAs' operands are to be known uniform
            id_lo |= (__shfl_sync(~0u, reinterpret_cast<volatile const uint32_t*>(sm + S::kOffWide)[j], 0) & 1) << 10;
          const uint64_t pb = p_desc + static_cast<uint64_t>((j * 32 * S::kPRow) >> 4);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const uint64_t va = k_desc + static_cast<uint64_t>(((g % kBufs * 4 + p) * S::kPanel + j * 32 * 128) >> 4);
            if constexpr (S::kSide) {
              mma_f8_elect(tmem + p * S::kOBlock, va, pb, id_hi, !first || j > 0);
            } else {
              mma_f8_elect(tmem + p * S::kOBlock, va, pb, id_hi, !first || j > 0);
              mma_f8_elect(tmem + p * S::kOBlock, va, pb + static_cast<uint64_t>(S::kPPanel >> 4), id_lo, 1);
            }
          }
          mma_commit_elect(bar(S::kPvDone0 + 4 * (g % kBufs) + j));
        }
      };
      // The scores of a tile need its rows, P . V of the tile before its P: whichever
      // comes first goes first, so each has a warp of its own (with one warp for both,
      // in a fixed order, the scores of a tile wait for P of the one before).
      const int role = warp - kIssueWarp;
      int g = 0;
      for (int ui = u0; ui < u1; ++ui) {
        const int n = (a.units[ui].tok_end - a.units[ui].tok_begin + kT - 1) / kT;
        if (role == 0) wait(S::kQReady, ui - u0);
        for (int i = 0; i < n; ++i, ++g) {
          if (role == 0) scores(g);
          else values(g, i == 0);
        }
      }
      mma_commit_elect(bar(S::kFinal0 + role));
      if (!ok && lane == 0) report_error(a.err, kErrTimeout);
      mbar_wait_drain(bar(S::kFinal0 + role), 0);   // every MMA issued is done before tensor memory is freed
      __syncwarp();
    }
  } else if (warp >= kSoftmaxWarps) {
    // ================= expanding warps =================
    set_registers<S::kRegs, S::kRegsExpand>();
    if (u0 < u1) {
      const int group = (warp - kSoftmaxWarps) / kTileWarps, ew = (warp - kSoftmaxWarps) % kTileWarps;
      int tiles = 0;
      for (int ui = u0; ui < u1; ++ui) tiles += (a.units[ui].tok_end - a.units[ui].tok_begin + kT - 1) / kT;
      const uint2* table = reinterpret_cast<const uint2*>(sm + S::kOffTable);
      auto rows_of = [&](int g) {
        wait(S::kRowsFull0 + g % S::kRowsAhead, g / S::kRowsAhead);
        Rows r(reinterpret_cast<const uint64_t*>(sm + S::kOffRows)[g % S::kRowsAhead * kTileWarps + ew]);
        if (!ok) r.n = 0;   // given up: nothing need be there
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::kRowsFree0 + g % S::kRowsAhead));
        return r;
      };
      // A lane takes whole groups (16 bytes of codes).  Of ckv, at a time, a warp takes kRun
      // rows of kSpan panels: eight lanes the four groups of two rows, which they write to
      // eight groups of banks.  Of kpe, group lane % 2 of row lane / 2.  Shifts of ckv: four of
      // row 8 i + lane / 4 a lane.
      constexpr int kSpan = 4 / S::kStages, kRun = 8 / kSpan, kRuns = kTokWarp / kRun;
      const int pair = lane & 3, panel = (lane >> 3) % kSpan, sub = ((lane >> 2) & 1) + 2 * ((lane >> 3) / kSpan);
      // Of kpe with eight rows a warp: half a group a lane, a quarter of row lane / 4.
      uint4 raw[kTokWarp / 2], raw_pe;
      uint32_t shifts[kTokWarp / 8], meta_pe;
      constexpr int kPeShift = kTokWarp == 16 ? 1 : 2;   // lanes of a row's kpe
      auto load_ckv = [&](const Rows& r, int i) {   // run i % kRuns of stage i / kRuns
        return __ldg(reinterpret_cast<const uint4*>(r.src + (kRun * (i % kRuns) + sub) * kQ4Row) + 4 * (kSpan * (i / kRuns) + panel) + pair);
      };
      auto load_meta = [&](const Rows& r) {
#pragma unroll
        for (int i = 0; i < kTokWarp / 8; ++i) {
          shifts[i] = 0;
          if (8 * i + (lane >> 2) < r.n) shifts[i] = __ldg(reinterpret_cast<const uint16_t*>(r.src + (8 * i + (lane >> 2)) * kQ4Row + kQ4Meta) + pair);
        }
        meta_pe = 127 << 8;
        if ((lane >> kPeShift) < r.n) meta_pe = __ldg(reinterpret_cast<const uint16_t*>(r.src + (lane >> kPeShift) * kQ4Row + kQ4Meta + 8));
      };
      auto load_pe = [&](const Rows& r) {
        raw_pe = make_uint4(0, 0, 0, 0);
        if ((lane >> kPeShift) < r.n) {
          const uint8_t* codes = r.src + (lane >> kPeShift) * kQ4Row + kDCkv / 2;
          if constexpr (kTokWarp == 16) {
            raw_pe = __ldg(reinterpret_cast<const uint4*>(codes) + (lane & 1));
          } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(codes) + (lane & 3));
            raw_pe.x = v.x, raw_pe.y = v.y;
          }
        }
      };
      auto load_part = [&](const Rows& r) {   // not all of a warp's rows: the others hold zeros
#pragma unroll
        for (int i = 0; i < kTokWarp / 2; ++i) {
          raw[i] = make_uint4(0, 0, 0, 0);
          if (kRun * (i % kRuns) + sub < r.n) raw[i] = load_ckv(r, i);
        }
      };
      // Tile g from registers, which take the rows `next` meanwhile.
      auto expand = [&](int g, const Rows& next) {
        uint32_t shift[kTokWarp / 8];
#pragma unroll
        for (int i = 0; i < kTokWarp / 8; ++i) shift[i] = shifts[i];
        const uint32_t meta = meta_pe;
        load_meta(next);
        // shifts past 11 lead to subnormal numbers, by a table
        uint32_t large = (meta & (meta << 1)) & 0x88u;
#pragma unroll
        for (int i = 0; i < kTokWarp / 8; ++i) large |= shift[i] & (shift[i] << 1) & 0x8888u;
        const bool whole = next.n == kTokWarp;
        // the tables of this lane's groups, made before the buffer is free
        uint2 tables[kTokWarp / 2], table_pe;
        auto make = [&](auto table_of) {
#pragma unroll
          for (int i = 0; i < kTokWarp / 2; ++i) {
            const int row = kRun * (i % kRuns);
            const uint32_t mine = __shfl_sync(~0u, shift[row / 8], 4 * (row % 8 + sub) + kSpan * (i / kRuns) + panel);
            tables[i] = table_of((mine >> (4 * pair)) & 15);
          }
          table_pe = table_of((meta >> (kTokWarp == 16 ? 4 * (lane & 1) : 2 * (lane & 2))) & 15);
        };
        if (__any_sync(~0u, large)) make([&](uint32_t k) { return k >= 12 ? table[k - 12] : normal_table(k); });
        else make([](uint32_t k) { return normal_table(k); });
        // the buffer was read by P . V of g - kBufs
        if (g >= kBufs) wait(S::kPvDone0 + 4 * (g % kBufs) + ew * kTokWarp / 32, g / kBufs - 1);
        {
          unsigned char* dst = sm + S::kOffK + g % kBufs * 4 * S::kPanel + panel * S::kPanel + (kTokWarp * ew + sub) * 128;
#pragma unroll
          for (int stage = 0; stage < S::kStages; ++stage) {
#pragma unroll
            for (int j = 0; j < kRuns; ++j) {
              const int i = stage * kRuns + j;
              const uint2 t = tables[i];
              // chunk 2 pair of a row is at 2 pair ^ row % 8
              unsigned char* at = dst + kSpan * stage * S::kPanel + kRun * j * 128;
              const int chunk = (2 * pair) ^ sub ^ (kRun * j % 8);
              *reinterpret_cast<uint4*>(at + (chunk << 4)) = expand16(t, raw[i].x, raw[i].y);
              *reinterpret_cast<uint4*>(at + ((chunk ^ 1) << 4)) = expand16(t, raw[i].z, raw[i].w);
              if (whole) raw[i] = load_ckv(next, i);
            }
            if (stage + 1 < S::kStages) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(S::kKFull0 + g % kBufs * S::kStages + stage));
            }
          }
          if (S::kPeBufs == 1 && g > 0) wait(S::kSFull0 + ((g - 1) & 1), (g - 1) >> 1);   // the scores before have read it
          const int row = kTokWarp * ew + (lane >> kPeShift);
          unsigned char* pe = sm + S::kOffKPe + (S::kPeBufs == 2 ? (g & 1) * kT * 64 : 0) + row * 64;
          const uint2 t = table_pe;
          if constexpr (kTokWarp == 16) {
            const int at = ((2 * (lane & 1)) ^ ((row >> 1) & 3)) << 4;
            *reinterpret_cast<uint4*>(pe + at) = expand16(t, raw_pe.x, raw_pe.y);
            *reinterpret_cast<uint4*>(pe + (at ^ 16)) = expand16(t, raw_pe.z, raw_pe.w);
          } else {
            *reinterpret_cast<uint4*>(pe + (((lane & 3) ^ ((row >> 1) & 3)) << 4)) = expand16(t, raw_pe.x, raw_pe.y);
          }
          if ((lane & ((1 << kPeShift) - 1)) == 0) sm[S::exp_at(g % kBufs, row)] = static_cast<unsigned char>(meta >> 8);
        }
        fence_proxy_async_smem();
        __syncwarp();
#ifdef MLA_STALL_TEST
        if (blockIdx.x == 0 && ew == 0 && g + 1 == g_q4_stall) return;
#endif
        if (lane == 0) mbar_arrive(bar(S::kKFull0 + g % kBufs * S::kStages + S::kStages - 1));
        load_pe(next);
        if (!whole) load_part(next);
      };
      {
        const Rows rows = rows_of(group);
        load_part(rows);
        load_meta(rows);
        load_pe(rows);
      }
      for (int g = group; g < tiles; g += S::kGroups) {
        expand(g, rows_of(g + S::kGroups));
      }
      if (!ok && lane == 0) report_error(a.err, kErrTimeout);
    }
  } else {
    // ================= softmax and epilogue =================
    set_registers<S::kRegs, S::kRegsSoftmax>();
    const int q = warp & 3, cg = warp >> 2;             // tokens 32 q .. of a tile (lane quadrant), query rows kJ cg ..
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const int tok = 32 * q + lane;
    float* refs = reinterpret_cast<float*>(sm + S::kOffRef) + kJ * cg;
    float* red = reinterpret_cast<float*>(sm + S::kOffRed) + 4 * cg * kJ;   // of the four warps of these query rows
    // ---- the query of a unit, a few rows a warp, two at a time ----
    auto put_query = [&](int req, int parity) {
      constexpr int kOwn = kRows / kSoftmaxWarps;
      const int rows = req < a.batch ? H : 0;
      float* out = reinterpret_cast<float*>(sm + S::kOffScale) + parity * kRows;
#pragma unroll 1
      for (int k = 0; k < kOwn; k += 2) {
        uint32_t w[2][9];   // dims 16 lane .. + 15 of q_nope, 2 lane and + 1 of q_pe
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = row0 + warp * kOwn + k + i;
#pragma unroll
          for (int j = 0; j < 9; ++j) w[i][j] = 0;
          if (r < rows) {
            const size_t row = static_cast<size_t>(req) * H + r;
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q_nope) + row * kDCkv + 16 * lane);
            const uint4 v0 = src[0], v1 = src[1];
            w[i][0] = v0.x, w[i][1] = v0.y, w[i][2] = v0.z, w[i][3] = v0.w;
            w[i][4] = v1.x, w[i][5] = v1.y, w[i][6] = v1.z, w[i][7] = v1.w;
            w[i][8] = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q_pe) + row * kDKpe)[lane];
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = warp * kOwn + k + i;
          uint32_t m = 0;
#pragma unroll
          for (int j = 0; j < 9; ++j) m = __vmaxu2(m, w[i][j] & 0x7fff7fffu);
          const uint32_t top = __reduce_max_sync(~0u, max(m >> 16, m & 0xffffu));   // bits of the largest magnitude
          // in -120 .. 126, where fp32 has 2^e and 2^-e, both normal: a row whose largest is below
          // 2^-119 is left under [2^7, 2^8)
          const int e = top == 0 ? 0 : min(7 - (static_cast<int>(top >> 7) - 127), 126);
          const float up = pow2(e);
          uint32_t hi[9], lo[9];
#pragma unroll
          for (int j = 0; j < 9; ++j)
            split_query(__uint_as_float(w[i][j] << 16) * up, __uint_as_float(w[i][j] & 0xffff0000u) * up, hi[j], lo[j]);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint32_t* c = t ? lo : hi;
            const int row = t * kRows + r;
            *reinterpret_cast<uint4*>(sm + S::kOffQ + (lane >> 3) * S::kQPanel + row * 128 + (((lane & 7) ^ (row & 7)) << 4)) =
                make_uint4(c[0] | c[1] << 16, c[2] | c[3] << 16, c[4] | c[5] << 16, c[6] | c[7] << 16);
            *reinterpret_cast<uint16_t*>(sm + S::kOffQPe + row * 64 + (((lane >> 3) ^ ((row >> 1) & 3)) << 4) + 2 * (lane & 7)) =
                static_cast<uint16_t>(c[8]);
          }
          // an infinite or NaN query has NaN scores
          if (lane == 0) out[r] = top >= 0x7f80u ? __int_as_float(0x7fffffff) : pow2(-e);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(S::kQReady));
    };
    if (u0 < u1) put_query(unit0.req, 0);
    int g = 0;
    for (int ui = u0; ui < u1; ++ui) {
      const WorkUnit u = a.units[ui];
      const float* scale = reinterpret_cast<const float*>(sm + S::kOffScale) + ((ui - u0) & 1) * kRows + kJ * cg;
      float lx[kJ], ld[kJ];
#pragma unroll
      for (int j = 0; j < kJ; ++j) lx[j] = ld[j] = 0.f;
      bool wide = false;   // 64 rows: lo is e5m2 from here to the unit's end
      int* want = reinterpret_cast<int*>(sm + S::kOffWant) + ((ui - u0) & 1);
      for (int t0 = u.tok_begin; t0 < u.tok_end; t0 += kT, ++g) {
        const bool first = t0 == u.tok_begin;
        // ---- scores of this thread's token and query rows, less the reference, in log2 ----
        wait(S::kSFull0 + (g & 1), g >> 1);
        tc_fence_after();
        float z[kJ];
        const int exponent = sm[S::exp_at(g % kBufs, tok)];
        const int e = exponent == kQ4NanExp ? 0 : exponent - 127;
        {
          uint32_t hi[kJ], lo[kJ];
          const uint32_t col = S::kColS + (g & 1) * S::kNS + kJ * cg;
          tmem_ld(lane_addr + col, hi);
          tmem_ld(lane_addr + col + kRows, lo);
          const float unit = exponent == kQ4NanExp ? __int_as_float(0x7fffffff) : pow2(e - 6) * (prm.sm_scale * kLog2e);
          const float fe = static_cast<float>(e);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(S::kSFree0 + (g & 1)));
#pragma unroll
          for (int j = 0; j < kJ; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(scale + j);
            const float4 ref = *reinterpret_cast<const float4*>(refs + j);
            auto two = [&](int i, float2 f2, float2 ref2) {
              const float2 s = fma2(make_float2(__uint_as_float(lo[i]), __uint_as_float(lo[i + 1])), make_float2(1 / kLoScale, 1 / kLoScale),
                                    make_float2(__uint_as_float(hi[i]), __uint_as_float(hi[i + 1])));
              // (the units first: their product is exact, and in range where the score is)
              const float2 y = fma2(s, mul2(make_float2(unit, unit), f2), add2(make_float2(fe, fe), ref2));
              z[i] = y.x;
              z[i + 1] = y.y;
            };
            two(j, make_float2(f.x, f.y), make_float2(ref.x, ref.y));
            two(j + 2, make_float2(f.z, f.w), make_float2(ref.z, ref.w));
          }
        }
        if (t0 + kT > u.tok_end - (prm.q_len > 1 ? prm.q_len - 1 : 0)) {
          // the query rows that see token t: of query tokens packed into rows, row h sees
          // the tokens before kv_len - (q_len - 1 - h / heads)
          const int t = t0 + tok;
          int from = t < u.tok_end ? 0 : 128;
          if (prm.q_len > 1 && t < u.tok_end) from = min(128, prm.heads_per_token * max(0, prm.q_len - u.kv_len + t));
          from -= row0 + kJ * cg;
#pragma unroll
          for (int j = 0; j < kJ; ++j) z[j] = j >= from ? z[j] : -INFINITY;
        }
        float top = z[0];
#pragma unroll
        for (int j = 1; j < kJ; ++j) top = fmaxf(top, z[j]);
        // ---- the reference moves: the four warps of these query rows together ----
        uint32_t moved = 0;   // rows whose reference moves
        float factor = 1.f;   // lane j: of row j
        const float limit = first ? -INFINITY : wide ? S::kTopWide : S::kTop;
        const bool moves = bar_any(1 + cg, 128, first || top > limit);
        // Another row's wish of two tiles ago: written before P of that tile was signalled, which
        // P . V waited for, and for that the warps here, before P of the last one.  A later
        // wish is for a later tile, seen here or not, so that all warps go over at once.
        if (!S::kSide && !first) wide |= g >= *reinterpret_cast<volatile int*>(want);
        if (moves) {
          const float most = warp_reduce<true>(z);
          if ((lane & (32 / kJ - 1)) == 0) red[q * kJ + lane * kJ / 32] = most;
          uint32_t* form = reinterpret_cast<uint32_t*>(sm + S::kOffForm) + cg;
          if (!S::kSide && q == 0 && lane == 0) *form = wide;
          named_bar_sync(1 + cg, 128);
          // The first warp's word on it, so that after a wait that ran out, too, the four meet at
          // the barriers below equally often.
          if (!S::kSide) wide = *form != 0;
          // lane j (and those kJ apart): row j.  The largest p becomes 2^(kTop - kSlack); a row that
          // sees no token in its unit's first tile sees none later, and keeps the reference 0
          // with p = 0
          const int r = lane % kJ;
          const float m = fmaxf(fmaxf(red[r], red[kJ + r]), fmaxf(red[2 * kJ + r], red[3 * kJ + r]));
          const float usual = wide ? S::kTopWide - S::kSlackWide : S::kTop - S::kSlack;
          float up = m > limit ? m - usual : 0.f;
          constexpr uint32_t kAll = (1u << kJ) - 1;
          const uint32_t rows = __ballot_sync(~0u, m > limit) & kAll;   // whose reference moves
#pragma unroll
          for (int j = 0; j < kJ; ++j)
            if (rows >> j & 1) z[j] -= __shfl_sync(~0u, up, j);
          if (!S::kSide && !wide) {
            uint4* small = reinterpret_cast<uint4*>(sm + S::kOffSmall) + 4 * cg;
            if constexpr (kJ == 16) {
              const uint4 mine = count_small(z);
              if (lane == 0) small[q] = mine;
            }
            named_bar_sync(1 + cg, 128);
            const uint4 s0 = small[0], s1 = small[1], s2 = small[2], s3 = small[3];   // bytes: up to 128 in all
            const uint32_t few = few_large(make_uint4(s0.x + s1.x + s2.x + s3.x, s0.y + s1.y + s2.y + s3.y, s0.z + s1.z + s2.z + s3.z,
                                                      s0.w + s1.w + s2.w + s3.w), S::kFewLarge);
            // (not a row that sees no token); in a unit's first tile all rows' warps are here
            bool any = (few & ~__ballot_sync(~0u, m == -INFINITY) & kAll) != 0;
            if (first) any = bar_any(5, 32 * kSoftmaxWarps, any);
            float further = 0.f;   // how much higher the largest p becomes
            if (first) {
              wide = any;
              if (any) further = (S::kTopWide - S::kSlackWide) - (S::kTop - S::kSlack);
              if (warp == 0 && lane == 0) reinterpret_cast<int*>(sm + S::kOffWant)[(ui - u0 + 1) & 1] = INT_MAX;   // the next unit's
            } else if (any) {
              if (lane == 0) atomicMin(want, g + 2);
              further = S::kSlack - S::kSlackFew;
            }
            if (further != 0.f) {
              if (m > limit) up -= further;
#pragma unroll
              for (int j = 0; j < kJ; ++j)
                if (rows >> j & 1) z[j] += further;
            }
          }
          if (!first) {
            moved = rows;
            factor = fast_exp2(-up);
#pragma unroll
            for (int j = 0; j < kJ; ++j)
              if (rows >> j & 1) {
                const float alpha = __shfl_sync(~0u, factor, j);
                lx[j] *= alpha;
                ld[j] *= alpha;
              }
          }
          if (q == 0 && lane < kJ) refs[lane] -= up;
        }
        // ---- p and its terms ----
        constexpr int kTerms = S::kSide ? 3 : 2;
        uint32_t c[kTerms][kJ / 4];
        const float2 weight = make_float2(pow2(-e), pow2(-e));
        auto make_terms = [&](auto lo_in_e5m2) {
          constexpr bool kWide = decltype(lo_in_e5m2)::value;
          const __half2 full = __float2half2_rn(kWide ? 1 / S::kFullWide : 1 / S::kFull);
#pragma unroll
          for (int j = 0; j < kJ; j += 2) {
            const float2 p = make_float2(fast_exp2(z[j]), fast_exp2(z[j + 1]));
            const float2 x = fma2(p, weight, make_float2(lx[j], lx[j + 1]));
            lx[j] = x.x;
            lx[j + 1] = x.y;
            const __half2 h = __floats2half2_rn(p.x, p.y);
            uint32_t code[kTerms];
            code[0] = to_fp8x2<__NV_E5M2>(h);
            __half2 rest = __hsub2(h, from_fp8x2<__NV_E5M2>(code[0]));   // exact
            if constexpr (S::kSide) {
              code[1] = to_fp8x2<__NV_E5M2>(rest);
              rest = __hsub2(rest, from_fp8x2<__NV_E5M2>(code[1]));
              code[2] = to_fp8x2<__NV_E5M2>(rest);
              rest = __hsub2(rest, from_fp8x2<__NV_E5M2>(code[2]));
            } else if constexpr (kWide) {
              code[1] = to_fp8x2<__NV_E5M2>(rest);
              rest = __hsub2(rest, from_fp8x2<__NV_E5M2>(code[1]));
            } else {
              code[1] = to_fp8x2<__NV_E4M3>(rest);
              rest = __hsub2(rest, from_fp8x2<__NV_E4M3>(code[1]));
            }
            // what the terms leave of p, counted in full from kFull on and less below
            rest = __hmul2(rest, __hmul2_sat(h, full));
            const float2 y = fma2(__half22float2(rest), weight, make_float2(ld[j], ld[j + 1]));
            ld[j] = y.x;
            ld[j + 1] = y.y;
#pragma unroll
            for (int i = 0; i < kTerms; ++i) c[i][j / 4] = j % 4 ? c[i][j / 4] | code[i] << 16 : code[i];
          }
        };
        if (wide) make_terms(std::true_type{});
        else make_terms(std::false_type{});
        if (g > 0) wait(S::kPvDone0 + 4 * ((g - 1) % kBufs) + q, (g - 1) / kBufs);   // P . V of the tile before has read these rows of P
        if (moves) {
          if (moved) {   // their columns of O, a row at a time: few move at once
            wait(S::kPvDone0 + 4 * ((g - 1) % kBufs) + 3, (g - 1) / kBufs);
            tc_fence_after();
            do {
              const int j = __ffs(moved) - 1;
              moved &= moved - 1;
              constexpr int kCols = S::kSide ? 12 : 4;
              uint32_t o[kCols];
#pragma unroll
              for (int i = 0; i < kCols; ++i) tmem_ld(lane_addr + (i & 3) * S::kOBlock + (i >> 2) * kRows + kJ * cg + j, o[i]);
              const float alpha = __shfl_sync(~0u, factor, j);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < kCols; ++i)
                tmem_st(lane_addr + (i & 3) * S::kOBlock + (i >> 2) * kRows + kJ * cg + j, __float_as_uint(__uint_as_float(o[i]) * alpha));
            } while (moved);
            tmem_st_wait();
            tc_fence_before();
          }
          named_bar_sync(1 + cg, 128);   // P is signalled once O and the references are right for all
        }
        unsigned char* prow = sm + S::kOffP + tok * S::kPRow;
#pragma unroll
        for (int i = 0; i < kTerms; ++i) {
          if constexpr (kRows == 64)
            *reinterpret_cast<uint4*>(prow + i * S::kPPanel + ((cg ^ ((tok >> 1) & 3)) << 4)) = make_uint4(c[i][0], c[i][1], c[i][2], c[i][3]);
          else if constexpr (kRows == 32)
            *reinterpret_cast<uint4*>(prow + (((2 * i + cg) ^ (tok & 7)) << 4)) = make_uint4(c[i][0], c[i][1], c[i][2], c[i][3]);
          else
            *reinterpret_cast<uint2*>(prow + ((i ^ ((tok >> 1) & 3)) << 4) + 8 * cg) = make_uint2(c[i][0], c[i][1]);
        }
        if constexpr (!S::kSide)
          if (cg == 0 && lane == 0) reinterpret_cast<volatile uint32_t*>(sm + S::kOffWide)[q] = wide;
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::kPReady0 + q));
      }
      // ---- epilogue: the sums over the unit's tokens of all lanes and quadrants; the second
      // ones are exchanged where these query rows had their P, which no MMA reads any more ----
      const bool split = u.out_slot >= 0;
      const int rows = u.req < a.batch ? H : 0;   // that are written
#pragma unroll
      for (int j = 0; j < kJ; ++j) ld[j] = lx[j] - ld[j];   // of what P stands for
      const float sx = warp_reduce<false>(lx), sr = warp_reduce<false>(ld);
      // the next unit's query: every score of this one is made
      if (ui + 1 < u1) put_query(a.units[ui + 1].req, (ui + 1 - u0) & 1);
      wait(S::kPvDone0 + 4 * ((g - 1) % kBufs) + 3, (g - 1) / kBufs);
      tc_fence_after();
      auto shared_sum = [&](int from, int j) -> float* {   // of quadrant `from`, row j
        const int at = from * kJ + j;                       // 4 kJ floats, in the first terms of tokens 0 ..
        const int t = at / (kJ / 4), chunk = kRows == 64 ? cg ^ ((t >> 1) & 3) : kRows == 32 ? cg ^ (t & 7) : (t >> 1) & 3;
        return reinterpret_cast<float*>(sm + S::kOffP + t * S::kPRow + (chunk << 4) + (kRows == 16 ? 8 * cg : 0)) + at % (kJ / 4);
      };
      if ((lane & (32 / kJ - 1)) == 0) {
        red[q * kJ + lane * kJ / 32] = sx;
        *shared_sum(q, lane * kJ / 32) = sr;
      }
      named_bar_sync(1 + cg, 128);
      // lane j joins the sums of row j (little code: the first unit of a launch waits for it)
      float inverse = 0.f;
      if (lane < kJ) {
        const float s = (*shared_sum(0, lane) + *shared_sum(1, lane)) + (*shared_sum(2, lane) + *shared_sum(3, lane));
        inverse = s == 0.f ? 0.f : 0x1p-6f / s;   // a row that saw no token: out 0
        const int h = row0 + kJ * cg + lane;
        if (q == 0 && h < rows) {
          const float sum = (red[lane] + red[kJ + lane]) + (red[2 * kJ + lane] + red[3 * kJ + lane]);
          const float lse = (log2f(sum) - refs[lane]) * kLn2;
          if (split) a.lse_part[lse_part_offset(u.out_slot, 0, h, H)] = lse;
          else a.lse[static_cast<size_t>(u.req) * H + h] = lse;
        }
      }
      __syncwarp();
      float inv[kJ];
#pragma unroll
      for (int j = 0; j < kJ; ++j) inv[j] = __shfl_sync(~0u, inverse, j);
#pragma unroll 1
      for (int p = 0; p < 4; ++p) {
        uint32_t o[kJ];
        float x[kJ];
        tmem_ld(lane_addr + p * S::kOBlock + kJ * cg, o);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < kJ; ++j) x[j] = __uint_as_float(o[j]);
        if constexpr (S::kSide) {
#pragma unroll
          for (int term = 1; term < 3; ++term) {
            tmem_ld(lane_addr + p * S::kOBlock + term * kRows + kJ * cg, o);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < kJ; ++j) x[j] += __uint_as_float(o[j]);
          }
        }
        const int d = 128 * p + tok;
        const int h0 = row0 + kJ * cg;
        const size_t row = static_cast<size_t>(u.req) * H + h0;
        if (split) {
#pragma unroll
          for (int j = 0; j < kJ; ++j)
            if (h0 + j < rows) a.o_part[part_offset(u.out_slot, h0 + j, d, H)] = x[j] * inv[j];
        } else if (kOutF32) {
#pragma unroll
          for (int j = 0; j < kJ; ++j)
            if (h0 + j < rows) static_cast<float*>(a.out)[(row + j) * kDCkv + d] = x[j] * inv[j];
        } else {
          // two lanes trade halves of two query rows: each stores two dims of one
#pragma unroll
          for (int j = 0; j < kJ; j += 2) {
            const float x0 = x[j] * inv[j], x1 = x[j + 1] * inv[j + 1];
            const bool odd = lane & 1;
            const float got = __shfl_xor_sync(~0u, odd ? x0 : x1, 1);
            const uint32_t w = odd ? pack_bf16x2(got, x1) : pack_bf16x2(x0, got);
            const int h = j + (odd ? 1 : 0);
            if (h0 + h < rows)
              *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + (row + h) * kDCkv + (d & ~1)) = w;
          }
        }
      }
      if (q == 0 && lane < kJ) refs[lane] = 0.f;   // the next unit's first tile sets them
      tc_fence_before();             // O is read: the next unit's first P . V waits for P of all warps
      named_bar_sync(1 + cg, 128);   // red and the references may be written again
    }
    if (!ok && lane == 0) report_error(a.err, kErrTimeout);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int kRows, bool kOutF32>
cudaError_t prepare() {
  return cudaFuncSetAttribute(decode_q4_kernel<kRows, kOutF32>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<kRows>());
}
template <int kRows, bool kOutF32>
cudaError_t launch(const DecodeArgs& a, int groups, cudaStream_t s) {
  return launch_dependent(decode_q4_kernel<kRows, kOutF32>, a.n_workers / groups * groups, Shape<kRows>::kThreads, smem_bytes<kRows>(), 1, s, a);
}

}  // namespace

#ifdef MLA_STALL_TEST
// Test build only: the signal CTA 0 leaves out (0: none).
extern "C" int mla_test_set_q4_stall(int signal) {
  return static_cast<int>(cudaMemcpyToSymbol(g_q4_stall, &signal, sizeof(signal)));
}
#endif

cudaError_t prepare_decode_q4() {
  for (const cudaError_t e : {prepare<16, false>(), prepare<16, true>(), prepare<32, false>(), prepare<32, true>(), prepare<64, false>(),
                              prepare<64, true>()})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

int decode_q4_groups(int rows) { return (rows + 63) / 64; }

cudaError_t launch_decode_q4(const DecodeArgs& a, bool out_f32, cudaStream_t s) {
  // as few columns as hold the query rows: N is what both products cost beyond A
  const int H = a.num_heads, groups = decode_q4_groups(H);
  if (H <= 16) return out_f32 ? launch<16, true>(a, groups, s) : launch<16, false>(a, groups, s);
  if (H <= 32) return out_f32 ? launch<32, true>(a, groups, s) : launch<32, false>(a, groups, s);
  return out_f32 ? launch<64, true>(a, groups, s) : launch<64, false>(a, groups, s);
}

}  // namespace mla
