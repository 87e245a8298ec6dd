// The row of a 4-bit cache (mla_decode.h, MLA_DTYPE_Q4): 304 bytes a token.
//
// A word of the codes holds 8 dims: the 3-bit index of dim i's magnitude at bit
// 4i, the signs of dims 0 .. 3 at bits 8i + 7 and of dims 4 .. 7 at 8 (i - 4) +
// 3.  So the low and the high half of the word, without the signs, select four
// bytes each out of a table of eight magnitudes (one byte permute), and one mask
// (of the word, of the word shifted by 4) puts the signs into the top bits of
// those bytes.
//
// Rows are 304 = 16 * 19 bytes apart: 16-byte aligned, and the same 16-byte
// chunk of eight consecutive rows in shared memory falls into eight different
// groups of banks (76 words = 12 modulo 32).
#pragma once
#include <cstdint>

#include "mla_decode.h"
#include "mla_internal.h"

namespace mla {

constexpr int kQ4Row = MLA_Q4_ROW_BYTES;
constexpr int kQ4Group = 32;                   // dims that share a shift
constexpr int kQ4Groups = kD / kQ4Group;       // 18
constexpr int kQ4Words = kD / 8;               // words of codes
constexpr int kQ4Meta = kQ4Words * 4;          // byte offset of the shifts (288)
constexpr int kQ4MinExp = -32, kQ4MaxExp = 63, kQ4MaxShift = 14;
constexpr int kQ4NanExp = 255;                 // exponent byte of a row that held a NaN
static_assert(kQ4Row == kQ4Meta + 16 && kQ4Row % 16 == 0, "row layout");

// The 16 bytes behind a row's codes.
struct Q4Meta {
  uint4 v;
  __device__ __forceinline__ int shift(int group) const {
    const uint32_t w = group < 8 ? v.x : group < 16 ? v.y : v.z;
    return (w >> (4 * (group & 7))) & 15;
  }
  __device__ __forceinline__ int exp_byte() const { return (v.z >> 8) & 255; }
};

// 2^e for e in -126 .. 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// The values of a word's 8 dims, times 2^-26: the magnitude's three bits, put
// where fp32 has the last exponent bits and the first of the mantissa, are the
// magnitude times 2^-126 (fp32's subnormals being e2m1's); one exact product
// brings that to 2^-26, from where every unit of a row (2^-46 .. 2^63) is one
// more exact product away.
__device__ __forceinline__ void q4_expand(uint32_t w, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t mag = (i < 6 ? w << (22 - 4 * i) : w >> (4 * i - 22)) & 0x01c00000u;
    const uint32_t sign = (i < 4 ? w << (24 - 8 * i) : w << (28 - 8 * (i - 4))) & 0x80000000u;
    x[i] = __uint_as_float(mag | sign) * 0x1p100f;
  }
}
// What takes q4_expand's numbers to a group's values: 2^(26 + E - k), NaN in a
// row that held one.
__device__ __forceinline__ float q4_unit(const Q4Meta& m, int group) {
  const int e = m.exp_byte();
  if (e == kQ4NanExp) return __int_as_float(0x7fffffff);
  return pow2(min(26 + e - 127 - m.shift(group), 127));
}


// A group's magnitudes as bf16 numbers, which are the upper halves of the fp32
// ones: the values 2^-47 .. 6 * 2^63 are exact in both.  Split into the numbers'
// upper and lower bytes, which the indices select as they do in the decode.
struct Q4Table {
  uint2 hi, lo;
};
__device__ __forceinline__ Q4Table q4_table(const Q4Meta& m, int group) {
  // 2^(E - k) has the exponent field f; index 1 is half of it, 2 itself, 3 1.5 times ..
  const uint32_t f = min(max(m.exp_byte() - m.shift(group), 1), 250), two = f * 0x00800080u;
  uint32_t w[4] = {(f - 1) << 23, two + 0x00400000u, two + 0x00c00080u, two + 0x01400100u};
  if (m.exp_byte() == kQ4NanExp) w[0] = w[1] = w[2] = w[3] = 0x7fff7fffu;
  return {make_uint2(__byte_perm(w[0], w[1], 0x7531), __byte_perm(w[2], w[3], 0x7531)),
          make_uint2(__byte_perm(w[0], w[1], 0x6420), __byte_perm(w[2], w[3], 0x6420))};
}
// The bf16 numbers of a word's 8 dims, two to a word.
__device__ __forceinline__ uint4 q4_bf16x8(const Q4Table& t, uint32_t w) {
  const uint32_t a = w & 0x77777777u;
  const uint32_t h0 = __byte_perm(t.hi.x, t.hi.y, a) | (w & 0x80808080u), l0 = __byte_perm(t.lo.x, t.lo.y, a);
  const uint32_t h1 = __byte_perm(t.hi.x, t.hi.y, a >> 16) | ((w << 4) & 0x80808080u), l1 = __byte_perm(t.lo.x, t.lo.y, a >> 16);
  return make_uint4(__byte_perm(l0, h0, 0x5140), __byte_perm(l0, h0, 0x7362), __byte_perm(l1, h1, 0x5140), __byte_perm(l1, h1, 0x7362));
}

}  // namespace mla
