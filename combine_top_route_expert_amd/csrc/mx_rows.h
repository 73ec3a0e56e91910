// Rows in two 6-bit parts, the form in which the 4-bit layer's products take their
// activations (the layer's input and act): for each 32 consecutive values x of a row
//   x ~ h + l,  h = E2M3(x / 2^s) 2^s,  l = E2M3((x - h) / 2^t) 2^t
// E2M3: sign, two exponent bits, three of mantissa (magnitudes 0, 1/8 .. 7 1/2), nearest,
// ties to even; s and t the least integers (at least -127) that clip nothing.
//
// Why: gfx950 multiplies 4-bit weights by 6-bit values, each side with a power of two
// for 32 of them, at four times the rate of bf16, so that two parts cost half of the bf16
// product, and the weights enter the matrix instruction as they lie in memory.  h + l is off
// by at most 2^-8.9 of the largest of the 32 values; over them it is closer than a
// rounding to bf16: root mean square 0.8e-3 of normally distributed values against
// 1.7e-3, 1.3e-3 where one in a hundred is a hundred times larger.  (Three parts would
// be exact to 2^-15 and cost half as much again.)
//
// Layout: as the packed weights' (fp4_layout.h), blocks of 32 rows by 64 columns, block
// after block along the columns, so that the products copy whole kilobytes (rows as
// 96-byte pieces, 64 columns each, came at 26 bytes a cycle to a CU instead of 36).  With
// entry 32 h + r for row r and columns 32 h .. + 31 of a block, 24 bytes of part h and
// 24 of part l, a block holds the first 16 bytes of all 64 entries, then the next 16, then the
// last 16: three reads give a lane both parts' operands in consecutive registers.  Two
// blocks' scales lie together, 256 bytes: bytes 4 (32 h + r) + 2 (k % 2) of part h and
// one more of part l for block k (exponent + 127; 255: NaN).
//
// An expert's rows start at a block of their own: block J / 32 + e for expert e with J rows
// before it (each expert before it adds at most one part of a block, so that no two
// overlap).  Rows past an expert's last are left as they are, and only feed output rows that
// are never stored.
#pragma once

#include "row_quantizer.h"

namespace moe {

constexpr int kMxBlockBytes = 3 * 1024, kMxScaleBytes = 256;  // of a block; of two blocks' scales

// Row blocks of `rows` rows shared out among E experts.
inline int64_t mx_row_blocks(int64_t rows, int E) { return rows / 32 + E; }
inline int64_t mx_value_bytes(int64_t row_blocks, int64_t cols) {
  return row_blocks * (cols / 64) * kMxBlockBytes;
}
inline int64_t mx_scale_bytes(int64_t row_blocks, int64_t cols) {
  return row_blocks * ((cols / 64 + 1) / 2) * kMxScaleBytes;
}

namespace {

typedef uint32_t u32x6 __attribute__((ext_vector_type(6)));
typedef float f32x16v __attribute__((ext_vector_type(16)));
typedef float f32x32 __attribute__((ext_vector_type(32)));

// The scale byte of values of which `big` is the bits of the largest magnitude (finite):
// with big = m 2^e, 7.5 2^s = 1.875 2^(s + 2) holds it from s = e - 2 (m <= 1.875) or
// e - 1 on.
__device__ __forceinline__ uint32_t e2m3_scale(uint32_t big) {
  const int byte = (int)((big + 0x0fffffu) >> 23) - 2;
  return byte > 0 ? (uint32_t)byte : 0u;
}

struct TwoParts {
  u32x6 h, l;
  uint32_t hs, ls;  // scale bytes
};

// The 32 values as their even and their odd ones (the conversion interleaves its two
// operands).  Magnitudes above 1.875 * 2^127, whose h would round to 2^128, count as infinite.
__device__ __forceinline__ TwoParts split32(f32x16v even, f32x16v odd) {
  TwoParts p{};
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t a = __float_as_uint(even[i]) & 0x7fffffffu;
    const uint32_t b = __float_as_uint(odd[i]) & 0x7fffffffu;
    big = a > big ? a : big;
    big = b > big ? b : big;
  }
  if (big > 0x7f700000u) {  // (unsigned: finite < infinity < NaN): the row's products are NaN
    p.hs = p.ls = 255;
    return p;
  }
  p.hs = e2m3_scale(big);
#if defined(__HIP_DEVICE_COMPILE__)
  const float hp = __uint_as_float(p.hs << 23);
  p.h = __builtin_amdgcn_cvt_scalef32_2xpk16_fp6_f32(even, odd, hp);
  const f32x32 back = __builtin_amdgcn_cvt_scalef32_pk32_f32_fp6(p.h, hp);
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    even[i] -= back[2 * i];
    odd[i] -= back[2 * i + 1];
    const uint32_t a = __float_as_uint(even[i]) & 0x7fffffffu;
    const uint32_t b = __float_as_uint(odd[i]) & 0x7fffffffu;
    most = a > most ? a : most;
    most = b > most ? b : most;
  }
  p.ls = e2m3_scale(most);
  p.l = __builtin_amdgcn_cvt_scalef32_2xpk16_fp6_f32(even, odd, __uint_as_float(p.ls << 23));
#endif
  return p;
}

// Row block and block behind row v of a tile's expert.
__device__ __forceinline__ int64_t mx_row_block(const TileRows& tr, int v) {
  return (tr.lo0 + tr.lo1) / 32 + tr.e + v / 32;
}

// Stores columns 32 group .. + 31 of row r of row block rb; nk blocks to a row.
__device__ __forceinline__ void store_parts(const TwoParts& p, const MxRows& to, int nk, int64_t rb,
                                            int r, int group) {
  const int k = group >> 1, entry = 32 * (group & 1) + r;
  char* at = to.values + (rb * nk + k) * kMxBlockBytes + entry * 16;
  *(u32x4*)at = u32x4{p.h[0], p.h[1], p.h[2], p.h[3]};
  *(u32x4*)(at + 1024) = u32x4{p.h[4], p.h[5], p.l[0], p.l[1]};
  *(u32x4*)(at + 2048) = u32x4{p.l[2], p.l[3], p.l[4], p.l[5]};
  *(uint16_t*)(to.scales + (rb * ((nk + 1) / 2) + k / 2) * kMxScaleBytes + entry * 4 + 2 * (k & 1)) =
      (uint16_t)(p.hs | p.ls << 8);
}

}  // namespace

}  // namespace moe
