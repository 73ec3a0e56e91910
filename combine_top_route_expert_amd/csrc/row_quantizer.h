// Rows of 16-byte vectors and their quantisation to 8-bit integers, shared by the
// row kernels (norm_quantize.hip) and the few-rows products (few_rows_i8.hip).
#pragma once

#include <type_traits>

#include "wave.h"

namespace moe {

namespace {

template <bool kBf16>
constexpr int kVecEl = kBf16 ? 8 : 4;  // elements of a 16-byte vector

template <bool kBf16>
__device__ __forceinline__ void unpack(const u32x4& q, float* f) {
  if constexpr (kBf16) {
    unpack_bf16x8(q, f);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(q[i]);
  }
}

template <bool kBf16>
__device__ __forceinline__ u32x4 pack(const float* f) {
  if constexpr (kBf16) {
    return pack_bf16x8(f);
  } else {
    return u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                 __float_as_uint(f[3])};
  }
}

// One row's quantiser, from the bits of its largest magnitude (as an unsigned
// number these order finite < infinity < NaN, so one maximum finds all three).
//
// q must be rne of the exact quotient 127 x / a: a rounded quotient can land on
// the other side of a tie.  bf16 rows: 127 x is exact in fp32, the residual of
// the approximate quotient is exact too (24 + 8 bits, of which all but the last
// few cancel), and one correction step gives the quotient to within far less
// than half a unit of any representable tie.  fp32 rows take the same steps in
// fp64.  Rows whose largest magnitude is beyond 2^+-64 are scaled by a power of
// two first, so neither 127 x nor 1 / a leaves the range.  A row that holds an
// infinity or a NaN has no quotient: q = 0 and a NaN scale, so every product
// with it is NaN.
template <bool kBf16>
struct RowQuantizer {
  typedef std::conditional_t<kBf16, float, double> real;
  float scale;
  real a, r, lift;  // lift: 127 times the power of two
  bool finite;

  __device__ __forceinline__ explicit RowQuantizer(uint32_t max_bits) {
    finite = max_bits < 0x7f800000u;
    const float m = __uint_as_float(max_bits);
    scale = finite ? m / 127.0f : __uint_as_float(0x7fc00000u);
    real p = 1;
    if constexpr (kBf16) p = m > 0x1p64f ? 0x1p-64f : m < 0x1p-64f ? 0x1p64f : 1.0f;
    a = (real)m * p;
    r = finite && max_bits != 0 ? (real)1 / a : (real)0;
    lift = (real)127 * p;
  }
  __device__ __forceinline__ uint32_t operator()(float x) const {
    const real n = (real)x * lift;
    real q = n * r;
    if constexpr (kBf16)
      q = rintf(__builtin_fmaf(__builtin_fmaf(-q, a, n), r, q));
    else
      q = rint(__builtin_fma(__builtin_fma(-q, a, n), r, q));
    return finite ? (uint32_t)(int)q & 0xffu : 0u;
  }
  // four consecutive elements as one word
  __device__ __forceinline__ uint32_t word(const float* f) const {
    return (*this)(f[0]) | (*this)(f[1]) << 8 | (*this)(f[2]) << 16 | (*this)(f[3]) << 24;
  }
  // kVecEl quantised elements of a vector as one 8- or 4-byte store
  __device__ __forceinline__ void store(const float* f, int8_t* q, int64_t v) const {
    constexpr int W = kVecEl<kBf16> / 4;
    uint32_t o[W];
#pragma unroll
    for (int i = 0; i < W; ++i) o[i] = word(f + 4 * i);
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    if constexpr (W == 2)
      *(u32x2*)(q + v * 8) = u32x2{o[0], o[1]};
    else
      *(uint32_t*)(q + v * 4) = o[0];
  }
};

template <int N>
__device__ __forceinline__ uint32_t max_magnitude(const float* f, uint32_t m) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t b = __float_as_uint(f[i]) & 0x7fffffffu;
    m = b > m ? b : m;
  }
  return m;
}

}  // namespace

}  // namespace moe
