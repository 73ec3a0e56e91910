// Packed 4-bit weights as operands of the bf16 matrix instructions.
#pragma once

#include "fp4_layout.h"
#include "gemm_tile.h"

namespace moe {

namespace {

// A lane's 8 weights of a dword times their group's power of two: exact, but a product past 2^128
// is an infinity, and scale byte 255 gives NaN.
__device__ __forceinline__ bf16x8 unpack_fp4(uint32_t w, uint32_t scale_byte) {
  bf16x8 v{};
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const float p = __uint_as_float(scale_byte << 23);
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p, 0);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p, 1);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p, 2);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, p, 3);
  v = bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
#endif
  return v;
}

}  // namespace

}  // namespace moe
