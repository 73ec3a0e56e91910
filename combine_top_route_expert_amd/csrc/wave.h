// Reductions over the 64 lanes of a wave by data-parallel shifts, shared by the row
// kernels, the router and the few-rows products.
#pragma once

#include <type_traits>

#include "moe_internal.h"

namespace moe {

namespace {

// v of another lane by a data-parallel shift (a few cycles; through LDS it would be
// some sixty), zero where there is none: 0x111..0x118 from 1..8 lanes before in the
// same row of 16, 0x142 / 0x143 from the last lane of the row / half before.  All
// lanes have to be active.
template <int kControl, int kRowMask>
__device__ __forceinline__ int wave_shift(int v) {
  return __builtin_amdgcn_update_dpp(0, v, kControl, kRowMask, 0xf, false);
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto with = [&](uint32_t o) __attribute__((always_inline)) { v = o > v ? o : v; };
  with(wave_shift<0x111, 0xf>(v));
  with(wave_shift<0x112, 0xf>(v));
  with(wave_shift<0x114, 0xf>(v));
  with(wave_shift<0x118, 0xf>(v));
  with(wave_shift<0x142, 0xa>(v));
  with(wave_shift<0x143, 0xc>(v));
  return __builtin_amdgcn_readlane(v, 63);
}

// Sum over the wave: within rows of 16 lanes, then each row's total into the row
// after it, so that lane 63 ends with all of it.
__device__ __forceinline__ float wave_sum(float v) {
  v += __int_as_float(wave_shift<0x111, 0xf>(__float_as_int(v)));
  v += __int_as_float(wave_shift<0x112, 0xf>(__float_as_int(v)));
  v += __int_as_float(wave_shift<0x114, 0xf>(__float_as_int(v)));
  v += __int_as_float(wave_shift<0x118, 0xf>(__float_as_int(v)));
  v += __int_as_float(wave_shift<0x142, 0xa>(__float_as_int(v)));
  v += __int_as_float(wave_shift<0x143, 0xc>(__float_as_int(v)));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

__device__ __forceinline__ double wave_sum(double v) {
  auto add = [&](auto control, auto rows) __attribute__((always_inline)) {
    constexpr int kControl = decltype(control)::value, kRows = decltype(rows)::value;
    v += __hiloint2double(wave_shift<kControl, kRows>(__double2hiint(v)),
                          wave_shift<kControl, kRows>(__double2loint(v)));
  };
  const std::integral_constant<int, 0xf> all{};
  add(std::integral_constant<int, 0x111>{}, all);
  add(std::integral_constant<int, 0x112>{}, all);
  add(std::integral_constant<int, 0x114>{}, all);
  add(std::integral_constant<int, 0x118>{}, all);
  add(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});
  add(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), 63),
                          __builtin_amdgcn_readlane(__double2loint(v), 63));
}

}  // namespace

}  // namespace moe
