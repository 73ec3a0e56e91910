// Weighted combine of the layer with 4-bit experts, whose output rows the second product leaves as
// fp16 numbers with a power of two for each 64 columns of a row.
//
// Bound by memory: 16384 tokens of 2048 values with 8 experts read 540 MB and write 67 in 100 us,
// 6 TB/s.  Scaled fp16 keeps y to 2^-11 of each value (and to 2^-39 of the largest of the 64, which
// counts for those 2^28 times smaller) in the two bytes in which bf16 would keep it to 2^-8; fp32
// would cost twice the bytes here and in the product's epilogue.
#include <algorithm>

#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kWaves = 4;        // tokens of a workgroup
constexpr int kVecPerLane = 4;   // 16-byte vectors a lane keeps in flight per pass
constexpr int kSplitTokens = 256;  // up to this many tokens share rows out over gridDim.y

// As combine_rows (permute_combine.hip): one wave per token, slots in groups of four, fp32
// sums in ascending slot order.  Tokens [t0, t_mid) read y0, the others y1.
__global__ void __launch_bounds__(64 * kWaves)
combine_scaled(const u32x4* __restrict__ y0, const uint8_t* __restrict__ s0,
               const u32x4* __restrict__ y1, const uint8_t* __restrict__ s1, int t_mid,
               const int32_t* __restrict__ dst_row, const float* __restrict__ w,
               u32x4* __restrict__ out, int t0, int t1, int k, int nvec, int row_scales) {
  typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
  const int lane = threadIdx.x & 63;
  const int t = t0 + blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (t >= t1) return;
  const u32x4* __restrict__ y = t < t_mid ? y0 : y1;  // wave-uniform
  const uint8_t* __restrict__ sc = t < t_mid ? s0 : s1;
  const int my_row = lane < k ? dst_row[(size_t)t * k + lane] : -1;
  const float my_w = lane < k ? w[(size_t)t * k + lane] : 0.0f;
  for (int v0 = blockIdx.y * 64 * kVecPerLane; v0 < nvec; v0 += gridDim.y * 64 * kVecPerLane) {
    float acc[kVecPerLane][8] = {};
    for (int j0 = 0; j0 < k; j0 += 4) {
      u32x4 rows[4][kVecPerLane];
      uint8_t power[4][kVecPerLane];
      int rj[4];
      float wj[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        rj[g] = j0 + g < k ? __shfl(my_row, j0 + g) : -1;
        wj[g] = __shfl(my_w, (j0 + g) & 63);
        if (rj[g] < 0) continue;
        const u32x4* src = y + (size_t)rj[g] * nvec;
        const uint8_t* ssrc = sc + (size_t)rj[g] * row_scales;
#pragma unroll
        for (int i = 0; i < kVecPerLane; ++i) {
          const int v = v0 + i * 64 + lane;
          if (v < nvec) {
            rows[g][i] = __builtin_nontemporal_load(&src[v]);
            power[g][i] = ssrc[v >> 3];
          }
        }
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (rj[g] < 0) continue;
#pragma unroll
        for (int i = 0; i < kVecPerLane; ++i) {
          if (v0 + i * 64 + lane >= nvec) continue;
          const f16x8 h = __builtin_bit_cast(f16x8, rows[g][i]);
          const float p = __uint_as_float((uint32_t)power[g][i] << 23);
          // (the power of two apart from the weight: their product could leave the range)
#pragma unroll
          for (int q = 0; q < 8; ++q)
            acc[i][q] = __builtin_fmaf(wj[g], (float)h[q] * p, acc[i][q]);
        }
      }
    }
    u32x4* dst = out + (size_t)t * nvec;
#pragma unroll
    for (int i = 0; i < kVecPerLane; ++i) {
      const int v = v0 + i * 64 + lane;
      if (v < nvec) __builtin_nontemporal_store(pack_bf16x8(acc[i]), &dst[v]);
    }
  }
}

}  // namespace

hipError_t launch_combine_scaled(const Shape& s, int t0, int t_mid, int t1, const ScaledRows (&y)[2],
                                 const int32_t* dst_row, const float* w, void* out,
                                 hipStream_t st) {
  if (t1 <= t0) return hipSuccess;
  const int nvec = s.H / 8;
  const int spans = (nvec + 64 * kVecPerLane - 1) / (64 * kVecPerLane);
  const unsigned parts = t1 - t0 <= kSplitTokens ? (unsigned)std::min(spans, 256) : 1u;
  // (a launch has less than 2^32 threads, 64 for every token)
  constexpr int kMost = 1 << 25;
  for (int64_t t = t0; t < t1; t += kMost) {
    const int end = (int)std::min<int64_t>(t + kMost, t1);
    const unsigned blocks = (unsigned)((end - t + kWaves - 1) / kWaves);
    hipLaunchKernelGGL(combine_scaled, dim3(blocks, parts), dim3(64 * kWaves), 0, st,
                       (const u32x4*)y[0].values, (const uint8_t*)y[0].scales,
                       (const u32x4*)y[1].values, (const uint8_t*)y[1].scales, t_mid, dst_row, w,
                       (u32x4*)out, (int)t, end, s.k, nvec, (int)mx_out_scales(s.H));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
