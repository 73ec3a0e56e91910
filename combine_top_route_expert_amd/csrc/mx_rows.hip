// Row kernels of the layer with 4-bit experts: the input rows, sorted by expert, in two
// 6-bit parts (mx_rows.h), and the weighted combine of the output rows, which the second
// product leaves as fp16 numbers with a power of two for each 64 columns of a row.
//
// Both are bound by memory.  A workgroup of the first takes a row block, found by the
// products' own tile map; its waves take 64 columns of the 32 rows at a time, 64 bytes of a
// row to a lane.  It does the layer's permute as well: k rows are written for every token, and
// the first product copies contiguous blocks.  16384 tokens of 2048 values with 8 experts:
// 145 us for 400 MB written and 540 read, most of them from the caches (6.5 TB/s).  Without
// effect: the next block's loads ahead of a split, eight times the workgroups (2% less time).
// One split of each token whose parts go to its k places, 16 bytes at a time: 0 to 20% more of
// the layer's time at every size, the most where rows are many.
//
// The combine reads 540 MB and writes 67 there in 100 us, 6 TB/s.  Scaled fp16 keeps y to 2^-12 in
// the two bytes that bf16 would spend on 2^-9: of the layer's roundings (two parts of x and
// act, y, out) y's was the largest but one.
#include <algorithm>

#include "mx_rows.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

struct SplitArgs {
  const u32x4* x;             // [T][H] bf16
  const int32_t *off0, *off1;
  const int32_t* gather[2];   // src_row slices
  int E, k, H;
  MxRows to;
};

__global__ void __launch_bounds__(kThreads) split_rows(SplitArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  MTileMap tm;
  tm.build(a.off0, a.off1, a.E, 32, 1);
  if ((int)blockIdx.x >= tm.total) return;
  const TileRows tr = tm.locate(a.off0, a.off1, 32, blockIdx.x);
  const int r = lane & 31, half = lane >> 5;
  if (r >= tr.rows) return;
  int part;
  const int cr = tr.split_row(tr.v0 + r, &part);
  const int32_t *g0 = a.gather[0], *g1 = a.gather[1];
  const int64_t token = (part ? g1 : g0)[cr] / a.k;
  const u32x4* x = a.x + token * (a.H / 8) + half * 4;
  const int nk = a.H / 64;
  const int64_t rb = mx_row_block(tr, tr.v0);
  for (int k = blockIdx.y * (kThreads / 64) + wave; k < nk; k += gridDim.y * (kThreads / 64)) {
    u32x4 v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = x[k * 8 + q];
    f32x16v even, odd;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const uint32_t two = v[q / 4][q % 4];
      even[q] = __uint_as_float(two << 16);
      odd[q] = __uint_as_float(two & 0xffff0000u);
    }
    store_parts(split32(even, odd), a.to, nk, rb, r, 2 * k + half);
  }
}

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

hipError_t launch_split_rows(const Shape& s, const MxIO& io, const void* x, const MxRows& to,
                             hipStream_t st) {
  if (io.rows_bound <= 0) return hipSuccess;
  SplitArgs a{};
  a.x = (const u32x4*)x;
  a.off0 = io.off[0];
  a.off1 = io.off[1];
  a.gather[0] = io.gather[0];
  a.gather[1] = io.off[1] ? io.gather[1] : io.gather[0];
  a.E = s.E;
  a.k = s.k;
  a.H = s.H;
  a.to = to;
  const int64_t blocks = m_tiles_bound(io.rows_bound, s.E, 32);
  if (blocks > 0x7fffffff / kThreads) return hipErrorInvalidConfiguration;
  // few row blocks: their columns to several workgroups
  const int parts = (int)std::max<int64_t>(
      1, std::min<int64_t>(s.H / 64 / (kThreads / 64), 2048 / std::max<int64_t>(blocks, 1)));
  hipLaunchKernelGGL(split_rows, dim3((unsigned)blocks, (unsigned)parts), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_combine_scaled(const Shape& s, int t0, int t_mid, int t1, const MxRows (&y)[2],
                                 const int32_t* dst_row, const float* w, void* out,
                                 hipStream_t st) {
  if (t1 <= t0) return hipSuccess;
  const int nvec = s.H / 8;
  const unsigned blocks = (unsigned)((t1 - t0 + kWaves - 1) / kWaves);
  const int spans = (nvec + 64 * kVecPerLane - 1) / (64 * kVecPerLane);
  const unsigned parts = t1 - t0 <= kSplitTokens ? (unsigned)std::min(spans, 256) : 1u;
  hipLaunchKernelGGL(combine_scaled, dim3(blocks, parts), dim3(64 * kWaves), 0, st,
                     (const u32x4*)y[0].values, (const uint8_t*)y[0].scales,
                     (const u32x4*)y[1].values, (const uint8_t*)y[1].scales, t_mid, dst_row, w,
                     (u32x4*)out, t0, t1, s.k, nvec, (int)mx_out_scales(s.H));
  return hipGetLastError();
}

}  // namespace moe
