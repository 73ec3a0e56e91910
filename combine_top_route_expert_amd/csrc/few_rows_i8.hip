// The 8-bit layer for a few assignments (a decoded token, or a handful), in two
// launches.
//
// The tiles of gemm_i8.hip need rows to share a weight panel and tiles to fill the
// chip: one token with four experts of H = 2048, I = 1024 gives them 64 workgroups
// that stream 16 stages of K one after the other (gate_up 16.3 us, down 10.7 us),
// between 5 us of sorting, 4 us of quantising and 4 us of combining.  Here nothing is
// sorted: row f of act belongs to assignment f, whose expert is top_k_index[f].
//  few_gate_up  every wave takes 4 gate rows and the up rows of the same columns for
//               one assignment (5.8 us for that token)
//  few_down     a workgroup takes one token's 16 output columns: it quantises the
//               token's act rows into LDS (its waves take them in turn), then each
//               wave multiplies 4 columns with two of the token's experts at a time
//               and adds the weighted results in slot order (8.6 us)
// A wave's lanes hold 16 bytes of each kilobyte of K of 8 weight rows, so that 8 KB
// or more are in flight.  few_gate_up has A I / 4 waves, one for every 8 weight
// rows, few_down T H / 4, one for every 4 k rows: 1024 and 512 for that token, the
// latter in 128 workgroups, half a wave for each SIMD.  Memory bounds both from about
// E = 256, H = 7168 on (one token: 6 TB/s).  Below that their own latency does, and
// few_down, with half the bytes, takes longer: fewer waves, slots in dependent rounds
// of two, and the quantiser before the first weight load.  An expert that two assignments share is read
// twice, mostly from the caches; few_rows() says when that is worth it.
//
// Dot products of four bytes at a time (v_dot4_i32_i8) give each lane 8 exact partial
// sums, added over the wave by halving exchanges: each step gives one half of the
// sums away and receives the other lanes' part of the half that is kept.  Sums are
// integers, and scaling, rounding, quantiser and the order of the slots are those of
// the sorted path, so the bits are the same.
#include "row_quantizer.h"

namespace moe {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;        // waves of a workgroup
constexpr int kCols = 4;         // output columns of a wave
constexpr int kRows = 8;         // weight rows of a wave at a time
constexpr int kLdsRows = 65536;  // bytes of quantised act rows a workgroup holds

struct FewArgs {
  const void* A;           // gate_up: hidden_q; down: act rows in the layer's dtype
  const float* a_scale;    // gate_up: hidden_scale
  const int8_t* B;
  const float* b_scale;
  const float* top_k_weights;  // down
  void* C;                 // gate_up: act [T*k][I]; down: out [T][H]
  const int32_t* idx;
  int32_t* dev_error;      // gate_up
  int rows, E, k, K, ncols;
};

// acc[i] += the dot product of the lane's 16 bytes of weight row i and of x.
template <int N>
__device__ __forceinline__ void dot16(const i32x4 (&w)[N], const i32x4& x, int* acc) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[i] = __builtin_amdgcn_sdot4(w[i][q], x[q], acc[i], false);
}

// Sums 8 values over the wave: lane l returns the sum of value l / 8.
__device__ __forceinline__ int wave_sum8(int (&acc)[kRows], int lane) {
#pragma unroll
  for (int half = 4, mask = 32; half > 0; half >>= 1, mask >>= 1) {
    const bool up = lane & mask;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const int give = up ? acc[i] : acc[i + half], keep = up ? acc[i + half] : acc[i];
      acc[i] = keep + __shfl_xor(give, mask);
    }
  }
  int s = acc[0];
#pragma unroll
  for (int mask = 4; mask > 0; mask >>= 1) s += __shfl_xor(s, mask);
  return s;
}

template <bool kBf16>
__global__ void __launch_bounds__(64 * kWaves) few_gate_up_i8(FewArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = a.ncols / (kWaves * kCols);
  const int f = blockIdx.x / groups;
  const int c0 = ((blockIdx.x % groups) * kWaves + wave) * kCols;
  if (blockIdx.x == 0 && wave == 0) {
    // at most 64 assignments, one per lane
    const int id = lane < a.rows ? a.idx[lane] : 0;
    const int dropped = __popcll(__ballot(lane < a.rows && (id < 0 || id >= a.E)));
    if (lane == 0) *a.dev_error = dropped;
  }
  const int e = __builtin_amdgcn_readfirstlane(a.idx[f]);
  if (e < 0 || e >= a.E) return;
  const int K = a.K, t = f / a.k;
  const int64_t brow0 = (int64_t)e * 2 * a.ncols + c0;  // the first gate row
  const int8_t* bp[kRows];
#pragma unroll
  for (int c = 0; c < kRows; ++c)
    bp[c] = a.B + (brow0 + (c >> 2) * a.ncols + (c & 3)) * K;
  const int my = lane >> 3;  // the row whose sum this lane gets
  const float cs = a.b_scale[brow0 + (my >> 2) * a.ncols + (my & 3)];
  const float rs = a.a_scale[t];
  const int8_t* x8 = (const int8_t*)a.A + (int64_t)t * K;
  int acc[kRows] = {};
#pragma unroll 2
  for (int k = lane * 16; k < K; k += 1024) {
    i32x4 w[kRows];
#pragma unroll
    for (int c = 0; c < kRows; ++c) w[c] = __builtin_nontemporal_load((const i32x4*)(bp[c] + k));
    dot16(w, *(const i32x4*)(x8 + k), acc);
  }
  // gate sums are in lanes 0..31, the up sums of the same columns in lanes 32..63
  const float v = (float)wave_sum8(acc, lane) * rs * cs;
  const float o = swiglu<kBf16>(v, __shfl_xor(v, 32));
  if (lane & 7 || lane >= 32) return;
  const int64_t at = (int64_t)f * a.ncols + c0 + my;
  if constexpr (kBf16)
    ((__bf16*)a.C)[at] = (__bf16)o;
  else
    ((float*)a.C)[at] = o;
}

template <bool kBf16>
__global__ void __launch_bounds__(64 * kWaves) few_down_i8(FewArgs a) {
  constexpr int kEl = kVecEl<kBf16>;
  extern __shared__ __attribute__((aligned(16))) int8_t xq[];  // [k][K]
  __shared__ float row_scale[64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = a.ncols / (kWaves * kCols);
  const int t = blockIdx.x / groups;
  const int c0 = ((blockIdx.x % groups) * kWaves + wave) * kCols;
  const int K = a.K;
  const int32_t* ids = a.idx + (int64_t)t * a.k;
  auto expert = [&](int j) __attribute__((always_inline)) {
    const int e = __builtin_amdgcn_readfirstlane(ids[j]);
    return e >= 0 && e < a.E ? e : -1;
  };
  for (int j = wave; j < a.k; j += kWaves) {
    if (expert(j) < 0) continue;  // a dropped slot has no act row
    const u32x4* act = (const u32x4*)a.A + ((int64_t)t * a.k + j) * (K / kEl);
    uint32_t big = 0;
    float v[kEl];
    for (int i = lane; i < K / kEl; i += 64) {
      unpack<kBf16>(act[i], v);
      big = max_magnitude<kEl>(v, big);
    }
    const RowQuantizer<kBf16> quant(wave_max(big));
    if (lane == 0) row_scale[j] = quant.scale;
    for (int i = lane; i < K / kEl; i += 64) {
      unpack<kBf16>(act[i], v);
      quant.store(v, xq + j * K, i);
    }
  }
  __syncthreads();
  const int my = lane >> 3, my_slot = my >> 2, my_col = my & 3;
  float out = 0.0f;  // of column my_col, the same in both halves of the wave
  for (int j = 0; j < a.k; j += 2) {
    const int e[2] = {expert(j), j + 1 < a.k ? expert(j + 1) : -1};
    int acc[kRows] = {};
#pragma unroll 2
    for (int k = lane * 16; k < K; k += 1024) {
      i32x4 w[2][kCols];
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (e[s] >= 0) {
          const int8_t* b = a.B + ((int64_t)e[s] * a.ncols + c0) * K + k;
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            w[s][c] = __builtin_nontemporal_load((const i32x4*)(b + (int64_t)c * K));
        }
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (e[s] >= 0) dot16(w[s], *(const i32x4*)(xq + (j + s) * K + k), acc + s * kCols);
    }
    const int me = my_slot ? e[1] : e[0];
    float y = (float)wave_sum8(acc, lane);
    if (me >= 0) y = y * row_scale[j + my_slot] * a.b_scale[(int64_t)me * a.ncols + c0 + my_col];
    // nothing is stored here, but the sorted path keeps y in bf16 (written and read
    // again there, which fp32 would double), and both give the same bits
    if constexpr (kBf16) y = (float)(__bf16)y;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const float ys = __shfl(y, s * 32 + my_col * 8);
      if (e[s] >= 0)
        out = __builtin_fmaf(a.top_k_weights[(int64_t)t * a.k + j + s], ys, out);
    }
  }
  if (lane & 7 || lane >= 32) return;
  const int64_t at = (int64_t)t * a.ncols + c0 + my;
  if constexpr (kBf16)
    ((__bf16*)a.C)[at] = (__bf16)out;
  else
    ((float*)a.C)[at] = out;
}

}  // namespace

// At most 32 assignments, and no more than there are experts (those of one token
// are distinct in any case), whose quantised rows fit a workgroup's LDS: an expert
// that several assignments share is read for each of them.  Whole layer in us,
// sorted tiles / this form, routed evenly:
//   E = 256, H = 7168, I = 2048, k = 8: 8 assignments 77 / 63, 32: 224 / 216
//   E = 16, H = I = 2880, k = 4:  4: 58 / 29, 16: 93 / 70, 32: 97 / 127
//   E = 8, H = 4096, I = 2048, k = 2:  2: 44 / 18, 8: 50 / 36, 16: 54 / 68
//   E = 4, H = 2048, I = 1408, k = 2:  4: 33 / 14, 16: 34 / 21, 32: 34 / 36
// The bound by E is on the safe side: it also leaves small experts that are shared
// a few times, whose repeats come from the caches, to the slower sorted tiles (E = 4,
// 16 assignments: 34 instead of 21 us).
bool few_rows(const Shape& s) {
  return s.A > 0 && s.A <= 32 && (s.T == 1 || s.A <= s.E) && (int64_t)s.k * s.I <= kLdsRows;
}

hipError_t launch_few_i8(const Shape& s, const int8_t* hidden_q, const float* hidden_scale,
                         const int32_t* top_k_index, const float* top_k_weights,
                         const int8_t* w_gate_up, const float* w_gate_up_scale,
                         const int8_t* w_down, const float* w_down_scale, void* act, void* out,
                         int32_t* dev_error, hipStream_t st) {
  FewArgs g{};
  g.idx = top_k_index;
  g.rows = (int)s.A;
  g.E = s.E;
  g.k = s.k;
  FewArgs d = g;
  g.A = hidden_q;
  g.a_scale = hidden_scale;
  g.B = w_gate_up;
  g.b_scale = w_gate_up_scale;
  g.C = act;
  g.dev_error = dev_error;
  g.K = s.H;
  g.ncols = s.I;
  d.A = act;
  d.B = w_down;
  d.b_scale = w_down_scale;
  d.top_k_weights = top_k_weights;
  d.C = out;
  d.K = s.I;
  d.ncols = s.H;
  // H and I are multiples of 64: whole workgroups of 16 columns
  const dim3 gg((unsigned)(s.A * (s.I / (kWaves * kCols))));
  const dim3 gd((unsigned)(s.T * (s.H / (kWaves * kCols))));
  const dim3 block(64 * kWaves);
  const size_t lds = (size_t)s.k * s.I;
  if (s.dtype == MOE_BF16) {
    hipLaunchKernelGGL(few_gate_up_i8<true>, gg, block, 0, st, g);
    hipLaunchKernelGGL(few_down_i8<true>, gd, block, lds, st, d);
  } else {
    hipLaunchKernelGGL(few_gate_up_i8<false>, gg, block, 0, st, g);
    hipLaunchKernelGGL(few_down_i8<false>, gd, block, lds, st, d);
  }
  return hipGetLastError();
}

}  // namespace moe
