// The 8-bit expert products of a few assignments (a decoded token, or a handful).
//
// The tiles of gemm_i8.hip need rows to share a weight panel and tiles to fill the
// chip; one token with four experts of H = 2048, I = 1024 gives them 64 workgroups
// that stream 16 stages of K one after the other: gate_up 16.3 us and down 10.7 us,
// behind 5 us of sorting and before 4 us of quantising.  Here every wave takes 8 rows
// of B (gate_up: 4 gate rows and the up rows of the same columns) for one
// assignment: its lanes hold 16 bytes of each kilobyte of K, so a wave has 8 KB or
// more in flight and a launch as many waves as the weights have rows: 6.4 and
// 5.2 us for that token.  An expert that two assignments share is read twice, mostly
// from the caches; few_rows() says when that is worth it.
//
// Dot products of four bytes at a time (v_dot4_i32_i8) give each lane 8 exact partial
// sums, added over the wave by halving exchanges: each step gives one half of the
// sums away and receives the other lanes' part of the half that is kept.  Sums are
// integers and the scaling is that of the tiles, so the bits are the same.
//
// The assignments are not sorted: row f of act and y belongs to assignment f, whose
// expert is top_k_index[f].  down quantises its act row on the way (every wave for
// itself: the row's maximum, then its values as they are multiplied), which costs
// less than a launch.
#include "row_quantizer.h"

namespace moe {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;  // waves of a workgroup, each with its own 8 rows of B

struct FewArgs {
  const void* A;           // gate_up: hidden_q; down: act rows in the layer's dtype
  const float* a_scale;    // gate_up: hidden_scale
  const int8_t* B;
  const float* b_scale;
  void* C;                 // [rows][ncols] in the layer's dtype
  const int32_t* idx;
  int32_t* dst_row;        // gate_up
  int32_t* dev_error;
  int rows, E, k, K, ncols;
};

template <bool kGateUp, bool kBf16>
__global__ void __launch_bounds__(64 * kWaves) few_rows_i8(FewArgs a) {
  constexpr int kCols = kGateUp ? 4 : 8;  // output columns of a wave
  constexpr int kEl = kVecEl<kBf16>, kVecs = 16 / kEl;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = a.ncols / (kWaves * kCols);
  const int f = blockIdx.x / groups;
  const int c0 = ((blockIdx.x % groups) * kWaves + wave) * kCols;
  if (kGateUp && blockIdx.x == 0 && wave == 0) {
    // at most 64 assignments, one per lane
    const int id = lane < a.rows ? a.idx[lane] : 0;
    const bool bad = lane < a.rows && (id < 0 || id >= a.E);
    if (lane < a.rows) a.dst_row[lane] = bad ? -1 : lane;
    const int dropped = __popcll(__ballot(bad));
    if (lane == 0) *a.dev_error = dropped;
  }
  const int e = __builtin_amdgcn_readfirstlane(a.idx[f]);
  if (e < 0 || e >= a.E) return;
  const int K = a.K;
  const int brows = kGateUp ? 2 * a.ncols : a.ncols;
  const int8_t* bp[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const int row = kGateUp ? (c >> 2) * a.ncols + c0 + (c & 3) : c0 + c;
    bp[c] = a.B + ((int64_t)e * brows + row) * K;
  }
  // after the reduction lane l holds the sum of row l >> 3 of the wave's 8
  const int my = lane >> 3;
  const int my_row = kGateUp ? (my >> 2) * a.ncols + c0 + (my & 3) : c0 + my;
  const float cs = a.b_scale[(int64_t)e * brows + my_row];
  float rs;
  const int8_t* x8 = nullptr;
  const u32x4* act = nullptr;
  RowQuantizer<kBf16> quant(0);
  if constexpr (kGateUp) {
    const int t = f / a.k;
    rs = a.a_scale[t];
    x8 = (const int8_t*)a.A + (int64_t)t * K;
  } else {
    act = (const u32x4*)a.A + (int64_t)f * (K / kEl);
    uint32_t big = 0;
    for (int k = lane * kEl; k < K; k += 64 * kEl) {
      float v[kEl];
      unpack<kBf16>(act[k / kEl], v);
      big = max_magnitude<kEl>(v, big);
    }
    quant = RowQuantizer<kBf16>(wave_max(big));
    rs = quant.scale;
  }
  int acc[8] = {};
#pragma unroll 2
  for (int k = lane * 16; k < K; k += 1024) {
    i32x4 w[8], x;
#pragma unroll
    for (int c = 0; c < 8; ++c) w[c] = __builtin_nontemporal_load((const i32x4*)(bp[c] + k));
    if constexpr (kGateUp) {
      x = *(const i32x4*)(x8 + k);
    } else {
      float v[16];
#pragma unroll
      for (int i = 0; i < kVecs; ++i) unpack<kBf16>(act[k / kEl + i], v + i * kEl);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[q] = (int)quant.word(v + 4 * q);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[c] = __builtin_amdgcn_sdot4(w[c][q], x[q], acc[c], false);
  }
#pragma unroll
  for (int half = 4, mask = 32; half > 0; half >>= 1, mask >>= 1) {
    const bool up = lane & mask;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const int give = up ? acc[i] : acc[i + half], keep = up ? acc[i + half] : acc[i];
      acc[i] = keep + __shfl_xor(give, mask);
    }
  }
#pragma unroll
  for (int mask = 4; mask > 0; mask >>= 1) acc[0] += __shfl_xor(acc[0], mask);
  float o = (float)acc[0] * rs * cs;
  // gate sums are in lanes 0..31, the up sums of the same columns in lanes 32..63
  if constexpr (kGateUp) o = swiglu(o, __shfl_xor(o, 32));
  if (lane & 7 || (kGateUp && lane >= 32)) return;
  const int64_t at = (int64_t)f * a.ncols + c0 + my;
  if constexpr (kBf16)
    ((__bf16*)a.C)[at] = (__bf16)o;
  else
    ((float*)a.C)[at] = o;
}

template <bool kGateUp>
hipError_t launch(const Shape& s, FewArgs a, hipStream_t st) {
  a.rows = (int)s.A;
  a.E = s.E;
  a.k = s.k;
  a.K = kGateUp ? s.H : s.I;
  a.ncols = kGateUp ? s.I : s.H;
  // ncols is a multiple of 64: whole workgroups of 16 (gate_up) or 32 columns
  const dim3 grid((unsigned)(a.rows * (a.ncols / (kWaves * (kGateUp ? 4 : 8)))));
  if (s.dtype == MOE_BF16)
    hipLaunchKernelGGL((few_rows_i8<kGateUp, true>), grid, dim3(64 * kWaves), 0, st, a);
  else
    hipLaunchKernelGGL((few_rows_i8<kGateUp, false>), grid, dim3(64 * kWaves), 0, st, a);
  return hipGetLastError();
}

}  // namespace

// At most 32 assignments, and few enough that two seldom share an expert (one
// token's are distinct).  Weight reads of gate_up + down, tiles against this form:
// E = 64, H = 2048, I = 1024, k = 4: 32 assignments 36.0 / 29.9 us, 64: 48.8 / 47.7;
// E = 256, H = 7168, I = 2048, k = 8: 8: 83.9 / 62.0, 32: 243.7 / 208.3, 64: 400 / 397,
// 128: 680 / 760.
bool few_rows(const Shape& s) {
  return s.A > 0 && s.A <= 32 && (s.T == 1 || 2 * s.A <= s.E);
}

hipError_t launch_few_gate_up_i8(const Shape& s, const int8_t* hidden_q, const float* hidden_scale,
                                 const int32_t* top_k_index, const int8_t* w, const float* w_scale,
                                 void* act, int32_t* dst_row, int32_t* dev_error, hipStream_t st) {
  FewArgs a{};
  a.A = hidden_q;
  a.a_scale = hidden_scale;
  a.B = w;
  a.b_scale = w_scale;
  a.C = act;
  a.idx = top_k_index;
  a.dst_row = dst_row;
  a.dev_error = dev_error;
  return launch<true>(s, a, st);
}

hipError_t launch_few_down_i8(const Shape& s, const void* act, const int32_t* top_k_index,
                              const int8_t* w, const float* w_scale, void* y, hipStream_t st) {
  FewArgs a{};
  a.A = act;
  a.B = w;
  a.b_scale = w_scale;
  a.C = y;
  a.idx = top_k_index;
  return launch<false>(s, a, st);
}

}  // namespace moe
