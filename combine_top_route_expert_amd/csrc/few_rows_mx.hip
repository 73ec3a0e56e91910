// The layer with 4-bit experts for a few assignments (a decoded token, or a handful), in two
// launches; nothing is sorted, row f of act belongs to assignment f.
//   few_gate_up  a workgroup takes 32 columns of act of one assignment
//   few_down     a workgroup takes 32 output columns of one token, over all its slots
// A wave multiplies 32 weight rows by 256 columns at a time (a unit: four kilobytes and
// their scales, from one or two places), all of whose loads it issues at once; the units of
// K, and in few_down those of the slots, are dealt to the waves.  The weights are converted to
// bf16 (exactly, subnormal ones too) and multiplied by matrix instructions of which one row, or two, are filled: only the lanes that hold those load any of x, where
// a dot product of a lane's 32 columns needs the whole row's in every lane (with v_dot2_f32_bf16
// 19.6 us for the token below instead of 18.9, 187 instead of 181 for four of them with 8 experts
// of H = 7168, I = 2048; with single multiply-adds 20 and 195).  act is kept as two bf16
// numbers, value and rest, off by 2^-16, which few_down multiplies as two rows; y stays in fp32,
// and out is rounded once.
//
// One token with 4 experts of H = 2048, I = 1024: few_gate_up 5.4 us, few_down 6.7, of which the
// 13 MB of weights are 3: latency bounds both.  16 assignments of H = 7168, I = 2048: 51 us and
// 36, 4.9 and 3.5 TB/s.  Workgroups of 4 waves cost 1 to 10% more.
//
// Sums are in fp32: over a wave's units column by column (few_down: over a unit's), then over
// the waves (few_down: the slots' units and then the waves), in that order whatever runs
// beside.
#include "fp4_operand.h"
#include "row_quantizer.h"

namespace moe {

namespace {

constexpr int kUnit = 4;   // blocks
constexpr int kWaves = 8;  // waves of a workgroup
constexpr int kRows = 32;  // weight rows of a block

struct FewMxArgs {
  const void* x;  // gate_up: hidden states [T][H] bf16; down: act [T*k][I / 32][2][32] bf16
  const char *b, *bs;
  int64_t b_expert, bs_expert;
  const int32_t* idx;
  const float* top_k_weights;  // down
  int32_t* dev_error;          // gate_up
  void* out;                   // gate_up: act; down: out [T][H] bf16
  int rows, E, k, ncols;       // assignments; columns of out
  int blocks, quads;           // 64-column blocks of K, scale dwords of a weight row
  int up;                      // gate_up: row blocks from a gate row to its up row
};

// One unit of N weight row blocks: rows rb[n] of expert e, columns 256 u .. (the last unit may
// have fewer blocks), with kParts rows at x, 64 bytes of each in turn.
template <int N, int kParts>
__device__ __forceinline__ void unit_mma(const FewMxArgs& a, int e, const int (&rb)[N], int u,
                                         const char* x, int lane, f32x16 (&acc)[N]) {
  const int r = lane & 31, half = lane >> 5, live = a.blocks - kUnit * u;
  u32x4 w[kUnit][N], v[kUnit][4];
  uint32_t s[N];
#pragma unroll
  for (int n = 0; n < N; ++n)
    s[n] = *(const uint32_t*)(a.bs + e * a.bs_expert +
                              ((int64_t)rb[n] * a.quads + u) * kFp4ScaleBytes + lane * 4);
#pragma unroll
  for (int k = 0; k < kUnit; ++k) {
    if (k >= live) break;
#pragma unroll
    for (int n = 0; n < N; ++n)
      w[k][n] = __builtin_nontemporal_load(
          (const u32x4*)(a.b + e * a.b_expert +
                         ((int64_t)rb[n] * a.blocks + kUnit * u + k) * kFp4BlockBytes) +
          lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (the rows of the other lanes may hold anything: their sums are not used)
      asm volatile("" : "=v"(v[k][i]));
      if (r < kParts) v[k][i] = ((const u32x4*)x)[((2 * (kUnit * u + k) + half) * kParts + r) * 4 + i];
    }
  }
#pragma unroll
  for (int k = 0; k < kUnit; ++k) {
    if (k >= live) break;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int n = 0; n < N; ++n)
        acc[n] = MmaBf16::mma(unpack_fp4(w[k][n][i], s[n] >> (8 * k) & 0xffu),
                              __builtin_bit_cast(bf16x8, v[k][i]), acc[n]);
  }
}

// The 32 sums of a wave for its first row: lane 32 h holds those of weight rows 8 g + 4 h + ..
__device__ __forceinline__ void put_sums(float* to, const f32x16& acc, int half) {
#pragma unroll
  for (int g = 0; g < 4; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i) to[8 * g + 4 * half + i] = acc[4 * g + i];
}

__global__ void __launch_bounds__(64 * kWaves) few_gate_up_mx(FewMxArgs a) {
  __shared__ float sums[kWaves][2][kRows];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = a.ncols / kRows;
  const int f = blockIdx.x / groups, g = blockIdx.x % groups;
  if (blockIdx.x == 0 && wave == 0) {
    // at most 32 assignments, one per lane
    const int id = lane < a.rows ? a.idx[lane] : 0;
    const int dropped = __popcll(__ballot(lane < a.rows && (id < 0 || id >= a.E)));
    if (lane == 0) *a.dev_error = dropped;
  }
  const int e = __builtin_amdgcn_readfirstlane(a.idx[f]);
  if (e < 0 || e >= a.E) return;
  const char* x = (const char*)a.x + (int64_t)(f / a.k) * a.blocks * 128;
  const int rb[2] = {g, g + a.up};
  f32x16 acc[2] = {f32x16{}, f32x16{}};
  for (int u = wave; u < a.quads; u += kWaves) unit_mma<2, 1>(a, e, rb, u, x, lane, acc);
#pragma unroll
  for (int n = 0; n < 2; ++n)
    if ((lane & 31) == 0) put_sums(sums[wave][n], acc[n], lane >> 5);
  __syncthreads();
  if (threadIdx.x >= kRows) return;
  float gate = 0.0f, up = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    gate += sums[w][0][lane];
    up += sums[w][1][lane];
  }
  const float act = swiglu<true>(gate, up);
  const __bf16 hi = (__bf16)act;
  // (an infinity has no rest: inf - inf would make NaN of it)
  const __bf16 lo = __builtin_fabsf((float)hi) < INFINITY ? (__bf16)(act - (float)hi) : (__bf16)0.0f;
  __bf16* to = (__bf16*)a.out + ((int64_t)f * groups + g) * 2 * kRows + lane;
  to[0] = hi;
  to[kRows] = lo;
}

__global__ void __launch_bounds__(64 * kWaves) few_down_mx(FewMxArgs a) {
  __shared__ float sums[kWaves][kRows];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = a.ncols / kRows;
  const int t = blockIdx.x / groups, g = blockIdx.x % groups;
  const int rb[1] = {g};
  f32x16 out{};
  for (int i = wave; i < a.k * a.quads; i += kWaves) {
    const int j = i / a.quads, u = i % a.quads;
    const int64_t f = (int64_t)t * a.k + j;
    const int e = __builtin_amdgcn_readfirstlane(a.idx[f]);
    if (e < 0 || e >= a.E) continue;
    f32x16 acc[1] = {f32x16{}};
    unit_mma<1, 2>(a, e, rb, u, (const char*)a.x + f * a.blocks * 256, lane, acc);
    const float weight = a.top_k_weights[f];
#pragma unroll
    for (int q = 0; q < 16; ++q) out[q] = __builtin_fmaf(weight, acc[0][q], out[q]);
  }
  // lane 1's row is the rest of lane 0's
#pragma unroll
  for (int q = 0; q < 16; ++q) out[q] += __shfl_xor(out[q], 1);
  if ((lane & 31) == 0) put_sums(sums[wave], out, lane >> 5);
  __syncthreads();
  if (threadIdx.x >= kRows) return;
  float o = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) o += sums[w][lane];
  ((__bf16*)a.out)[(int64_t)t * a.ncols + g * kRows + lane] = (__bf16)o;
}

}  // namespace

// At most 32 assignments, and no more than there are experts (those of one token are distinct
// in any case): an expert that several assignments share is read for each of them.  And at most
// 512 MB of weights to read, counted for every assignment: beyond that what the sorted form's
// launches cost is less than what its loads gain.  Whole layer in us, sorted streaming tiles / this
// form:
//   E = 64, H = 2048, I = 1024, k = 4 (3.3 MB an expert): 4 assignments 40 / 19, 16: 44 / 26, 32: 48 / 38
//   E = 128, H = 4096, I = 1536, k = 8 (10 MB): 32 assignments 93 / 91
//   E = 160, H = 5120, I = 2048, k = 8 (17 MB): 24: 113 / 107, 32: 121 / 143
//   E = 256, H = 7168, I = 2048, k = 8 (23 MB): 8: 90 / 59, 16: 107 / 95, 24: 142 / 143, 32: 166 / 181
//   E = 64, H = 8192, I = 4096 (53 MB): 8: 123 / 114, 12: 166 / 162
//   E = 8, H = 4096, I = 2048, k = 2:  2: 60 / 24;  E = 16, H = I = 2880, k = 4:  16: 74 / 68, 32: 75 / 114
bool few_rows_mx(const Shape& s) {
  const double bytes = 3.0 * s.H * s.I * 17 / 32 * s.A;
  return s.A > 0 && s.A <= 32 && (s.T == 1 || s.A <= s.E) && bytes <= 0x1p29;
}

hipError_t launch_few_mx(const Shape& s, const void* hidden_states, const int32_t* top_k_index,
                         const float* top_k_weights, const uint8_t* w_gate_up_q,
                         const uint8_t* w_gate_up_scale, const uint8_t* w_down_q,
                         const uint8_t* w_down_scale, void* act, void* out, int32_t* dev_error,
                         hipStream_t st) {
  FewMxArgs g{};
  g.idx = top_k_index;
  g.rows = (int)s.A;
  g.E = s.E;
  g.k = s.k;
  FewMxArgs d = g;
  g.x = hidden_states;
  g.b = (const char*)w_gate_up_q;
  g.bs = (const char*)w_gate_up_scale;
  g.b_expert = (int64_t)2 * s.I * s.H / 2;
  g.bs_expert = fp4_scale_bytes(2 * (int64_t)s.I, s.H);
  g.dev_error = dev_error;
  g.out = act;
  g.ncols = s.I;
  g.blocks = s.H / kFp4BlockCols;
  g.quads = (int)fp4_scale_quads(s.H);
  g.up = s.I / kFp4BlockRows;
  d.x = act;
  d.b = (const char*)w_down_q;
  d.bs = (const char*)w_down_scale;
  d.b_expert = (int64_t)s.H * s.I / 2;
  d.bs_expert = fp4_scale_bytes(s.H, s.I);
  d.top_k_weights = top_k_weights;
  d.out = out;
  d.ncols = s.H;
  d.blocks = s.I / kFp4BlockCols;
  d.quads = (int)fp4_scale_quads(s.I);
  // (few workgroups: at most 512 MB of weights, of which each reads a kilobyte or more)
  const int64_t gate = s.A * (s.I / kRows), down = (int64_t)s.T * (s.H / kRows);
  hipLaunchKernelGGL(few_gate_up_mx, dim3((unsigned)gate), dim3(64 * kWaves), 0, st, g);
  hipLaunchKernelGGL(few_down_mx, dim3((unsigned)down), dim3(64 * kWaves), 0, st, d);
  return hipGetLastError();
}

}  // namespace moe
