// Layer norm of the layer's input rows (forward, backward, and a form that also
// quantises its rows to 8-bit integers) and the row quantiser by itself.
//
//   s = rd(x + residual)           (or x), rd: rounding to the layer's dtype
//   y = (s - mean) * rstd * weight + bias,  mean and rstd over the row's H values
//   backward, with xh = (s - mean) rstd and h = grad_y weight:
//     grad_x = rstd (h - mean_H(h) - xh mean_H(h xh)) [+ grad_sum]
//     grad_weight = sum_t grad_y xh,  grad_bias = sum_t grad_y
//   quantise: a = max |row|, scale = a / 127, q = rne(127 row / a)
//
// All of it is bound by memory: a row is read once, held in registers as fp32
// while its statistics are reduced, and written once.  The variance is the
// mean of the squared distances from the mean (a second pass over registers).
// A common offset costs no precision, since the mean is that of an exact or
// nearly exact sum: bf16 values of one binade sum to 22 bits at most and fp32
// holds them; fp32 rows are summed in fp64 and their mean is subtracted as two
// floats (one fp32 mean: values around 1000 that spread by 0.01 had y off by 0.01;
// at most 1% more time, 6.4 -> 6.5 us for 1000 x 2052).  fp64 for bf16
// rows too: one token 4.0 -> 4.15 us, 16384 x 8192 124 -> 129 us, and nothing gained.
//
// A row takes 64 to 1024 threads of at most 16 values each (up to 1024 values: a
// wave's row, four to a workgroup, no barrier).  Threads take 16-byte vectors round
// robin, so every load and store of a wave is one contiguous kilobyte.  32 values
// per thread: 16384 x 2048 with residual 57.7 against 54.3 us, 4096 x 7168
// quantising 59.9 against 55.5 us, one token 5.5 against 4.4 us; eight: the same
// within 1% but 65.6 us quantising.  What one pass reads or writes once is
// streamed non-temporally: 16384 x 2048 fp32 with residual 103.6 -> 92.9 us, 16384 x
// 8192 bf16 127 -> 123.5 us (4.35 TB/s), though rows that partly stay in the caches
// lose up to 4% (16384 x 2048 bf16 with residual 50.4 -> 52 us, 5.2 TB/s).
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "row_quantizer.h"

namespace moe {

namespace {

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

// Reductions over the THREADS threads of a row; `red` is a slot of THREADS / 64
// values used by no other reduction that a barrier does not separate.  Every
// thread gets the same bits.
template <int THREADS, class T>
__device__ __forceinline__ T row_sum(T v, T* red) {
  v = wave_sum(v);
  if constexpr (THREADS > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) v += red[w];
  }
  return v;
}

template <int THREADS>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
  v = wave_max(v);
  if constexpr (THREADS > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < THREADS / 64; ++w) v = red[w] > v ? red[w] : v;
  }
  return v;
}

// kEl consecutive floats of a [H] parameter, or `none` where there is none.
template <int kEl>
__device__ __forceinline__ void load_param(const float* p, int64_t v, float none, float* f) {
#pragma unroll
  for (int i = 0; i < kEl; ++i) f[i] = p ? p[v * kEl + i] : none;
}

constexpr int kRowValues = 16;  // values of a row per thread

// A row: THREADS threads of kRowValues values each.
template <int THREADS>
struct RowOf {
  static constexpr int kPerGroup = THREADS == 64 ? 4 : 1;
  static constexpr int kGroup = THREADS == 64 ? 256 : THREADS;  // workgroup size
  static __device__ __forceinline__ int tid() {
    return THREADS == 64 ? (int)threadIdx.x & 63 : (int)threadIdx.x;
  }
  static __device__ __forceinline__ int64_t row() {
    return THREADS == 64 ? (int64_t)blockIdx.x * kPerGroup + (threadIdx.x >> 6)
                         : (int64_t)blockIdx.x;
  }
  static dim3 grid(int64_t rows) { return dim3((unsigned)((rows + kPerGroup - 1) / kPerGroup)); }
};

// Rows of one launch: a launch holds fewer than 2^32 threads, and a row takes
// at most 1024 of them.  More rows go in several launches.
constexpr int64_t kRowsPerLaunch = 1 << 21;

template <bool kBf16, int THREADS, bool kQuant>
__global__ void __launch_bounds__(RowOf<THREADS>::kGroup)
norm_rows(NormIO io, int64_t row0, int64_t rows, int nvec) {
  constexpr int kEl = kVecEl<kBf16>, VPT = kRowValues / kEl, NW = THREADS / 64;
  const int64_t row = row0 + RowOf<THREADS>::row();
  if (row >= rows) return;
  typedef std::conditional_t<kBf16, float, double> sum_t;
  __shared__ sum_t red_total[NW];
  __shared__ float red[2][NW];
  const int tid = RowOf<THREADS>::tid();
  const u32x4* x = (const u32x4*)io.x + row * nvec;
  u32x4 xv[VPT], rv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (i * THREADS + tid < nvec) xv[i] = __builtin_nontemporal_load(&x[i * THREADS + tid]);
  if (io.residual) {
    const u32x4* r = (const u32x4*)io.residual + row * nvec;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (i * THREADS + tid < nvec) rv[i] = __builtin_nontemporal_load(&r[i * THREADS + tid]);
  }
  float f[VPT][kEl];
  sum_t total = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * THREADS + tid;
    if (v >= nvec) continue;
    unpack<kBf16>(xv[i], f[i]);
    if (io.residual) {
      float g[kEl];
      unpack<kBf16>(rv[i], g);
#pragma unroll
      for (int e = 0; e < kEl; ++e) f[i][e] += g[e];
      // the sum is what later layers read: its statistics are those of the
      // rounded values
      const u32x4 p = pack<kBf16>(f[i]);
      __builtin_nontemporal_store(p, &((u32x4*)io.sum)[row * nvec + v]);
      unpack<kBf16>(p, f[i]);
    }
#pragma unroll
    for (int e = 0; e < kEl; ++e) total += (sum_t)f[i][e];
  }
  const float h = (float)(nvec * kEl);
  const sum_t sum = row_sum<THREADS>(total, red_total);
  sum_t exact = sum / (sum_t)h;
  // a sum past fp32's range has no mean in it: NaN, as for a row with an infinity
  if constexpr (!kBf16)
    if (!(fabs(sum) <= (double)FLT_MAX)) exact = __builtin_nan("");
  const float mean = (float)exact, mean_low = (float)(exact - (sum_t)mean);
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (i * THREADS + tid >= nvec) continue;
#pragma unroll
    for (int e = 0; e < kEl; ++e) {
      f[i][e] -= mean;
      if constexpr (!kBf16) f[i][e] -= mean_low;
      sq = __builtin_fmaf(f[i][e], f[i][e], sq);
    }
  }
  // squares past fp32's range would leave rstd 0 and y the bias: NaN instead, as above
  const float var = row_sum<THREADS>(sq, red[0]) / h + io.eps;
  const float rstd = var < __builtin_inff() ? 1.0f / sqrtf(var) : __builtin_nanf("");
  if (tid == 0) {
    if (io.mean) io.mean[row] = mean;
    if (io.rstd) io.rstd[row] = rstd;
  }
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * THREADS + tid;
    if (v >= nvec) continue;
    float w[kEl], b[kEl];
    load_param<kEl>(io.weight, v, 1.0f, w);
    load_param<kEl>(io.bias, v, 0.0f, b);
#pragma unroll
    for (int e = 0; e < kEl; ++e) f[i][e] = __builtin_fmaf(f[i][e] * rstd, w[e], b[e]);
    const u32x4 p = pack<kBf16>(f[i]);
    if (!kQuant || io.y) __builtin_nontemporal_store(p, &((u32x4*)io.y)[row * nvec + v]);
    if constexpr (kQuant) {
      // quantised from the rounded y: the same bits as the two calls one after
      // the other
      unpack<kBf16>(p, f[i]);
      big = max_magnitude<kEl>(f[i], big);
    }
  }
  if constexpr (kQuant) {
    const RowQuantizer<kBf16> quant(row_max<THREADS>(big, (uint32_t*)red[1]));
    if (tid == 0) io.scale[row] = quant.scale;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * THREADS + tid;
      if (v < nvec) quant.store(f[i], io.q, row * nvec + v);
    }
  }
}

// EPT = 0: rows wider than the registers hold; read twice (the second time
// mostly from the caches).
template <bool kBf16, int THREADS, int EPT>
__global__ void __launch_bounds__(RowOf<THREADS>::kGroup)
quantize_rows(const u32x4* __restrict__ x, int8_t* __restrict__ q, float* __restrict__ scale,
              int64_t row0, int64_t rows, int64_t nvec, const int32_t* __restrict__ valid0,
              const int32_t* __restrict__ valid1) {
  constexpr int kEl = kVecEl<kBf16>, VPT = EPT / kEl, NW = THREADS / 64;
  const int64_t row = row0 + RowOf<THREADS>::row();
  if (row >= rows) return;
  if (valid0 && row >= (int64_t)*valid0 + (valid1 ? *valid1 : 0)) return;
  __shared__ uint32_t red[NW];
  const int tid = RowOf<THREADS>::tid();
  x += row * nvec;
  uint32_t big = 0;
  if constexpr (EPT > 0) {
    u32x4 xv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (i * THREADS + tid < nvec) xv[i] = x[i * THREADS + tid];
    float f[VPT][kEl];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (i * THREADS + tid >= nvec) continue;
      unpack<kBf16>(xv[i], f[i]);
      big = max_magnitude<kEl>(f[i], big);
    }
    const RowQuantizer<kBf16> quant(row_max<THREADS>(big, red));
    if (tid == 0) scale[row] = quant.scale;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * THREADS + tid;
      if (v < nvec) quant.store(f[i], q, row * nvec + v);
    }
  } else {
    float f[kEl];
    for (int64_t v = tid; v < nvec; v += THREADS) {
      unpack<kBf16>(x[v], f);
      big = max_magnitude<kEl>(f, big);
    }
    const RowQuantizer<kBf16> quant(row_max<THREADS>(big, red));
    if (tid == 0) scale[row] = quant.scale;
    for (int64_t v = tid; v < nvec; v += THREADS) {
      unpack<kBf16>(x[v], f);
      quant.store(f, q, row * nvec + v);
    }
  }
}

// Backward.  A workgroup of 1024 threads holds kPar = 1024 / THREADS rows at a
// time, rows b kPar + p, p < kPar, then those gridDim kPar further; bf16 rows of up
// to 8192 values are loaded while those before them are reduced (where the next
// row fits the 128 registers of a thread).  A thread keeps its columns' sums of
// grad_y xh and grad_y in registers over all its rows; the kPar groups' sums are
// joined in LDS in order and written once, as row b of the partials
// ([workgroups][2][H]).  norm_grad_reduce adds those rows in a fixed order: no
// atomics, the same bits every time.  4096 x 7168 with grad_sum: 46 + 5 us, 4.7 TB/s;
// with 512 workgroups of one row each, no loads ahead and partials to match 63 + 12.
constexpr int kGradThreads = 1024;
constexpr int kGradGroups = 256;  // one workgroup per CU: the fewest partials

template <bool kBf16, int THREADS>
__global__ void __launch_bounds__(kGradThreads) norm_grad_rows(NormGradIO io, int T, int nvec) {
  constexpr int kEl = kVecEl<kBf16>, VPT = kRowValues / kEl, NW = THREADS / 64;
  constexpr int kPar = kGradThreads / THREADS;
  constexpr bool kAhead = kBf16 && THREADS < 1024;
  __shared__ float red[2][kPar][2][NW];
  const int tid = threadIdx.x % THREADS;
  const int grp = __builtin_amdgcn_readfirstlane(threadIdx.x / THREADS);
  const float inv_h = 1.0f / (float)(nvec * kEl);
  float w[VPT][kEl], dw[VPT][kEl], db[VPT][kEl];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * THREADS + tid;
#pragma unroll
    for (int e = 0; e < kEl; ++e) w[i][e] = dw[i][e] = db[i][e] = 0.0f;
    if (v < nvec) load_param<kEl>(io.weight, v, 1.0f, w[i]);
  }
  const int64_t stride = (int64_t)gridDim.x * kPar;
  u32x4 gv[VPT] = {}, xv[VPT] = {};
  float mean = 0.0f, rstd = 0.0f;
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {
    if (row >= T) return;
    const u32x4* gy = (const u32x4*)io.grad_y + row * nvec;
    const u32x4* x = (const u32x4*)io.x + row * nvec;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (i * THREADS + tid < nvec) {
        gv[i] = __builtin_nontemporal_load(&gy[i * THREADS + tid]);
        xv[i] = __builtin_nontemporal_load(&x[i * THREADS + tid]);
      }
    mean = io.mean[row];
    rstd = io.rstd[row];
  };
  int64_t row = (int64_t)blockIdx.x * kPar + grp;
  if constexpr (kAhead) fetch(row);
  // every group takes part in every barrier: the first group's rows end last
  int par = 0;
  for (int64_t first = (int64_t)blockIdx.x * kPar; first < T; first += stride, row += stride) {
    if constexpr (!kAhead) fetch(row);
    u32x4 g0[VPT], x0[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      g0[i] = gv[i];
      x0[i] = xv[i];
    }
    const float m = mean, rs = rstd;
    const bool live = row < T;
    if constexpr (kAhead) fetch(row + stride);
    float s1 = 0.0f, s2 = 0.0f;
    if (live) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (i * THREADS + tid >= nvec) continue;
        float g[kEl], s[kEl];
        unpack<kBf16>(g0[i], g);
        unpack<kBf16>(x0[i], s);
#pragma unroll
        for (int e = 0; e < kEl; ++e) {
          const float xh = (s[e] - m) * rs, h = g[e] * w[i][e];
          s1 += h;
          s2 = __builtin_fmaf(h, xh, s2);
          dw[i][e] = __builtin_fmaf(g[e], xh, dw[i][e]);
          db[i][e] += g[e];
        }
      }
    }
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if constexpr (THREADS > 64) {
      // two slots in turn: a wave can be one row ahead of the slowest, not two
      if ((tid & 63) == 0) {
        red[par][grp][0][tid >> 6] = s1;
        red[par][grp][1][tid >> 6] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.0f;
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        s1 += red[par][grp][0][k];
        s2 += red[par][grp][1][k];
      }
      par ^= 1;
    }
    if (!live) continue;
    const float m1 = s1 * inv_h, m2 = s2 * inv_h;
    // (loaded here: any earlier it cost the registers of the next row, 46 -> 53 us)
    const u32x4* gs = io.grad_sum ? (const u32x4*)io.grad_sum + row * nvec : nullptr;
    u32x4* gx = (u32x4*)io.grad_x + row * nvec;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * THREADS + tid;
      if (v >= nvec) continue;
      float g[kEl], s[kEl], o[kEl];
      unpack<kBf16>(g0[i], g);
      unpack<kBf16>(x0[i], s);
      if (gs)
        unpack<kBf16>(__builtin_nontemporal_load(&gs[v]), o);
      else
#pragma unroll
        for (int e = 0; e < kEl; ++e) o[e] = 0.0f;
#pragma unroll
      for (int e = 0; e < kEl; ++e) {
        const float xh = (s[e] - m) * rs, h = g[e] * w[i][e];
        o[e] = __builtin_fmaf(rs, __builtin_fmaf(-xh, m2, h - m1), o[e]);
      }
      __builtin_nontemporal_store(pack<kBf16>(o), &gx[v]);
    }
  }
  if (!io.partials) return;
  const int H = nvec * kEl;
  // one workgroup alone has the whole sums
  float* to[2] = {io.grad_weight, io.grad_bias};
  if (gridDim.x > 1) {
    to[0] = io.partials + (int64_t)blockIdx.x * 2 * H;
    to[1] = to[0] + H;
  }
  if constexpr (kPar == 1) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * THREADS + tid;
      if (v >= nvec) continue;
#pragma unroll
      for (int e = 0; e < kEl; ++e) {
        if (to[0]) to[0][v * kEl + e] = dw[i][e];
        if (to[1]) to[1][v * kEl + e] = db[i][e];
      }
    }
  } else {
    __shared__ float cols[kGradThreads * kRowValues];  // [kPar][H] of one of the two sums
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      if (which) __syncthreads();
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * THREADS + tid;
        if (v >= nvec) continue;
#pragma unroll
        for (int e = 0; e < kEl; ++e)
          cols[grp * H + v * kEl + e] = which ? db[i][e] : dw[i][e];
      }
      __syncthreads();
      for (int c = threadIdx.x; c < H; c += kGradThreads) {
        float sum = cols[c];
#pragma unroll
        for (int k = 1; k < kPar; ++k) sum += cols[k * H + c];
        if (to[which]) to[which][c] = sum;
      }
    }
  }
}

// grad_weight / grad_bias: the column sums of the partials' n rows.  A
// workgroup takes 64 columns (16 threads of four) with its rows dealt to 16
// groups of threads, whose sums are joined in order.
__global__ void __launch_bounds__(256)
norm_grad_reduce(const float* __restrict__ part, int n, int H, float* __restrict__ grad_weight,
                 float* __restrict__ grad_bias) {
  __shared__ float4 sums[16][16];
  float* out = blockIdx.y ? grad_bias : grad_weight;
  if (!out) return;
  const int cx = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int c = blockIdx.x * 64 + cx * 4;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < H)
#pragma unroll 4
    for (int r = g; r < n; r += 16) {
      const float4 p = *(const float4*)(part + ((int64_t)r * 2 + blockIdx.y) * H + c);
      a.x += p.x;
      a.y += p.y;
      a.z += p.z;
      a.w += p.w;
    }
  sums[g][cx] = a;
  __syncthreads();
  if (g != 0 || c >= H) return;
  for (int k = 1; k < 16; ++k) {
    const float4 p = sums[k][cx];
    a.x += p.x;
    a.y += p.y;
    a.z += p.z;
    a.w += p.w;
  }
  *(float4*)(out + c) = a;
}

// Threads of a row, by its width.
int row_threads(int64_t width) {
  int t = 64;
  while (t * kRowValues < width) t *= 2;
  return t;
}

// Workgroups of norm_grad_rows.  Two rows after one another in a single workgroup
// take less than a second launch to join two of them: 4 rows of 7168 values 9.3
// against 10.8 us a call (9.3 / 9.4 in a graph), 32 rows of 324 8.3 / 10.8 (5.8 / 6.6);
// three do not (6 rows of 7168: 11.8 against 10.8).
int norm_grad_groups(const Shape& s) {
  const int par = kGradThreads / row_threads(s.H);
  if (s.T <= 2 * par) return 1;
  return (int)std::min<int64_t>(((int64_t)s.T + par - 1) / par, kGradGroups);
}

template <bool kBf16, bool kQuant>
hipError_t norm_launch(const Shape& s, const NormIO& io, hipStream_t st) {
  const int nvec = s.H / kVecEl<kBf16>;
  for (int64_t r0 = 0; r0 < s.T; r0 += kRowsPerLaunch) {
    const int64_t end = std::min<int64_t>(s.T, r0 + kRowsPerLaunch);
#define MOE_NORM(THREADS)                                                                   \
  hipLaunchKernelGGL((norm_rows<kBf16, THREADS, kQuant>), RowOf<THREADS>::grid(end - r0),   \
                     dim3(RowOf<THREADS>::kGroup), 0, st, io, r0, end, nvec)
    switch (row_threads(s.H)) {
      case 64: MOE_NORM(64); break;
      case 128: MOE_NORM(128); break;
      case 256: MOE_NORM(256); break;
      case 512: MOE_NORM(512); break;
      default: MOE_NORM(1024); break;
    }
#undef MOE_NORM
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool kBf16>
hipError_t norm_grad_launch(const Shape& s, const NormGradIO& io, hipStream_t st) {
  const int nvec = s.H / kVecEl<kBf16>, groups = norm_grad_groups(s);
  const int threads = row_threads(s.H);
#define MOE_NORM_GRAD(THREADS)                                                          \
  hipLaunchKernelGGL((norm_grad_rows<kBf16, THREADS>), dim3((unsigned)groups),          \
                     dim3(kGradThreads), 0, st, io, s.T, nvec)
  switch (threads) {
    case 64: MOE_NORM_GRAD(64); break;
    case 128: MOE_NORM_GRAD(128); break;
    case 256: MOE_NORM_GRAD(256); break;
    case 512: MOE_NORM_GRAD(512); break;
    default: MOE_NORM_GRAD(1024); break;
  }
#undef MOE_NORM_GRAD
  return hipGetLastError();
}

template <bool kBf16>
hipError_t quantize_launch(int64_t rows, int64_t cols, const void* x, int8_t* q, float* scale,
                           const int32_t* valid0, const int32_t* valid1, hipStream_t st) {
  const int64_t nvec = cols / kVecEl<kBf16>;
  for (int64_t r0 = 0; r0 < rows; r0 += kRowsPerLaunch) {
    const int64_t end = std::min(rows, r0 + kRowsPerLaunch);
#define MOE_QUANTIZE(THREADS, EPT)                                                         \
  hipLaunchKernelGGL((quantize_rows<kBf16, THREADS, EPT>), RowOf<THREADS>::grid(end - r0), \
                     dim3(RowOf<THREADS>::kGroup), 0, st, (const u32x4*)x, q, scale, r0, end, \
                     nvec, valid0, valid1)
    switch (row_threads(std::min<int64_t>(cols, 2048 * kRowValues))) {
      case 64: MOE_QUANTIZE(64, kRowValues); break;
      case 128: MOE_QUANTIZE(128, kRowValues); break;
      case 256: MOE_QUANTIZE(256, kRowValues); break;
      case 512: MOE_QUANTIZE(512, kRowValues); break;
      case 1024: MOE_QUANTIZE(1024, kRowValues); break;
      default: MOE_QUANTIZE(1024, 0); break;
    }
#undef MOE_QUANTIZE
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_layer_norm(const Shape& s, const NormIO& io, hipStream_t st) {
  if (s.T <= 0) return hipSuccess;
  if (s.dtype == MOE_BF16)
    return io.q ? norm_launch<true, true>(s, io, st) : norm_launch<true, false>(s, io, st);
  return io.q ? norm_launch<false, true>(s, io, st) : norm_launch<false, false>(s, io, st);
}

size_t norm_grad_partial_bytes(const Shape& s) {
  return (size_t)norm_grad_groups(s) * 2 * s.H * 4;
}

hipError_t launch_layer_norm_backward(const Shape& s, const NormGradIO& io, hipStream_t st) {
  if (s.T > 0) {
    const hipError_t e = s.dtype == MOE_BF16 ? norm_grad_launch<true>(s, io, st)
                                             : norm_grad_launch<false>(s, io, st);
    if (e != hipSuccess) return e;
  }
  if (!io.grad_weight && !io.grad_bias) return hipSuccess;
  if (s.T > 0 && norm_grad_groups(s) == 1) return hipSuccess;  // written by the one workgroup
  hipLaunchKernelGGL(norm_grad_reduce, dim3((unsigned)((s.H + 63) / 64), 2), dim3(256), 0, st,
                     io.partials, s.T > 0 ? norm_grad_groups(s) : 0, s.H, io.grad_weight,
                     io.grad_bias);
  return hipGetLastError();
}

hipError_t launch_quantize_rows(int64_t rows, int64_t cols, bool bf16, const void* x, int8_t* q,
                                float* scale, const int32_t* valid0, const int32_t* valid1,
                                hipStream_t st) {
  if (rows <= 0) return hipSuccess;
  return bf16 ? quantize_launch<true>(rows, cols, x, q, scale, valid0, valid1, st)
              : quantize_launch<false>(rows, cols, x, q, scale, valid0, valid1, st);
}

}  // namespace moe
