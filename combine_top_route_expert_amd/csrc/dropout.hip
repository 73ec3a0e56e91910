// Dropout of the layer's output on its way into the residual stream:
//   out[i] = rd(residual[i] + (kept(i) ? x[i] / (1 - p) : 0)),  rd: rounding to the dtype
// and its gradient, which is the same map of grad_out without a residual: the mask
// is computed again, never stored.
//
// The mask comes from Philox 4x32 with ten rounds (Salmon, Moraes, Dror, Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011): one counter gives 128 bits,
// which is 16 for each element of an 8-element group, a 16-byte vector of bf16.
// With 32 bits for an element the generator alone would need two counters for a
// vector; at 16 bits p is a multiple of 2^-16 and the factor 1 / (1 - p) that of the
// rounded p, so that the expectation is exact.  A counter is the group's number and
// the call's offset, so the mask depends neither on the dtype nor on the launch.
//
// Bound by memory: 16384 rows of 2048 without a residual 24 us, 5.6 TB/s (a copy of 2 GiB: 4.85);
// 64 rows of 7168 with one 3.0 us, the launch.
#include <algorithm>

#include "row_quantizer.h"

namespace moe {

namespace {

// Four words of Philox 4x32-10 for counter (v, offset) under `key`.
__device__ __forceinline__ u32x4 philox(uint64_t v, uint64_t offset, uint64_t key) {
  uint32_t c0 = (uint32_t)v, c1 = (uint32_t)(v >> 32);
  uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    const uint32_t n0 = (uint32_t)(b >> 32) ^ c1 ^ k0, n2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c0 = n0;
    c1 = (uint32_t)b;
    c2 = n2;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

constexpr int kThreads = 256;
constexpr int kGroups = 2;  // 8-element groups of a thread
// Elements of a launch (4 M threads).  A thread that took several passes over a larger tensor
// would cost 10% of 2^29 elements' time.
constexpr int64_t kMostElements = (int64_t)1 << 30;

// n elements (a multiple of 4) from x on, the first of them in group `first` of the tensor.  out
// may be x or residual: a thread reads its groups before it writes them.
template <bool kBf16, bool kResidual>
__global__ void __launch_bounds__(kThreads)
dropout_add(const u32x4* x, const u32x4* residual, const uint64_t* seed_offset, uint32_t least,
            float factor, u32x4* out, int64_t n, int64_t first) {
  constexpr int kEl = kVecEl<kBf16>, kVecs = 8 / kEl;
  const uint64_t seed = seed_offset[0], offset = seed_offset[1];
  const int64_t groups = (n + 7) / 8;
  const int64_t nvec = n / kEl;  // (fp32: the last group may be half a one)
  const int64_t g0 = (int64_t)blockIdx.x * kThreads * kGroups + threadIdx.x;
  u32x4 a[kGroups][kVecs], r[kGroups][kVecs];
#pragma unroll
  for (int i = 0; i < kGroups; ++i)
#pragma unroll
    for (int q = 0; q < kVecs; ++q) {
      const int64_t v = (g0 + (int64_t)i * kThreads) * kVecs + q;
      if (v < nvec) {
        a[i][q] = __builtin_nontemporal_load(x + v);
        if constexpr (kResidual) r[i][q] = __builtin_nontemporal_load(residual + v);
      }
    }
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int64_t g = g0 + (int64_t)i * kThreads;
    if (g >= groups) break;
    const u32x4 bits = philox((uint64_t)(first + g), offset, seed);
#pragma unroll
    for (int q = 0; q < kVecs; ++q) {
      const int64_t v = g * kVecs + q;
      if (v >= nvec) break;
      float f[kEl], base[kEl];
      unpack<kBf16>(a[i][q], f);
      if constexpr (kResidual) unpack<kBf16>(r[i][q], base);
#pragma unroll
      for (int j = 0; j < kEl; ++j) {
        const int e = q * kEl + j;
        const uint32_t half = e & 1 ? bits[e / 2] >> 16 : bits[e / 2] & 0xffffu;
        // what is dropped is not multiplied: an infinity there leaves no NaN
        if constexpr (kResidual)
          f[j] = half >= least ? __builtin_fmaf(f[j], factor, base[j]) : base[j];
        else
          f[j] = half >= least ? f[j] * factor : 0.0f;
      }
      __builtin_nontemporal_store(pack<kBf16>(f), out + v);
    }
  }
}

}  // namespace

hipError_t launch_dropout_add(const Shape& s, const void* x, const void* residual, double p,
                              const uint64_t* seed_offset, void* out, hipStream_t st) {
  const int64_t n = (int64_t)s.T * s.H;
  if (n == 0) return hipSuccess;
  // p in 16 bits: the least half that is kept (something always is)
  const uint32_t least = (uint32_t)std::min(65535.0, __builtin_rint(p * 65536.0));
  const float factor = 65536.0f / (float)(65536u - least);
  auto go = [&](auto kernel) {
    for (int64_t at = 0; at < n; at += kMostElements) {
      const int64_t left = std::min(n - at, kMostElements), bytes = at * s.elem;
      const int64_t blocks = ((left + 7) / 8 + kThreads * kGroups - 1) / (kThreads * kGroups);
      const char* res = residual ? (const char*)residual + bytes : nullptr;
      hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, st,
                         (const u32x4*)((const char*)x + bytes), (const u32x4*)res, seed_offset, least,
                         factor, (u32x4*)((char*)out + bytes), left, at / 8);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  };
  if (s.dtype == MOE_BF16)
    return residual ? go(dropout_add<true, true>) : go(dropout_add<true, false>);
  return residual ? go(dropout_add<false, true>) : go(dropout_add<false, false>);
}

}  // namespace moe
