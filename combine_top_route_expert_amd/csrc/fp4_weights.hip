// Matrices as 4-bit floating point numbers (E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives) with a power of two for each group of 32 columns, in the packed layout of
// fp4_layout.h:
//   s = least integer with max|group| <= 6 2^s,  q = x / 2^s rounded to the nearest
//   E2M1 number, ties to the even one
// With this s nothing is clipped (the exponent one less, which leaves the largest value
// anywhere in [4, 8) 2^s, would clip up to a quarter of it).  x / 2^s is exact, so every q
// is the correctly rounded one; the conversion instruction gives that for all bf16 values
// and scales, subnormal ones too.  Read back, q 2^s is exact in bf16.
//
// Bound by memory.  A workgroup takes 32 rows by 256 columns, a row's 256 columns to 32
// lanes of 8, so that its reads are contiguous in the rows; the four lanes of a group
// share their maximum by data-parallel shifts.  The 4 KB that it writes go through LDS
// and leave contiguously.  32768 x 7168 in bf16: 91 us to 4 bits and 83 back, 6.5 and 7.1 TB/s.
#include "fp4_layout.h"
#include "row_quantizer.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 32;                            // lanes of a row's 256 columns
constexpr int kPasses = kFp4BlockRows * kLanes / kThreads;  // rows / 8

// Byte offset within the workgroup's four blocks of the 4 bytes that lane `piece` of row r holds.
__device__ __forceinline__ int place(int r, int piece) {
  return (piece >> 3) * kFp4BlockBytes + (((piece >> 2) & 1) * 32 + r) * 16 + (piece & 3) * 4;
}
// The same within their 256 bytes of scales, for the group that the lane belongs to.
__device__ __forceinline__ int scale_place(int r, int piece) {
  return (((piece >> 2) & 1) * 32 + r) * 4 + (piece >> 3);
}

// v of lane l ^ kMask of the quad
template <int kControl>
__device__ __forceinline__ uint32_t quad(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kControl, 0xf, 0xf, true);
}

// Eight values of a row, those of a group in four lanes, as 4 bytes; *scale: the group's.
__device__ __forceinline__ uint32_t quantize8(const float (&f)[8], uint32_t* scale) {
  uint32_t big = max_magnitude<8>(f, 0);  // unsigned: finite < infinity < NaN
  uint32_t o = quad<0xb1>(big);  // lanes 1 0 3 2
  big = o > big ? o : big;
  o = quad<0x4e>(big);  // lanes 2 3 0 1
  big = o > big ? o : big;
  if (big >= 0x7f800000u) {
    *scale = 255;
    return 0;
  }
  // big = m 2^e, 1 <= m < 2: 6 2^s >= big from s = e - 2 (m <= 1.5) or e - 1 on.  The bits
  // of a number give e + 127 above its mantissa, and adding just less than a half to the
  // mantissa carries into it where m > 1.5.  Below 2^-126 byte 0, 2^-127, is enough (6 2^-127).
  const int byte = (int)((big + 0x3fffffu) >> 23) - 2;
  *scale = byte > 0 ? (uint32_t)byte : 0u;
  const float s = __uint_as_float(*scale << 23);
  // values above 3 2^126 would round to 2^128: held at 3
  const float top = *scale == 253 ? 3.0f * 0x1p126f : INFINITY;
  uint32_t q = 0;
#if defined(__HIP_DEVICE_COMPILE__)
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __builtin_fminf(__builtin_fmaxf(f[i], -top), top);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], s, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], s, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], s, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], s, 3);
#else
  (void)s;
  (void)top;
#endif
  return q;
}

// What a workgroup's lanes hold of 32 rows by 256 columns: fetch(row, first column, &scale)
// gives 4 bytes of values and, in each lane of a group, its scale.
template <class F>
__device__ __forceinline__ void write_blocks(int64_t cols, uint8_t* q, uint8_t* scale, F fetch) {
  __shared__ __attribute__((aligned(16))) uint8_t values[4 * kFp4BlockBytes];
  __shared__ __attribute__((aligned(16))) uint8_t scales[kFp4ScaleBytes];
  const int64_t quads = fp4_scale_quads(cols);
  const int64_t rb = blockIdx.x / quads, kq = blockIdx.x % quads;
  const int piece = threadIdx.x % kLanes, row0 = threadIdx.x / kLanes;
  const int64_t col = kq * 256 + piece * 8;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = row0 + i * (kThreads / kLanes);
    uint32_t v = 0, s = 0;
    // (cols is a multiple of 64: the lanes of a group, and of a quad, agree)
    if (col < cols) v = fetch(rb * kFp4BlockRows + r, col, &s);
    *(uint32_t*)(values + place(r, piece)) = v;
    if ((piece & 3) == 0) scales[scale_place(r, piece)] = (uint8_t)s;
  }
  __syncthreads();
  const int64_t nk = cols / kFp4BlockCols;
  const int64_t left = nk - kq * 4;  // blocks from here to the row's end
  const int bytes = (left < 4 ? (int)left : 4) * kFp4BlockBytes;
  u32x4* qd = (u32x4*)(q + (rb * nk + kq * 4) * kFp4BlockBytes);
  if ((int)threadIdx.x * 16 < bytes) qd[threadIdx.x] = ((const u32x4*)values)[threadIdx.x];
  u32x4* sd = (u32x4*)(scale + (rb * quads + kq) * kFp4ScaleBytes);
  if (threadIdx.x < kFp4ScaleBytes / 16) sd[threadIdx.x] = ((const u32x4*)scales)[threadIdx.x];
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads)
quantize_fp4(int64_t cols, const void* x, uint8_t* q, uint8_t* scale) {
  write_blocks(cols, q, scale, [&](int64_t row, int64_t col, uint32_t* s) {
    constexpr int kEl = kVecEl<kBf16>;
    const u32x4* p = (const u32x4*)x + (row * cols + col) / kEl;
    float f[8];
#pragma unroll
    for (int i = 0; i < 8 / kEl; ++i) unpack<kBf16>(__builtin_nontemporal_load(p + i), f + i * kEl);
    return quantize8(f, s);
  });
}

__global__ void __launch_bounds__(kThreads)
pack_fp4(int64_t cols, const uint8_t* q_rows, const uint8_t* scale_rows, uint8_t* q,
         uint8_t* scale) {
  write_blocks(cols, q, scale, [&](int64_t row, int64_t col, uint32_t* s) {
    *s = scale_rows[(row * cols + col) / kFp4Group];
    return *(const uint32_t*)(q_rows + (row * cols + col) / 2);
  });
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads)
dequantize_fp4(int64_t cols, const uint8_t* q, const uint8_t* scale, void* x) {
  const int64_t quads = fp4_scale_quads(cols);
  const int64_t rb = blockIdx.x / quads, kq = blockIdx.x % quads;
  const int piece = threadIdx.x % kLanes, row0 = threadIdx.x / kLanes;
  const int64_t col = kq * 256 + piece * 8;
  if (col >= cols) return;
  const uint8_t* qs = q + (rb * (cols / kFp4BlockCols) + kq * 4) * kFp4BlockBytes;
  const uint8_t* ss = scale + (rb * quads + kq) * kFp4ScaleBytes;
  uint32_t v[kPasses], s[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = row0 + i * (kThreads / kLanes);
    v[i] = *(const uint32_t*)(qs + place(r, piece));
    s[i] = ss[scale_place(r, piece)];
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = row0 + i * (kThreads / kLanes);
    const float power = __uint_as_float(s[i] << 23);
    constexpr int kEl = kVecEl<kBf16>;
    u32x4* dst = (u32x4*)x + ((rb * kFp4BlockRows + r) * cols + col) / kEl;
#if defined(__HIP_DEVICE_COMPILE__)
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], power, 0),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], power, 1),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], power, 2),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[i], power, 3)};
    const u32x4 w = {__builtin_bit_cast(uint32_t, p[0]), __builtin_bit_cast(uint32_t, p[1]),
                     __builtin_bit_cast(uint32_t, p[2]), __builtin_bit_cast(uint32_t, p[3])};
    if constexpr (kBf16) {
      __builtin_nontemporal_store(w, dst);
    } else {  // exact in bf16, so also in fp32
      float f[8];
      unpack_bf16x8(w, f);
      __builtin_nontemporal_store(pack<false>(f), dst);
      __builtin_nontemporal_store(pack<false>(f + 4), dst + 1);
    }
#else
    (void)power;
    (void)dst;
#endif
  }
}

unsigned blocks(int64_t rows, int64_t cols) {
  return (unsigned)(rows / kFp4BlockRows * fp4_scale_quads(cols));
}

}  // namespace

hipError_t launch_quantize_fp4(int64_t rows, int64_t cols, bool bf16, const void* x, uint8_t* q,
                               uint8_t* scale, hipStream_t st) {
  const dim3 grid(blocks(rows, cols)), block(kThreads);
  if (bf16)
    hipLaunchKernelGGL(quantize_fp4<true>, grid, block, 0, st, cols, x, q, scale);
  else
    hipLaunchKernelGGL(quantize_fp4<false>, grid, block, 0, st, cols, x, q, scale);
  return hipGetLastError();
}

hipError_t launch_pack_fp4(int64_t rows, int64_t cols, const uint8_t* q_rows,
                           const uint8_t* scale_rows, uint8_t* q, uint8_t* scale,
                           hipStream_t st) {
  hipLaunchKernelGGL(pack_fp4, dim3(blocks(rows, cols)), dim3(kThreads), 0, st, cols, q_rows,
                     scale_rows, q, scale);
  return hipGetLastError();
}

hipError_t launch_dequantize_fp4(int64_t rows, int64_t cols, bool bf16, const uint8_t* q,
                                 const uint8_t* scale, void* x, hipStream_t st) {
  const dim3 grid(blocks(rows, cols)), block(kThreads);
  if (bf16)
    hipLaunchKernelGGL(dequantize_fp4<true>, grid, block, 0, st, cols, q, scale, x);
  else
    hipLaunchKernelGGL(dequantize_fp4<false>, grid, block, 0, st, cols, q, scale, x);
  return hipGetLastError();
}

}  // namespace moe
