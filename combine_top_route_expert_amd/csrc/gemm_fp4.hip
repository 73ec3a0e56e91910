// Grouped expert products with packed 4-bit weights (fp4_layout.h) and rows in two 6-bit
// parts (mx_rows.h):
//   gate_up: act[r] = silu(g) u in two parts,  g, u = x_r . W[e][i], x_r . W[e][I + i]
//   down   : y[r][n] = act_r . W[e][n] in scaled fp16
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 x 64 E2M1 weights by 32 x 64 E2M3 values
// with a power of two for each 32 of either side, in the 32 cycles in which the bf16
// instruction multiplies a quarter of that; the two parts of the rows make it half the
// matrix time of bf16.  Weights go from memory to the instruction as they lie, in one load:
// lane 32 h + r holds the 16 bytes of columns 32 h .. of row r and a dword with its scales of
// four blocks, of which the instruction picks a byte.  (Converted to bf16 in registers
// instead, with bf16 rows and instructions: 2.05 ms for gate_up of 4096 tokens on 256
// experts, H = 7168, I = 2048, instead of 1.24.)  Sums are fp32, over K in ascending order,
// part h before part l in each 64 columns, whatever the tile: both forms give the same bits.
#include <algorithm>
#include <type_traits>

#include "fp4_layout.h"
#include "gemm_tile.h"
#include "mx_rows.h"

namespace moe {

namespace {

typedef int i32x12 __attribute__((ext_vector_type(12)));

struct MxArgs {
  MxRows a;                   // rows of A
  const int32_t *off0, *off1; // E + 1 offsets of the chunk(s); off1 may be null
  const char *b, *bs;         // packed weights and scales, expert after expert
  int64_t b_expert, bs_expert;
  int E, ncols, n_tiles;      // columns of C, column tiles
  int blocks, quads;          // 64-column blocks of K, scale dwords of a weight row
  int up;                     // gate_up: row blocks from a gate row to its up row
  MxRows c;                   // gate_up: act
  MxRows y[2];                // down: the two chunks' rows
  int c_split;
};

// One product of 64 columns: weights w (16 bytes a lane) and a part of the rows (the first
// or the last 24 of a lane's 48 bytes), with byte kWs of the weights' scales and byte kAs + kPart
// of the rows'.
template <int kPart, int kWs, int kAs>
__device__ __forceinline__ f32x16 mx_mma(const i32x4& w, uint32_t ws, const i32x12& a, uint32_t as,
                                         const f32x16& c) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef int i32x8 __attribute__((ext_vector_type(8)));
  const i32x8 wv = __builtin_shufflevector(w, w, 0, 1, 2, 3, -1, -1, -1, -1);
  i32x8 av;
  if constexpr (kPart == 0)
    av = __builtin_shufflevector(a, a, 0, 1, 2, 3, 4, 5, -1, -1);
  else
    av = __builtin_shufflevector(a, a, 6, 7, 8, 9, 10, 11, -1, -1);
  // (4: E2M1, 2: E2M3)
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv, av, c, 4, 2, kWs, (int)ws, kAs + kPart,
                                                         (int)as);
#else
  return c;
#endif
}

// A lane's 48 bytes of a row block, from its thirds.
__device__ __forceinline__ i32x12 both_parts(const i32x4 (&a)[3]) {
  return __builtin_shufflevector(
      __builtin_shufflevector(a[0], a[1], 0, 1, 2, 3, 4, 5, 6, 7),
      __builtin_shufflevector(a[2], a[2], 0, 1, 2, 3, -1, -1, -1, -1), 0, 1, 2, 3, 4, 5, 6, 7, 8, 9,
      10, 11);
}

// Row block of the packed weights behind block j of a tile's NB (FN to a wave): gate_up, a
// wave's first half gate and the matching up rows after; clamped, since what lies past C
// is never stored.
template <bool kGateUp, int FN>
__device__ __forceinline__ int weight_block(const MxArgs& g, int nt, int nb, int j) {
  const int last = g.ncols / kFp4BlockRows - 1;
  if constexpr (kGateUp) {
    const int q = j % FN / (FN / 2);
    const int rb = nt * (nb / 2) + j / FN * (FN / 2) + j % (FN / 2);
    return (rb < last ? rb : last) + q * g.up;
  } else {
    const int rb = nt * nb + j;
    return rb < last ? rb : last;
  }
}

// ---------------------------------------------------------------- many rows an expert
// A workgroup of four waves, one for each SIMD with all its 512 registers, computes up to 128
// rows by 512 columns, a wave all the rows of its own 128 columns (R x 4 blocks of 32 x 32).
// The weights, which no other wave uses, go from memory straight into registers, three stages
// (of 64 columns of K) ahead; the rows go through LDS, a unit of four stages at a time in
// two buffers, and a row block's operands are read while the one before is multiplied.
//
// Why this shape: a column of A is 12 bits and one of the weights 4, so that of tiles of 65536
// sums, all that a CU's registers hold, the one of 128 x 512 copies less than 256 x 256 (28 KB
// a stage against 32); and with the weights past LDS a stage's 1024 cycles of matrix
// instructions go with 48 KB of reads and 12 KB of writes there.  256 x 256 with both sides in
// LDS, two by two waves (64 and 32 KB) took 2000 cycles a stage, about the sum of what its reads
// and its copies cost: the layer of 4096 tokens with 8 of 256 experts of H = 7168, I = 2048 2.67
// ms instead of 2.36, of 1024 tokens 1.53 instead of 1.24, of 16384 tokens with 8 of 128 experts
// of H = 2048, I = 768 1.26 instead of 1.13 to 1.21.
//
// The first of these: gate_up 1.21 ms and down 0.80, 1.43 PFLOP/s, 4.9 TB/s of weights.  Neither
// the matrix pipe (0.64 and 0.32 ms at the 6 PF/s that the instruction reaches, power being what
// limits it) nor memory (0.59 and 0.29) is full: tiles whose last row block holds a few rows,
// prologues and epilogues with one workgroup on a CU, and LDS take the rest.  Without effect:
// seven stages ahead for up to 64 rows (0 to 5% slower); twice the row tiles to a group of an
// XCD's workgroups; experts in order instead of large ones first (0 to 2% slower); weights that
// leave no trace in the caches (1% slower, 7% where the layer fits them).
constexpr int kWaves = 4, kWideFN = 4;  // waves; column blocks of a wave
constexpr int kUnit = 4;                // stages of a unit
constexpr int kWideRows = 128;

template <int R>
struct WideUnit {
  static constexpr int kAtScales = R * kUnit * kMxBlockBytes;
  static constexpr int kBytes = kAtScales + R * kUnit / 2 * kMxScaleBytes;
  static constexpr int kValues = R * kUnit * 3 / kWaves;               // a wave's copies
  static constexpr int kScales = (R * kUnit / 2 + kWaves - 1) / kWaves;
  static constexpr int kCopies = kValues + kScales;
};

// The K loop of a wave.
template <bool kGateUp, int R>
__device__ __forceinline__ void wide_k_loop(f32x16 (&acc)[R][kWideFN], const MxArgs& g,
                                            const TileRows& tr, int nt, int lane, int wave,
                                            char* smem) {
  using U = WideUnit<R>;
  constexpr int FN = kWideFN;
  const int e = __builtin_amdgcn_readfirstlane(tr.e);
  const int KB = g.blocks, units = g.quads, pairs = (KB + 1) / 2, full = KB / kUnit;
  const int64_t rb0 = mx_row_block(tr, tr.v0);
  const char* av = g.a.values + rb0 * KB * kMxBlockBytes + lane * 16;
  const char* as = g.a.scales + rb0 * pairs * kMxScaleBytes + lane * 4;
  // Copy q of unit u: kilobyte q of the values, then 256 bytes of scales; blocks past the last
  // of K repeat that, and copies past a unit's last repeat it.
  auto copy = [&](int u, int t) __attribute__((always_inline)) {
    char* base = smem + (u & 1) * U::kBytes;
    if (t < U::kValues) {
      const int q = t * kWaves + wave, i = q / (3 * kUnit), k = kUnit * u + q % (3 * kUnit) / 3;
      __builtin_amdgcn_global_load_lds(
          (const void*)(av + ((int64_t)i * KB + (k < KB ? k : KB - 1)) * kMxBlockBytes + q % 3 * 1024),
          (lds_void*)(base + q * 1024), 16, 0, 0);
    } else {
      int q = (t - U::kValues) * kWaves + wave;
      q = q < R * kUnit / 2 ? q : R * kUnit / 2 - 1;
      const int i = q / (kUnit / 2), pair = kUnit / 2 * u + q % (kUnit / 2);
      __builtin_amdgcn_global_load_lds(
          (const void*)(as + ((int64_t)i * pairs + (pair < pairs ? pair : pairs - 1)) * kMxScaleBytes),
          (lds_void*)(base + U::kAtScales + q * kMxScaleBytes), 4, 0, 0);
    }
  };
  const i32x4* b[FN];
  const uint32_t* bs[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int rb = weight_block<kGateUp, FN>(g, nt, kWaves * FN, wave * FN + j);
    b[j] = (const i32x4*)(g.b + e * g.b_expert + (int64_t)rb * KB * kFp4BlockBytes) + lane;
    bs[j] = (const uint32_t*)(g.bs + e * g.bs_expert + (int64_t)rb * units * kFp4ScaleBytes) + lane;
  }
  i32x4 w[kUnit][FN];
  uint32_t sc[FN], sn[FN];
  struct Row {
    i32x4 thirds[3];
    uint32_t s;
  };
  Row row[2];
  auto load = [&](int k, int j, i32x4& to) __attribute__((always_inline)) {
    to = b[j][(int64_t)k * (kFp4BlockBytes / 16)];
  };
  auto read = [&](Row& to, int u, int k, int i, int t) __attribute__((always_inline)) {
    const char* base = smem + (u & 1) * U::kBytes;
    if (t < 3)
      to.thirds[t] = *(const i32x4*)(base + (i * kUnit + k) * kMxBlockBytes + t * 1024 + lane * 16);
    else
      to.s = *(const uint32_t*)(base + U::kAtScales + (i * (kUnit / 2) + k / 2) * kMxScaleBytes +
                                lane * 4);
  };
#pragma unroll
  for (int t = 0; t < U::kCopies; ++t) copy(0, t);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int j = 0; j < FN; ++j) sn[j] = sc[j] = bs[j][0];
#pragma unroll
  for (int k = 0; k < kUnit - 1; ++k)
    if (k < KB) {
#pragma unroll
      for (int j = 0; j < FN; ++j) load(k, j, w[k][j]);
    }
  __builtin_amdgcn_sched_barrier(0);
  // (the copies have landed: at most what came after them is pending)
  if (KB >= kUnit - 1)
    __builtin_amdgcn_s_waitcnt(wait_vm((kUnit - 1) * FN));
  else
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int t = 0; t < 4; ++t) read(row[0], 0, 0, 0, t);

  // Stage k of unit u.  kFull: unit u + 1 is a whole one.
  auto stage = [&](int u, auto k_tag, auto full_tag) __attribute__((always_inline)) {
    constexpr int k = decltype(k_tag)::value;
    constexpr bool kFull = decltype(full_tag)::value;
    const bool next = kFull || u + 1 < units;              // there is a unit u + 1
    const bool ahead = kFull || kUnit * u + k + kUnit - 1 < KB;  // the stage to load
    if (k == 0 && next) {
#pragma unroll
      for (int j = 0; j < FN; ++j) sn[j] = bs[j][(u + 1) * (kFp4ScaleBytes / 4)];
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const bool last = k == kUnit - 1 && i == R - 1;
      if (last && next) {
        // every wave has read this unit; the copies of the next, issued in the first stage, have
        // landed once at most the loads issued after that stage are pending
        constexpr int kLoads = (R > 1 ? kUnit - 1 : kUnit - 2) * FN;
        __builtin_amdgcn_s_waitcnt(kFull ? wait_vm(kLoads) : wait_vm(0));
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }
      const Row& now = row[(k * R + i) & 1];
      Row& then = row[(k * R + i + 1) & 1];
      const i32x12 rows = both_parts(now.thirds);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < 2 * FN; ++m) {
        const int j = m % FN;
        acc[i][j] = m < FN ? mx_mma<0, k, 2 * (k & 1)>(w[k][j], sc[j], rows, now.s, acc[i][j])
                           : mx_mma<1, k, 2 * (k & 1)>(w[k][j], sc[j], rows, now.s, acc[i][j]);
        // (the compiler moves matrix instructions down past branches, and so past the copies
        // and the barrier that they are to cover, unless their results are named before)
        asm volatile("" : "+a"(acc[i][j]));
        __builtin_amdgcn_sched_barrier(0);
        if (m < 4) {
          if (i < R - 1)
            read(then, u, k, i + 1, m);
          else if (k < kUnit - 1)
            read(then, u, k + 1, 0, m);  // (of a stage past the last, unused)
          else if (next)
            read(then, u + 1, 0, 0, m);
        }
        if (i == 0 && m >= 2 * FN - FN && ahead)
          load(kUnit * u + k + kUnit - 1, m - FN, w[(k + kUnit - 1) % kUnit][m - FN]);
        if (k == 0 && next) {
          constexpr int kMma = 2 * FN * R;
          const int at = i * 2 * FN + m;
#pragma unroll
          for (int t = at * U::kCopies / kMma; t < (at + 1) * U::kCopies / kMma; ++t) copy(u + 1, t);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  const std::integral_constant<int, 0> k0{};
  const std::integral_constant<int, 1> k1{};
  const std::integral_constant<int, 2> k2{};
  const std::integral_constant<int, 3> k3{};
  const std::true_type whole{};
  const std::false_type part{};
  int u = 0;
  for (; u + 1 < full; ++u) {
    stage(u, k0, whole);
    stage(u, k1, whole);
    stage(u, k2, whole);
    stage(u, k3, whole);
#pragma unroll
    for (int j = 0; j < FN; ++j) sc[j] = sn[j];
  }
  for (; u < units; ++u) {
    stage(u, k0, part);
    if (kUnit * u + 1 < KB) stage(u, k1, part);
    if (kUnit * u + 2 < KB) stage(u, k2, part);
    if (kUnit * u + 3 < KB) stage(u, k3, part);
#pragma unroll
    for (int j = 0; j < FN; ++j) sc[j] = sn[j];
  }
}

// act of 32 rows by 32 columns of two row blocks, from the accumulators of gate and up
// columns: lane l holds row l % 32 of a block and its columns 8 (q / 4) + 4 (l / 32) + q % 4.
// Swapping the upper half of one block's registers with the lower half of the other's
// leaves lane l all 32 columns of one row, in the first block (l < 32) or the second.
__device__ __forceinline__ TwoParts act_parts(const f32x16& g0, const f32x16& u0, const f32x16& g1,
                                              const f32x16& u1) {
  f32x16v even, odd;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const float a = swiglu<true>(g0[q], u0[q]), b = swiglu<true>(g1[q], u1[q]);
    float lo = a, hi = b;  // columns 8 (q / 4) + q % 4 and 4 more of the lane's row
#if defined(__HIP_DEVICE_COMPILE__)
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false,
                                                    false);
    lo = __uint_as_float(s[0]);
    hi = __uint_as_float(s[1]);
#endif
    const int c = 4 * (q / 4) + q % 4 / 2;  // half of the first's column
    if (q % 2 == 0) {
      even[c] = lo;
      even[c + 2] = hi;
    } else {
      odd[c] = lo;
      odd[c + 2] = hi;
    }
  }
  return split32(even, odd);
}

// Stores the act rows of a wave's FM row blocks, 32-column blocks block0 on.
template <int FM, int FN>
__device__ __forceinline__ void store_act(const MxArgs& a, const f32x16 (&acc)[FM][FN],
                                          const TileRows& tr, int block0, int lane) {
  constexpr int FC = FN / 2;
  const int r = lane & 31, half = lane >> 5;
  const int nk = a.ncols / 64;
#pragma unroll
  for (int i = 0; i < FM; i += 2) {
    constexpr int kLast = FM - 1;
    const int i1 = i < kLast ? i + 1 : i;
    const int row = 32 * (i + half) + r;
    const bool live = row < tr.rows && (half == 0 || i + 1 < FM);
    const int64_t rb = mx_row_block(tr, tr.v0 + 32 * (i + half));
#pragma unroll
    for (int j = 0; j < FC; ++j) {
      const int block = block0 + j;
      if (block * 32 >= a.ncols) break;
      const TwoParts p = act_parts(acc[i][j], acc[i][j + FC], acc[i1][j], acc[i1][j + FC]);
      if (live) store_parts(p, a.c, nk, rb, r, block);
      __builtin_amdgcn_sched_barrier(0);  // one block at a time: a split holds a hundred registers
    }
  }
}

// Scaled fp16 of 64 columns of a row (two blocks' accumulators): the byte of the power of two
// that brings the largest finite magnitude into [2^14, 2^15).
__device__ __forceinline__ uint32_t out_scale(const f32x16& a, const f32x16& b) {
  uint32_t big = 0;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const uint32_t x = __float_as_uint(a[q]) & 0x7fffffffu, y = __float_as_uint(b[q]) & 0x7fffffffu;
    big = x > big && x < 0x7f800000u ? x : big;
    big = y > big && y < 0x7f800000u ? y : big;
  }
  const uint32_t other = (uint32_t)__shfl_xor((int)big, 32);  // the row's other columns
  big = other > big ? other : big;
  const int byte = (int)(big >> 23) - 14;
  return byte > 14 ? (uint32_t)byte : 14u;  // (its reciprocal has to be a number)
}
__device__ __forceinline__ float out_factor(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// down's epilogue of a wide tile: fp16 rows through the freed LDS, row-major, with a row's scale
// bytes behind them, out in 16-byte pieces.
template <int FM, int FN, int BM, int BN, int NT>
__device__ __forceinline__ void store_out(const MxArgs& a, const f32x16 (&acc)[FM][FN],
                                          const TileRows& tr, int nt, int wn, int lane, char* smem) {
  typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
  constexpr int CPR = BN / 8;  // 16-byte chunks of a tile row
  auto at = [](int r, int c) {
    return r * (BN * 2) + (((c >> 3) ^ (r & (CPR - 1))) << 4) + (c & 7) * 2;
  };
  uint8_t* scales = (uint8_t*)smem + BM * BN * 2;
  const int r0 = lane & 31, cq = 4 * (lane >> 5);
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int r = r0 + i * 32;
#pragma unroll
    for (int j = 0; j < FN; j += 2) {
      const uint32_t byte = out_scale(acc[i][j], acc[i][j + 1]);
      const float p = out_factor(byte);
      if (lane < 32) scales[r * (BN / 64) + (wn * FN + j) / 2] = (uint8_t)byte;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x16& x = acc[i][j + h];
          *(f16x4*)(smem + at(r, (wn * FN + j + h) * 32 + 8 * g + cq)) =
              f16x4{(_Float16)(x[4 * g] * p), (_Float16)(x[4 * g + 1] * p),
                    (_Float16)(x[4 * g + 2] * p), (_Float16)(x[4 * g + 3] * p)};
        }
    }
  }
  __syncthreads();
  const int col0 = nt * BN;
  for (int ch = threadIdx.x; ch < BM * CPR; ch += NT) {
    const int r = ch / CPR, c = (ch % CPR) * 8;
    if (r >= tr.rows || col0 + c >= a.ncols) continue;
    int part = 0, row = tr.joint_row(tr.v0 + r);
    if (a.c_split) row = tr.split_row(tr.v0 + r, &part);
    char *y0 = a.y[0].values, *y1 = a.y[1].values;
    __builtin_nontemporal_store(*(const u32x4*)(smem + at(r, c)),
                                (u32x4*)((part ? y1 : y0) + ((int64_t)row * a.ncols + col0 + c) * 2));
  }
  constexpr int kDwords = BN / 256;  // of a tile row's scales
  const int64_t row_scales = mx_out_scales(a.ncols);
  for (int i = threadIdx.x; i < tr.rows * kDwords; i += NT) {
    const int r = i / kDwords, d = nt * kDwords + i % kDwords;
    if (d * 256 >= a.ncols) continue;
    int part = 0, row = tr.joint_row(tr.v0 + r);
    if (a.c_split) row = tr.split_row(tr.v0 + r, &part);
    char *s0 = a.y[0].scales, *s1 = a.y[1].scales;
    *(uint32_t*)((part ? s1 : s0) + row * row_scales + d * 4) = *(const uint32_t*)(scales + i * 4);
  }
}

// Scaled fp16 of 32 rows of the 64 columns from col0 on, straight from the accumulators: lane
// l holds row l % 32 and columns 8 (q / 4) + 4 (l / 32) + q % 4 of each block.
__device__ __forceinline__ void store_out_rows(const MxArgs& a, const f32x16 (&acc)[2],
                                               const TileRows& tr, int col0, int lane) {
  typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
  const uint32_t byte = out_scale(acc[0], acc[1]);
  const float p = out_factor(byte);
  const int r = lane & 31, half = lane >> 5;
  if (r >= tr.rows || col0 >= a.ncols) return;
  int part = 0, row = tr.joint_row(tr.v0 + r);
  if (a.c_split) row = tr.split_row(tr.v0 + r, &part);
  char* to = (part ? a.y[1].values : a.y[0].values) + ((int64_t)row * a.ncols + col0) * 2;
  if (half == 0)
    ((uint8_t*)(part ? a.y[1].scales : a.y[0].scales))[row * mx_out_scales(a.ncols) + col0 / 64] =
        (uint8_t)byte;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const f32x16& x = acc[j];
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *(f16x4*)(to + (32 * j + 8 * g + 4 * half) * 2) =
          f16x4{(_Float16)(x[4 * g] * p), (_Float16)(x[4 * g + 1] * p),
                (_Float16)(x[4 * g + 2] * p), (_Float16)(x[4 * g + 3] * p)};
  }
}

template <bool kGateUp>
__global__ void __launch_bounds__(64 * kWaves, 1) grouped_gemm_mx(MxArgs a) {
  constexpr int FN = kWideFN, BN = 32 * FN * kWaves, NT = 64 * kWaves;
  constexpr int kTile = kGateUp ? 0 : kWideRows * (BN * 2 + BN / 64), kUnits = 2 * WideUnit<4>::kBytes;
  __shared__ __attribute__((aligned(1024))) char smem[kUnits > kTile ? kUnits : kTile];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  MTileMap tm;
  tm.build(a.off0, a.off1, a.E, kWideRows, kWideRows);
  int mt, nt;
  if (!xcd_tile_at(tm, a.n_tiles, blockIdx.x & 7, blockIdx.x >> 3,
                   (32 + a.n_tiles - 1) / a.n_tiles, &mt, &nt))
    return;
  const TileRows tr = tm.locate(a.off0, a.off1, kWideRows, mt);
  auto run = [&](auto r_tag) __attribute__((always_inline)) {
    constexpr int R = decltype(r_tag)::value;
    f32x16 acc[R][FN];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};
    wide_k_loop<kGateUp, R>(acc, a, tr, nt, lane, wave, smem);
    if constexpr (kGateUp) {
      store_act<R, FN>(a, acc, tr, (nt * kWaves + wave) * (FN / 2), lane);
    } else {
      __syncthreads();  // every wave is done with the rows
      store_out<R, FN, 32 * R, BN, NT>(a, acc, tr, nt, wave, lane, smem);
    }
  };
  if (tr.rows <= 32)
    run(std::integral_constant<int, 1>{});
  else if (tr.rows <= 64)
    run(std::integral_constant<int, 2>{});
  else if (tr.rows <= 96)
    run(std::integral_constant<int, 3>{});
  else
    run(std::integral_constant<int, 4>{});
}

template <bool kGateUp>
hipError_t launch_wide(MxArgs a, int64_t rows_bound, hipStream_t st) {
  constexpr int cols = kWaves * kWideFN * (kGateUp ? 16 : 32);
  a.n_tiles = (a.ncols + cols - 1) / cols;
  const int64_t grid = xcd_grid(m_tiles_bound(rows_bound, a.E, kWideRows), a.n_tiles);
  if (grid <= 0) return hipSuccess;
  if (grid > 0x7fffffff / (64 * kWaves)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(grouped_gemm_mx<kGateUp>, dim3((unsigned)grid), dim3(64 * kWaves), 0, st, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------- few rows an expert
// Products with up to 32 rows a tile, bound by streaming the weights: every wave reads its own
// 64 weight rows (gate_up: 32 gate rows and their up rows) straight into registers, a unit of
// four stages ahead, and no other wave reads them; only the rows of A, which the waves of a
// workgroup share, go through LDS, a unit at a time in two buffers with one barrier for it.
// Of an H = 7168, I = 2048 layer with 64 tokens on 8 of 256 experts (2 rows each) gate_up
// reads 3.4 GB in 590 us and down 1.7 in 285, 5.9 and 6.1 TB/s (a plain read of such weights:
// 6.8).  Loads that leave the weights in the caches cost 6% more; two or six waves a
// workgroup 0 and 19%.
constexpr int kStreamWaves = 4;
// Rows an expert, on average, up to which these products are taken.  The layer above in ms, these
// and the wide ones: 1 row (an expert that has any) 0.45 and 0.51, 2 rows 0.89 and 0.97, 8 rows
// 1.06 and 1.11, 16 rows 1.13 and 1.14, 32 rows 1.63 and 1.24; with H = 2048, I = 1024, 64
// experts 4 rows 0.066 and 0.066, 32 rows 0.085 and 0.077.
constexpr int kStreamRows = 24;

template <bool kGateUp>
__global__ void __launch_bounds__(64 * kStreamWaves) stream_mx(MxArgs a) {
  constexpr int BM = 32, FN = 2;
  constexpr int kUnitBytes = kUnit * kMxBlockBytes + kUnit / 2 * kMxScaleBytes;
  __shared__ __attribute__((aligned(1024))) char smem[2 * kUnitBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  MTileMap tm;
  tm.build(a.off0, a.off1, a.E, BM, BM);
  int mt, nt;
  if (!xcd_tile_at(tm, a.n_tiles, blockIdx.x & 7, blockIdx.x >> 3,
                   (32 + a.n_tiles - 1) / a.n_tiles, &mt, &nt))
    return;
  const TileRows tr = tm.locate(a.off0, a.off1, BM, mt);
  const int e = __builtin_amdgcn_readfirstlane(tr.e);
  const int units = a.quads, KB = a.blocks, pairs = (KB + 1) / 2;
  const int r = lane & 31;

  // Unit u of A: twelve kilobytes of values, three to a wave, and two dwords a row of scales.
  // Blocks past the last of K repeat that; the entries of rows past the tile's are not copied.
  const int64_t rb0 = mx_row_block(tr, tr.v0);
  const char* av = a.a.values + rb0 * KB * kMxBlockBytes + lane * 16;
  const char* as = a.a.scales + rb0 * pairs * kMxScaleBytes + lane * 4;
  auto copy = [&](int u) __attribute__((always_inline)) {
    if (r >= tr.rows) return;
    char* base = smem + (u & 1) * kUnitBytes;
#pragma unroll
    for (int t = 0; t < kUnit * 3 / kStreamWaves; ++t) {
      const int q = t * kStreamWaves + wave, k = kUnit * u + q / 3;
      __builtin_amdgcn_global_load_lds(
          (const void*)(av + (int64_t)(k < KB ? k : KB - 1) * kMxBlockBytes + q % 3 * 1024),
          (lds_void*)(base + q * 1024), 16, 0, 0);
    }
    const int d = wave & 1, pair = 2 * u + d;
    __builtin_amdgcn_global_load_lds(
        (const void*)(as + (int64_t)(pair < pairs ? pair : pairs - 1) * kMxScaleBytes),
        (lds_void*)(base + kUnit * kMxBlockBytes + d * kMxScaleBytes), 4, 0, 0);
  };
  const i32x4* b[FN];
  const uint32_t* bs[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int rb = weight_block<kGateUp, FN>(a, nt, kStreamWaves * FN, wave * FN + j);
    b[j] = (const i32x4*)(a.b + e * a.b_expert + (int64_t)rb * KB * kFp4BlockBytes) + lane;
    bs[j] = (const uint32_t*)(a.bs + e * a.bs_expert + (int64_t)rb * units * kFp4ScaleBytes) + lane;
  }
  f32x16 acc[1][FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) acc[0][j] = f32x16{};

  i32x4 w[kUnit][FN];
  uint32_t sc[FN], sn[FN];
  auto load = [&](int k, i32x4 (&to)[FN]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
      to[j] = __builtin_nontemporal_load(b[j] + (int64_t)k * (kFp4BlockBytes / 16));
  };
  copy(0);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int j = 0; j < FN; ++j) sn[j] = sc[j] = bs[j][0];
#pragma unroll
  for (int k = 0; k < kUnit; ++k)
    if (k < KB) load(k, w[k]);
  auto stage = [&](const char* sa, auto k_tag, const i32x4 (&x)[FN]) __attribute__((always_inline)) {
    constexpr int k = decltype(k_tag)::value;
    i32x4 thirds[3];
#pragma unroll
    for (int t = 0; t < 3; ++t)
      thirds[t] = *(const i32x4*)(sa + k * kMxBlockBytes + t * 1024 + lane * 16);
    const uint32_t s =
        *(const uint32_t*)(sa + kUnit * kMxBlockBytes + k / 2 * kMxScaleBytes + lane * 4);
    const i32x12 row = both_parts(thirds);
#pragma unroll
    for (int j = 0; j < FN; ++j)
      acc[0][j] = mx_mma<0, k, 2 * (k & 1)>(x[j], sc[j], row, s, acc[0][j]);
#pragma unroll
    for (int j = 0; j < FN; ++j)
      acc[0][j] = mx_mma<1, k, 2 * (k & 1)>(x[j], sc[j], row, s, acc[0][j]);
  };
  const std::integral_constant<int, 0> k0{};
  const std::integral_constant<int, 1> k1{};
  const std::integral_constant<int, 2> k2{};
  const std::integral_constant<int, 3> k3{};
  const int full = KB / kUnit;  // whole units
  for (int u = 0; u < units; ++u) {
    __builtin_amdgcn_sched_barrier(0);
    // this unit's rows have landed once only the loads of a whole unit's stages, which were
    // issued after them, are pending
    if (u < full)
      __builtin_amdgcn_s_waitcnt(wait_vm(kUnit * FN));
    else
      __builtin_amdgcn_s_waitcnt(wait_vm(0));
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);  // and this wave's reads of the other buffer are done
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const char* sa = smem + (u & 1) * kUnitBytes;
    if (u + 1 < units) copy(u + 1);
    __builtin_amdgcn_sched_barrier(0);  // (that count: no load moves up past the copies)
    if (u + 1 < units) {
#pragma unroll
      for (int j = 0; j < FN; ++j) sn[j] = bs[j][(u + 1) * (kFp4ScaleBytes / 4)];
    }
    if (u + 1 < full) {
      stage(sa, k0, w[0]);
      load(kUnit * (u + 1), w[0]);
      stage(sa, k1, w[1]);
      load(kUnit * (u + 1) + 1, w[1]);
      stage(sa, k2, w[2]);
      load(kUnit * (u + 1) + 2, w[2]);
      stage(sa, k3, w[3]);
      load(kUnit * (u + 1) + 3, w[3]);
    } else {
      auto part = [&](auto k_tag) __attribute__((always_inline)) {
        constexpr int k = decltype(k_tag)::value;
        if (kUnit * u + k < KB) stage(sa, k_tag, w[k]);
        if (kUnit * (u + 1) + k < KB) load(kUnit * (u + 1) + k, w[k]);
      };
      part(k0);
      part(k1);
      part(k2);
      part(k3);
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) sc[j] = sn[j];
  }

  if constexpr (kGateUp) {
    store_act<1, FN>(a, acc, tr, nt * kStreamWaves + wave, lane);
  } else {
    store_out_rows(a, acc[0], tr, (nt * kStreamWaves + wave) * 64, lane);
  }
}

template <bool kGateUp>
hipError_t launch_stream(MxArgs a, int64_t rows_bound, hipStream_t st) {
  constexpr int cols = kStreamWaves * (kGateUp ? 32 : 64);
  a.n_tiles = (a.ncols + cols - 1) / cols;
  const int64_t grid = xcd_grid(m_tiles_bound(rows_bound, a.E, 32), a.n_tiles);
  if (grid <= 0) return hipSuccess;
  if (grid > 0x7fffffff / (64 * kStreamWaves)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((stream_mx<kGateUp>), dim3((unsigned)grid), dim3(64 * kStreamWaves), 0, st,
                     a);
  return hipGetLastError();
}

template <bool kGateUp>
hipError_t launch(const MxArgs& a, int64_t rows_bound, hipStream_t st) {
  if (rows_bound <= 0) return hipSuccess;
  if (rows_bound <= (int64_t)kStreamRows * a.E) return launch_stream<kGateUp>(a, rows_bound, st);
  return launch_wide<kGateUp>(a, rows_bound, st);
}

// K columns; `rows` rows of an expert's weights.
MxArgs mx_args(const Shape& s, const MxIO& io, const MxRows& rows_of_a, int K, int rows) {
  MxArgs a{};
  a.a = rows_of_a;
  a.off0 = io.off[0];
  a.off1 = io.off[1];
  a.b = (const char*)io.w;
  a.bs = (const char*)io.w_scale;
  a.b_expert = (int64_t)rows * K / 2;
  a.bs_expert = fp4_scale_bytes(rows, K);
  a.E = s.E;
  a.blocks = K / kFp4BlockCols;
  a.quads = (int)fp4_scale_quads(K);
  return a;
}

}  // namespace

hipError_t launch_gate_up_mx(const Shape& s, const MxIO& io, const MxRows& x, const MxRows& act,
                             hipStream_t st) {
  MxArgs a = mx_args(s, io, x, s.H, 2 * s.I);
  a.ncols = s.I;
  a.up = s.I / kFp4BlockRows;
  a.c = act;
  return launch<true>(a, io.rows_bound, st);
}

hipError_t launch_down_mx(const Shape& s, const MxIO& io, const MxRows& act, const MxRows (&y)[2],
                          hipStream_t st) {
  MxArgs a = mx_args(s, io, act, s.I, s.H);
  a.ncols = s.H;
  a.y[0] = y[0];
  a.y[1] = io.off[1] ? y[1] : y[0];
  a.c_split = io.off[1] != nullptr;
  return launch<false>(a, io.rows_bound, st);
}

}  // namespace moe
