// Grouped expert products with bf16 rows and packed 4-bit weights (fp4_layout.h):
//   gate_up: act[r] = rd(silu(g) u),  g, u = x_r . W[e][i], x_r . W[e][I + i]
//   down   : y[r][n] = act_r . W[e][n] in scaled fp16
//
// A weight is an E2M1 number times a power of two, which bf16 holds exactly, and the rows are
// those that the caller gave, so all products are exact, as those of the bf16 layer with the
// weights written out.  Weights go from memory straight into registers as they lie: lane 32 h + r
// of a load holds the 16 bytes of columns 32 h .. + 31 of row r, and of a dword its scales of four
// blocks; v_cvt_scalef32_pk_bf16_fp4 makes two operands and their power of two in one instruction,
// right before the matrix instructions that they feed.  Instruction q of a block's four
// multiplies columns 8 q .. + 7 of both halves; the rows' fragments are read to match.  Sums are
// fp32, over K in ascending order of the instructions, whatever the tile: both forms give the same
// bits.
//
// Against this, rows in two 6-bit parts on v_mfma_scale_f32_32x32x64_f8f6f4, which multiplies
// the packed weights at up to four times the rate, halve the matrix time, but keep of a row only
// 2^-9 of the largest of 32 neighbours: small values beside a large one are lost.
#include <algorithm>
#include <type_traits>

#include "fp4_operand.h"

namespace moe {

namespace {

// A: hidden states or act; B: packed weights; C (gate_up): act.
struct MxArgs : GemmArgs {
  const char* bs;             // scales, expert after expert
  int64_t bs_expert;
  int blocks, quads;          // 64-column blocks of K, scale dwords of a weight row
  int up;                     // gate_up: row blocks from a gate row to its up row
  ScaledRows y[2];            // down: the two chunks' rows
};

// A stage is 64 columns of K, 128 bytes of a row: 32 rows of one are 4 KB of LDS, chunk c of 16
// bytes of row r at slot c ^ swz(r), copied a kilobyte (8 rows) at a time.
using Stage = StageGeom<128>;
constexpr int kRowBlockBytes = 32 * Stage::ROW_BYTES;

// What this lane copies of row `row` of a tile (one past its last repeats that): the address of
// its 16 bytes of the row's first stage.
template <bool kGateUp>
__device__ __forceinline__ const char* row_piece(const MxArgs& g, const TileRows& tr, int row,
                                                 int lane) {
  const int v = tr.v0 + (row < tr.rows ? row : tr.rows - 1);
  int64_t r;
  if constexpr (kGateUp) {  // the permute, in the rows' addresses
    int part;
    const int cr = tr.split_row(v, &part);
    const int32_t *g0 = g.gather[0], *g1 = g.gather[1];
    r = (part ? g1 : g0)[cr] / g.gather_k;
  } else {
    r = tr.joint_row(v);
  }
  return g.A[0] + r * g.row_bytes + ((lane % Stage::CH) ^ Stage::swz(row)) * 16;
}

// Offset within a row block of a lane's fragment for instruction q of a stage.
__device__ __forceinline__ int fragment_at(int lane, int q) {
  const int r = lane & 31, half = lane >> 5;
  return r * Stage::ROW_BYTES + (((4 * half + q) ^ Stage::swz(r)) << 4);
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
// two buffers, their fragments read two steps (of four matrix instructions) ahead.
//
// Why this shape: of tiles of 65536 sums, all that a CU's registers hold, it copies the least for a
// stage (16 KB of rows and 17 of weights; 256 x 256: 32 and 8.5), and with the weights past LDS a
// stage's 2048 cycles of matrix instructions go with 64 KB of reads and 16 KB of writes there.  Converting
// a wave's weights takes one instruction beside every matrix instruction at four row blocks, four
// at one.
//
// 4096 tokens with 8 of 256 experts of H = 7168, I = 2048: gate_up 1.56 to 1.64 ms on several cards, its
// matrix pipe busy for 71% of them at the 1.85 GHz that the power limit leaves; down 1.00 to 1.09 ms,
// 54%: 1.06 to 1.13 PFLOP/s together.
// Tiles whose last row block holds a few rows, and prologues and epilogues with one workgroup on a CU,
// take the rest.
constexpr int kWaves = 4, kWideFN = 4;  // waves; column blocks of a wave
constexpr int kUnit = 4;                // stages of a unit
constexpr int kWideRows = 128;

// The K loop of a wave.
template <bool kGateUp, int R>
__device__ __forceinline__ void wide_k_loop(f32x16 (&acc)[R][kWideFN], const MxArgs& g,
                                            const TileRows& tr, int nt, int lane, int wave,
                                            char* smem) {
  constexpr int FN = kWideFN, kSteps = 4 * R;  // steps of a stage: instruction q, row block i
  constexpr int kUnitBytes = R * kUnit * kRowBlockBytes, kCopies = R * kUnit;  // a wave's copies
  constexpr int kAhead = 2;                    // steps from a fragment's read to its use
  const int e = __builtin_amdgcn_readfirstlane(tr.e);
  const int KB = g.blocks, units = g.quads, full = KB / kUnit;
  // Of each row block a wave copies eight rows.
  const char* rows[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    rows[i] = row_piece<kGateUp>(g, tr, 32 * i + 8 * wave + lane / Stage::CH, lane);
  // Copy t of unit u; stages past the last of K repeat that.
  auto copy = [&](int u, int t) __attribute__((always_inline)) {
    const int k = kUnit * u + t % kUnit;
    __builtin_amdgcn_global_load_lds(
        (const void*)(rows[t / kUnit] + (int64_t)(k < KB ? k : KB - 1) * Stage::ROW_BYTES),
        (lds_void*)(smem + (u & 1) * kUnitBytes + t * kRowBlockBytes + wave * 1024), 16, 0, 0);
  };
  const i32x4* b[FN];
  const uint32_t* bs[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int rb = weight_block<kGateUp, FN>(g, nt, kWaves * FN, wave * FN + j);
    b[j] = (const i32x4*)(g.B + e * g.b_expert_bytes + (int64_t)rb * KB * kFp4BlockBytes) + lane;
    bs[j] = (const uint32_t*)(g.bs + e * g.bs_expert + (int64_t)rb * units * kFp4ScaleBytes) + lane;
  }
  i32x4 w[kUnit][FN] = {};
  uint32_t sc[FN], sn[FN];           // scales of this unit's stages and of the next's
  bf16x8 wb[2][FN], frag[4];
  auto load = [&](int k, int j, i32x4& to) __attribute__((always_inline)) {
    to = b[j][(int64_t)k * (kFp4BlockBytes / 16)];
  };
  const int at = fragment_at(lane, 0);
  // step n of stage k of unit u
  auto read = [&](int u, int k, int n) __attribute__((always_inline)) {
    frag[n & 3] = *(const bf16x8*)(smem + (u & 1) * kUnitBytes + (n % R * kUnit + k) * kRowBlockBytes +
                                   (at ^ (n / R << 4)));
  };
  // operands of instruction q from stage k's weights, whose scales are s
  auto convert = [&](int k, int q, int j, uint32_t s) __attribute__((always_inline)) {
    const int v = w[k][j][q];
    wb[q & 1][j] = unpack_fp4((uint32_t)v, s >> (8 * k) & 0xffu);
  };
#pragma unroll
  for (int t = 0; t < kCopies; ++t) copy(0, t);
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
  for (int n = 0; n < kAhead; ++n) read(0, 0, n);
#pragma unroll
  for (int j = 0; j < FN; ++j) convert(0, 0, j, sc[j]);

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
    for (int n = 0; n < kSteps; ++n) {
      const int q = n / R, i = n % R;
      const int to = n + kAhead;  // the step whose fragment is read
      if (k == kUnit - 1 && to == kSteps && next) {
        // every wave has read this unit; the copies of the next, issued in the first stage, have
        // landed once at most the three stages' loads issued after them are pending
        __builtin_amdgcn_s_waitcnt(kFull ? wait_vm((kUnit - 1) * FN) : wait_vm(0));
        __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < FN; ++m) {
        acc[i][m] = MmaBf16::mma(wb[q & 1][m], frag[n & 3], acc[i][m]);
        // (the compiler moves matrix instructions down past branches, and so past the copies
        // and the barrier that they are to cover, unless their results are named before)
        asm volatile("" : "+a"(acc[i][m]));
        __builtin_amdgcn_sched_barrier(0);
        if (m == 0) {
          if (to < kSteps)
            read(u, k, to);
          else if (k < kUnit - 1)
            read(u, k + 1, to - kSteps);  // (of a stage past the last, unused)
          else if (next)
            read(u + 1, 0, to - kSteps);
        }
        // the next instruction's operands, R steps of FN slots for FN of them
        const int slot = i * FN + m;
        if (slot % R == 0) {
          if (q < 3)
            convert(k, q + 1, slot / R, sc[slot / R]);
          else
            convert((k + 1) % kUnit, 0, slot / R, k < kUnit - 1 ? sc[slot / R] : sn[slot / R]);
        }
        if (n == 0 && ahead) load(kUnit * u + k + kUnit - 1, m, w[(k + kUnit - 1) % kUnit][m]);
        if (k == 0 && m == FN - 1 && next) copy(u + 1, n);
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
  constexpr int kTile = kGateUp ? kWideRows * BN : kWideRows * (BN * 2 + BN / 64);
  constexpr int kUnits = 2 * (kWideRows / 32) * kUnit * kRowBlockBytes;
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
    __syncthreads();  // every wave is done with the rows
    if constexpr (kGateUp)
      store_tile_lds<true, 1, R, FN, 32 * R, BN, 32 * R, 32 * FN, NT>(a, acc, tr, nt, 0, R, wave, lane,
                                                                     smem);
    else
      store_out<R, FN, 32 * R, BN, NT>(a, acc, tr, nt, wave, lane, smem);
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

// ---------------------------------------------------------------- few rows an expert
// Products with up to 32 rows a tile, bound by streaming the weights: every wave reads its own
// 64 weight rows (gate_up: 32 gate rows and their up rows) straight into registers, a unit of
// four stages ahead, and no other wave reads them; only the rows of A, which the waves of a
// workgroup share, go through LDS, a unit at a time in two buffers with one barrier for it.
// Of an H = 7168, I = 2048 layer with 64 tokens on 8 of 256 experts (2 rows each) gate_up
// reads 3.4 GB in 545 to 571 us and down 1.7 in 285 to 302, 6.1 and 5.9 TB/s on average (a plain read
// of such weights: 6.8).
constexpr int kStreamWaves = 4;
// Rows an expert, on average (dropped ids count as rows: the host does not know them), up to which
// these products are taken.  That layer in ms, these and the wide ones: 1 row (an expert that has
// any) 0.44 and 0.52, 2 rows 0.89 and 0.96, 8 rows 1.08 and 1.11, 16 rows 1.12 and 1.16, 32 rows
// 1.61 and 1.31; with H = 4096, I = 1024, 128 experts 32 rows 0.26 and 0.23; with H = 2048,
// I = 1024, 64 experts 4 rows 0.065 and 0.061, 32 rows 0.084 and 0.073.
constexpr int kStreamRows = 24;

template <bool kGateUp>
__global__ void __launch_bounds__(64 * kStreamWaves) stream_mx(MxArgs a) {
  constexpr int BM = 32, FN = 2, BN = 32 * FN * kStreamWaves;
  constexpr int kUnitBytes = kUnit * kRowBlockBytes;
  static_assert(2 * kUnitBytes >= BM * BN, "act of a tile fits the rows' buffers");
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
  const int units = a.quads, KB = a.blocks;

  // Unit u of A: eight rows to a wave, nothing to one whose rows all lie past the tile's.  Stages
  // past the last of K repeat that.
  const char* rows = row_piece<kGateUp>(a, tr, 8 * wave + lane / Stage::CH, lane);
  auto copy = [&](int u) __attribute__((always_inline)) {
    if (8 * wave >= tr.rows) return;
#pragma unroll
    for (int t = 0; t < kUnit; ++t) {
      const int k = kUnit * u + t;
      __builtin_amdgcn_global_load_lds(
          (const void*)(rows + (int64_t)(k < KB ? k : KB - 1) * Stage::ROW_BYTES),
          (lds_void*)(smem + (u & 1) * kUnitBytes + t * kRowBlockBytes + wave * 1024), 16, 0, 0);
    }
  };
  const i32x4* b[FN];
  const uint32_t* bs[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int rb = weight_block<kGateUp, FN>(a, nt, kStreamWaves * FN, wave * FN + j);
    b[j] = (const i32x4*)(a.B + e * a.b_expert_bytes + (int64_t)rb * KB * kFp4BlockBytes) + lane;
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
  int at[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) at[q] = fragment_at(lane, q);
  auto stage = [&](const char* sa, auto k_tag, const i32x4 (&x)[FN]) __attribute__((always_inline)) {
    constexpr int k = decltype(k_tag)::value;
    bf16x8 row[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) row[q] = *(const bf16x8*)(sa + k * kRowBlockBytes + at[q]);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int v = x[j][q];
        acc[0][j] = MmaBf16::mma(unpack_fp4((uint32_t)v, sc[j] >> (8 * k) & 0xffu), row[q], acc[0][j]);
      }
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
    __syncthreads();  // every wave is done with the rows
    store_tile_lds<true, 1, 1, FN, BM, BN, BM, 32 * FN, 64 * kStreamWaves>(a, acc, tr, nt, 0, 1, wave,
                                                                          lane, smem);
  } else {
    store_out_rows(a, acc[0], tr, (nt * kStreamWaves + wave) * 64, lane);
  }
}

// Form, column tiles and workgroups of one product.
struct MxLaunch {
  bool stream;
  int n_tiles;
  int64_t grid;
};
MxLaunch mx_launch(bool gate_up, int64_t rows_bound, int E, int ncols) {
  MxLaunch l;
  l.stream = rows_bound <= (int64_t)kStreamRows * E;
  const int cols = (l.stream ? kStreamWaves * 64 : kWaves * kWideFN * 32) / (gate_up ? 2 : 1);
  l.n_tiles = (int)(((int64_t)ncols + cols - 1) / cols);
  l.grid = xcd_grid(m_tiles_bound(rows_bound, E, l.stream ? 32 : kWideRows), l.n_tiles);
  return l;
}

template <bool kGateUp>
hipError_t launch(MxArgs a, int64_t rows_bound, hipStream_t st) {
  if (rows_bound <= 0) return hipSuccess;
  const MxLaunch l = mx_launch(kGateUp, rows_bound, a.E, a.ncols);
  a.n_tiles = l.n_tiles;
  const dim3 grid((unsigned)l.grid);  // (in range: mx_launches_fit)
  if (l.stream)
    hipLaunchKernelGGL(stream_mx<kGateUp>, grid, dim3(64 * kStreamWaves), 0, st, a);
  else
    hipLaunchKernelGGL(grouped_gemm_mx<kGateUp>, grid, dim3(64 * kWaves), 0, st, a);
  return hipGetLastError();
}

// K columns of A; `rows` rows of an expert's weights, ncols columns of C.
MxArgs mx_args(const Shape& s, const MxIO& io, const void* rows_of_a, int K, int rows, int ncols) {
  MxArgs a{};
  a.A[0] = a.A[1] = (const char*)rows_of_a;
  a.B = (const char*)io.w;
  a.bs = (const char*)io.w_scale;
  a.off0 = io.off[0];
  a.off1 = io.off[1];
  a.E = s.E;
  a.I = s.I;
  a.ncols = ncols;
  a.row_bytes = (int64_t)K * 2;
  a.b_expert_bytes = (int64_t)rows * K / 2;
  a.bs_expert = fp4_scale_bytes(rows, K);
  a.blocks = K / kFp4BlockCols;
  a.quads = (int)fp4_scale_quads(K);
  return a;
}

}  // namespace

bool mx_launches_fit(const Shape& s, int64_t rows_bound) {
  constexpr int threads = 64 * kWaves;
  static_assert(kStreamWaves == kWaves, "one limit for both forms");
  return mx_launch(true, rows_bound, s.E, s.I).grid <= 0x7fffffff / threads &&
         mx_launch(false, rows_bound, s.E, s.H).grid <= 0x7fffffff / threads;
}

hipError_t launch_gate_up_mx(const Shape& s, const MxIO& io, const void* hidden_states, void* act,
                             hipStream_t st) {
  MxArgs a = mx_args(s, io, hidden_states, s.H, 2 * s.I, s.I);
  a.gather[0] = io.gather[0];
  a.gather[1] = io.off[1] ? io.gather[1] : io.gather[0];
  a.gather_k = s.k;
  a.up = s.I / kFp4BlockRows;
  a.C[0] = a.C[1] = (uint16_t*)act;
  return launch<true>(a, io.rows_bound, st);
}

hipError_t launch_down_mx(const Shape& s, const MxIO& io, const void* act, const ScaledRows (&y)[2],
                          hipStream_t st) {
  MxArgs a = mx_args(s, io, act, s.I, s.H, s.H);
  a.y[0] = y[0];
  a.y[1] = io.off[1] ? y[1] : y[0];
  a.c_split = io.off[1] != nullptr;
  return launch<false>(a, io.rows_bound, st);
}

}  // namespace moe
