// Grouped expert GEMMs on gfx950 bf16 matrix cores (v_mfma_f32_32x32x16_bf16).
//
// The expert computation of the MindSpeed Chunk MoE article (core principle /
// timing-diagram sections) is read as a SwiGLU FFN per expert; each expert
// multiplies its block of permuted rows:
//   gate_up: act[r][i] = silu(x_r . Wg[e][i]) * (x_r . Wu[e][i])   (K = H)
//   down   : y[r][n]   = act_r . Wd[e][n]                          (K = I)
// Both operands are K-contiguous ([rows][K] activations, [cols][K] weights).
// One launch covers one chunk or both chunks of a pair (GroupedIO): an
// expert's rows are its rows in the first chunk followed by its rows in the
// second, so its weights are streamed once per launch.  gate_up may read its
// rows straight from hidden_states through src_row (GroupedIO::gather): the
// permute fused into the A loader's addresses.
//
// (Stage loads and K loops, shared with the int8 GEMMs, are in gemm_tile.h.)
//
// Pipeline: K advances 64 at a time.  Each stage of the A (rows) and B
// (weight) tiles is copied HBM -> LDS by the direct-to-LDS load (64 lanes x 16
// bytes land as one contiguous 1 KB block), so loads need no VGPRs and
// STAGES-1 stages are in flight while the matrix cores work on the oldest one
// (the wide 256 x 256 kernel: two A stages and three B stages, k_loop_roles).
// The buffer form of that load (a descriptor per operand, 32-bit offsets) is
// used whenever the rows fit a 4 GiB window: with the global form, a FLAT
// instruction, in flight, the compiler drains every LDS read before each MFMA
// group; with descriptors it waits only for the fragments in use, and each
// 16-deep sub-step's fragment reads overlap the previous sub-step's MFMAs
// (gate/up 4-6% faster on the MFMA-bound workloads).  Completion is tracked
// with explicit vmcnt waits plus a plain s_barrier (no fence that would drain
// every load).  LDS rows are XOR-swizzled (StageGeom) so that 16-byte fragment
// reads are free of bank conflicts (measured).
//
// Matrix instruction: on gfx950 v_mfma_f32_32x32x16_bf16 and
// v_mfma_f32_16x16x32_bf16 both occupy the matrix pipe for about 32 cycles, so
// only the 32x32x16 form reaches the chip's dense bf16 peak (measured 2.47
// versus 1.26 PFLOP/s with back-to-back independent MFMAs); every tile here is
// built from 32 x 32 blocks.
//
// Tiling: a workgroup computes BM x BN with WAVES_M x WAVES_N waves; each wave
// owns (BM/WAVES_M) x (BN/WAVES_N) as 32 x 32 MFMA blocks with fp32
// accumulators.  For gate_up half of every wave's columns are gate columns and
// the other half the matching up columns, so each lane holds the gate and up
// accumulators of the same (row, i) and SwiGLU runs in registers: no
// [rows][2I] intermediate is written.
//
// Grouping: every workgroup numbers the m-tiles of all experts from the
// device-resident offsets (MTileMap: the large experts' m-tiles first, then
// the small experts' by size class), so the host never reads group sizes.
// Each XCD takes a contiguous range of the large experts' m-tiles and an even
// share of the small ones, interleaved, each with all its n-tiles (xcd_tile).
// The grid is bounded from the launch's assignment count and surplus
// workgroups exit.  Rows past an expert's block are loaded from a clamped row
// (A blocks wholly past it are not loaded at all) and never stored.
//
// Epilogue: the accumulators go through the freed stage buffers as a
// row-major bf16 tile and leave as 16-byte row segments (store_tile_lds).
//
// Small tiles: an m-tile of at most 32, 64, 128 or 160 rows (a small expert's
// only tile) has little MFMA work and is bound by streaming its weight panel, so
// it runs a K loop with a compact stage layout (its rows of A, then B) and three
// stages, two in flight (k_loop_small): 41 -> 33 us per gate/up tile of at most
// 32 rows on the Zipf workload; the 160-row case (three 52 KB stages, 156 KB of
// LDS) took the DeepSeek-V3-shaped layer, whose experts hold 95-160 rows, from
// 4.89 to 4.79 ms (down 1724 -> 1683 us).  When such a tile holds all of its
// expert's rows its 32-row blocks are split between the two wave rows
// (compact_f0 / compact_f1), so that both waves on each SIMD run MFMAs.
//
// Also measured and dropped, on these launches: a persistent form (one
// workgroup per CU taking its XCD's tiles in sequence, the next tile's first
// stages loaded during the current tile's last steps), for weight-streaming
// and for MFMA-bound launches; two workgroups per CU with 32-deep stages; K
// stages rotated per expert.  The hardware's dynamic dispatch of one-tile
// workgroups balances the tiles better than any fixed sequence per CU.
//
// What bounds it (measured with per-workgroup timestamps): the MFMA loop alone
// (no global loads) runs at ~94% of the matrix peak at the clock it gets, and
// adding the LDS fragment reads costs nothing.  With the operand streaming on
// top, the chip's power management lowers the shader clock (about 2.2 GHz ->
// 1.5-2.1 GHz) and a full 256 x 256 tile takes ~1.45x the cycles of its MFMAs.
// Per-K-step timestamps place the loss at the start of each step: a load
// instruction holds its wave until the texture unit takes it, so while the
// eight waves issued a 64 KB stage no MFMA ran for 800-1150 of ~3300 cycles.
// The wide 256 x 256 kernel therefore gives the two waves of a SIMD different
// load roles (k_loop_roles, with a third weight buffer): 3280 -> 2875 cycles
// per step, of which the power limit returns part as a lower clock (layer
// 2-3% faster on packed16k, the Zipf workload and, in the tile-loop form, the
// two-expert skew; same bits).  Alone, a third
// weight buffer, loads spread over the sub-steps, one wave row issuing every
// load, BK 32 with 4-5 stages, a 256 x 128 tile with three stages,
// register-staged loads, round-robin XCD dealing of all m-tiles and 4-wave
// 128 x 128 wave tiles all measured no faster.  What did help besides: a K
// loop whose body holds no branch, with the wave's count of live 32-row blocks
// chosen once before the loop (5-12% on the larger workloads); the
// size-balanced, interleaved tile order (xcd_tile); the staged epilogue; the
// compact small-tile loop.
#include <algorithm>
#include <type_traits>

#include "gemm_tile.h"

namespace moe {

namespace {

// kLoop: the workgroup takes tile after tile of its XCD's sequence (launched
// when the grid is capped below the tile bound); otherwise exactly one.
template <bool kGateUp, bool kSaveGU, int BM, int BN, int WAVES_M, int WAVES_N, int SB,
          int STAGES, bool kBuf, bool kLoop>
__global__ void __launch_bounds__(64 * WAVES_M * WAVES_N) grouped_gemm_bf16(GemmArgs a) {
  constexpr int NW = WAVES_M * WAVES_N;
  constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  constexpr int FM = WM / 32, FN = WN / 32;
  using Loader = TileLoader<MmaBf16, kGateUp, BM, BN, NW, WN, SB, kBuf>;
  // the wide kernel splits the loads by wave role (k_loop_roles)
  constexpr bool kRoles = NW == 8;
  using RoleLoader =
      TileLoader<MmaBf16, kGateUp, BM, BN, kRoles ? NW / 2 : NW, WN, SB, kBuf>;
  static_assert(WM % 32 == 0 && WN % 32 == 0, "wave tile");
  static_assert(!kGateUp || WN % 64 == 0, "gate/up halves");
  static_assert(STAGES >= 2, "pipeline depth");
  static_assert((STAGES - 2) * (Loader::LA + Loader::LB) <= 24, "wait_loads range");
  constexpr int kSmemBytes =
      cmax(kRoles ? 2 * Loader::A_BYTES + 3 * Loader::B_BYTES : STAGES * Loader::STAGE_BYTES,
           FM >= 4 ? cmax(3 * Loader::template small_stage<160>(),
                          cmax(3 * Loader::template small_stage<32>(),
                               3 * Loader::template small_stage<64>()))
                   : 0);
  __shared__ __attribute__((aligned(1024))) char smem[kSmemBytes];

  const int lane0 = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  // Tiles of this workgroup: position q of its XCD's sequence, and with kLoop
  // also q + G, q + 2G, ... (G = the XCD's workgroups: the host then launches
  // fewer workgroups than the tile bound, so that a launch whose row count
  // allows many more tiles than the routing produced does not dispatch
  // thousands of workgroups that find none).
  const int xcd = blockIdx.x & 7, wg_per_xcd = gridDim.x >> 3;
  for (int q = blockIdx.x >> 3;; q += wg_per_xcd) {
    // In the tile loop the compiler hoisted every lane-derived address (loader
    // offsets, fragment offsets) out of the loop and kept them all live: 256
    // VGPRs and spills.  An opaque copy of the lane index per tile keeps them
    // inside (238 VGPRs, no VGPR spills with the load roles).
    int lane = lane0;
    if constexpr (kLoop) asm volatile("" : "+v"(lane));
    // (built per tile: kept across the K loop it would cost registers)
    MTileMap tm;
    // the wide tile (one workgroup per CU) orders small experts' m-tiles by size
    // to balance the XCDs; the narrow tile (three per CU) keeps expert order,
    // which mixes weight-streaming and MFMA-bound tiles on a CU (measured faster)
    tm.build(a.off0, a.off1, a.E, BM, BM >= 128 ? BM : 1);
    int mt, nt;
    if (!xcd_tile_at(tm, a.n_tiles, xcd, q, (32 + a.n_tiles - 1) / a.n_tiles, &mt, &nt)) break;
    const TileRows tr = tm.locate(a.off0, a.off1, BM, mt);

    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};

    const int KT = (int)(a.row_bytes / SB);
    // tiles of at most 32, 64, 128 or 160 rows: three compact stages (a fourth
    // stage for the 32-row tiles, in 16 KB more LDS, measured no faster; the
    // 128-row case, 144 KB, took the DeepSeek-V3-shaped layer's gate/up from 3.18
    // to 3.01 ms, its experts holding 95-160 rows each, and the 160-row case,
    // 156 KB, the layer from 4.89 to 4.79 ms)
    constexpr bool kSmallPath = FM >= 4 && WAVES_M == 2;
    // The weight panel of a tile that holds all of its expert's rows is read by
    // no other tile of the launch, so it is streamed non-temporally (decode
    // 3.28 -> 2.95 ms with the stores below); panels shared by several m-tiles
    // of one expert stay cached (non-temporal there cost the two-expert skew 13%).
    auto run_k = [&](auto nt_tag) __attribute__((always_inline)) {
    constexpr bool kNt = decltype(nt_tag)::value;
#define MOE_K_SMALL(SR)                                                                          \
  do {                                                                                           \
    constexpr int F0 = compact_f0(SR, kNt), F1 = compact_f1(SR, kNt);                            \
    if (wm == 0)                                                                                 \
      k_loop_small<F0, SR, 3, FM, FN, WN, SB, kNt, Loader>(acc, ld, smem, KT, per_stage, lane,   \
                                                           wn, 0);                               \
    else                                                                                         \
      k_loop_small<F1, SR, 3, FM, FN, WN, SB, kNt, Loader>(acc, ld, smem, KT, per_stage, lane,   \
                                                           wn, F0 * 32);                         \
  } while (0)
    if (kSmallPath && tr.rows <= 160) {
      if constexpr (kSmallPath) {
        Loader ld;
        ld.init(a, tr, nt, lane, wave);
        const int per_stage = ld.live_a + Loader::LB;  // loads this wave issues per stage
        if (tr.rows <= 32)
          MOE_K_SMALL(32);
        else if (tr.rows <= 64)
          MOE_K_SMALL(64);
        else if (tr.rows <= 128)
          MOE_K_SMALL(128);
        else
          MOE_K_SMALL(160);
      }
    } else if constexpr (kRoles) {
      RoleLoader ld;
      ld.init(a, tr, nt, lane, wave % (NW / 2));
      wide_k<FM, FN, WM, WN, BM, SB, STAGES, kNt, true, RoleLoader>(acc, ld, smem, KT, 0, lane, wm,
                                                                    wn, tr.rows);
    } else {
      Loader ld;
      ld.init(a, tr, nt, lane, wave);
      const int per_stage = ld.live_a + Loader::LB;
      wide_k<FM, FN, WM, WN, BM, SB, STAGES, kNt, false, Loader>(acc, ld, smem, KT, per_stage, lane,
                                                                 wm, wn, tr.rows);
    }
#undef MOE_K_SMALL
    };
    if (tr.single)
      run_k(std::true_type{});
    else
      run_k(std::false_type{});
    static_assert(BM * (kGateUp ? BN / 2 : BN) * 2 <= STAGES * Loader::STAGE_BYTES,
                  "C tile fits the stage buffers");
    __syncthreads();  // every wave is done with the stage buffers
    // this wave's rows: its wave row's WM on the wide path, the compact split
    // (recomputed here so that nothing more stays live across the K loop)
    int band0 = wm * WM, nblk = FM;
    if constexpr (kSmallPath) {
      if (tr.rows <= 160) {
        const bool spread = tr.single != 0;
        const int f0 = compact_f0(tr.rows, spread);
        band0 = wm * f0 * 32;
        nblk = wm == 0 ? f0 : compact_f1(tr.rows, spread);
      }
    }
    store_tile_lds<kGateUp, kSaveGU ? 3 : 1, FM, FN, BM, BN, WM, WN, 64 * NW>(a, acc, tr, nt, band0,
                                                                             nblk, wn, lane, smem);
    if constexpr (!kLoop) break;
    __syncthreads();  // the C tile has left LDS before the next tile's stage loads
  }
}

// Tile instances.  Both use the same MFMA instruction and the same order of
// K steps, so either gives the same bits for a row; the choice only affects
// speed.  The wide 256 x 256 tile (8 waves, one workgroup per CU) moves the
// fewest bytes per MFMA; the 64 x 128 tile (three workgroups per CU) wins on
// small launches.  A compile-time override forces one instance.
enum Instance { kAuto = 0, kWide = 1, kNarrow = 2 };
#ifndef MOE_GEMM_FORCE
#define MOE_GEMM_FORCE 0
#endif

// With the small-tile loop and the size-balanced tile order the wide tile also
// wins on launches of a few thousand rows with short expert blocks (8192 rows
// over 54 experts: gate/up 145 against 158 us, down 84 against 100 us); the
// narrow one still wins on decode-sized launches (512 rows), which are pure
// weight streaming.
bool prefer_wide(int64_t rows_bound) { return rows_bound >= 4096; }

template <bool kGateUp, bool kSaveGU, int BM, int BN, int WM_, int WN_, int SB, int ST,
          bool kBuf>
hipError_t launch_instance(GemmArgs a, const Shape& s, int64_t rows_bound, hipStream_t st) {
  constexpr int threads = 64 * WM_ * WN_;
  // gate_up tiles cover BN/2 intermediate columns (gate and up halves)
  a.n_tiles = kGateUp ? s.I / (BN / 2) : (s.H + BN - 1) / BN;
  const int64_t grid = xcd_grid(m_tiles_bound(rows_bound, s.E, BM), a.n_tiles);
  if (grid <= 0) return hipSuccess;
  if (grid > 0x7fffffff) return hipErrorInvalidConfiguration;
  // The bound counts a partial m-tile for each of up to E experts.  When that
  // far exceeds what the rows can fill (few active experts out of many), each
  // surplus workgroup still costs a dispatch of the whole tile's waves and
  // LDS (the two-expert E = 256 launch: 4096 of 4608), so the wide tile caps
  // each XCD at twice its full-tile positions (at least 128 workgroups) and
  // its workgroups take several tiles each: gate/up 410 -> 395 us and down
  // 265 -> 257 us on that launch.  Only where the cap removes more than half
  // the grid: elsewhere the tile loop, with its larger register footprint,
  // measured 0-2% slower than the one-tile kernel.
  if constexpr (BM == 256 && kBuf) {
    const int64_t cap = 8 * std::max<int64_t>(128, 2 * ((rows_bound / BM + 7) / 8) * a.n_tiles);
    if (2 * cap < grid) {
      hipLaunchKernelGGL((grouped_gemm_bf16<kGateUp, kSaveGU, BM, BN, WM_, WN_, SB, ST, kBuf, true>),
                         dim3((unsigned)cap), dim3(threads), 0, st, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((grouped_gemm_bf16<kGateUp, kSaveGU, BM, BN, WM_, WN_, SB, ST, kBuf, false>),
                     dim3((unsigned)grid), dim3(threads), 0, st, a);
  return hipGetLastError();
}

template <bool kGateUp, bool kSaveGU, bool kBuf>
hipError_t launch_kind(int inst, GemmArgs a, const Shape& s, int64_t rows_bound, hipStream_t st) {
  // a 256-column gate_up tile holds 128 intermediate columns
  const bool wide_ok = !kGateUp || s.I % 128 == 0;
  if (inst == kAuto) {
    inst = prefer_wide(rows_bound) ? kWide : kNarrow;
  }
  if (inst == kWide && wide_ok)
    return launch_instance<kGateUp, kSaveGU, 256, 256, 2, 4, 128, 2, kBuf>(a, s, rows_bound, st);
  return launch_instance<kGateUp, kSaveGU, 64, 128, 2, 2, 128, 2, kBuf>(a, s, rows_bound, st);
}

template <bool kGateUp, bool kSaveGU>
hipError_t launch_kind(bool buf, int inst, GemmArgs a, const Shape& s, int64_t rows_bound,
                       hipStream_t st) {
  return buf ? launch_kind<kGateUp, kSaveGU, true>(inst, a, s, rows_bound, st)
             : launch_kind<kGateUp, kSaveGU, false>(inst, a, s, rows_bound, st);
}

// Descriptor loads take 32-bit byte offsets: every A row (a row of
// hidden_states when gathered, else of one or both row buffers, each bounded
// by the launch's rows) must lie within 4 GiB above the lower base, and each
// expert's weight block within 4 GiB of its start.  Sets a.a_base.
bool descriptor_loads_fit(GemmArgs& a, const Shape& s, int64_t rows_bound) {
  const char* a1 = a.a_split ? a.A[1] : a.A[0];
  a.a_base = std::min(a.A[0], a1);
  return rows_fit_4g(a.A[0], a1, a.gather[0] ? s.T : rows_bound, a.row_bytes / 2) &&
         (uint64_t)a.b_expert_bytes < ((uint64_t)1 << 32);
}

hipError_t launch(bool gate_up, const Shape& s, const GroupedIO& io, const void* B,
                  hipStream_t st) {
  const int64_t rows_bound = io.rows_bound;
  if (rows_bound <= 0) return hipSuccess;
  GemmArgs a{};
  a.A[0] = (const char*)io.a[0];
  a.A[1] = (const char*)(io.a_split ? io.a[1] : io.a[0]);
  a.C[0] = (uint16_t*)io.c[0];
  a.C[1] = (uint16_t*)(io.c_split ? io.c[1] : io.c[0]);
  a.off0 = io.off[0];
  a.off1 = io.off[1];
  a.a_split = io.a_split && io.off[1];
  a.c_split = io.c_split && io.off[1];
  a.gu = gate_up ? (uint16_t*)io.gu : nullptr;
  a.gather[0] = gate_up ? io.gather[0] : nullptr;
  a.gather[1] = gate_up && io.off[1] ? io.gather[1] : a.gather[0];
  a.gather_k = io.gather_k;
  a.B = (const char*)B;
  a.E = s.E;
  a.I = s.I;
  const int inst = MOE_GEMM_FORCE;
  if (gate_up) {
    a.row_bytes = (int64_t)s.H * 2;
    a.ncols = s.I;
    a.b_expert_bytes = (int64_t)2 * s.I * s.H * 2;
    // the backward's recompute also saves g and u (its own instance, so the
    // forward kernel keeps its registers)
    const bool buf = descriptor_loads_fit(a, s, rows_bound);
    if (a.gu) return launch_kind<true, true>(buf, inst, a, s, rows_bound, st);
    return launch_kind<true, false>(buf, inst, a, s, rows_bound, st);
  }
  a.row_bytes = (int64_t)s.I * 2;
  a.ncols = s.H;
  a.b_expert_bytes = (int64_t)s.H * s.I * 2;
  const bool buf = descriptor_loads_fit(a, s, rows_bound);
  return launch_kind<false, false>(buf, inst, a, s, rows_bound, st);
}

}  // namespace

hipError_t launch_gate_up_bf16(const Shape& s, const GroupedIO& io, const void* w_gate_up,
                               hipStream_t st) {
  return launch(true, s, io, w_gate_up, st);
}

hipError_t launch_down_bf16(const Shape& s, const GroupedIO& io, const void* w_down,
                            hipStream_t st) {
  return launch(false, s, io, w_down, st);
}

}  // namespace moe
