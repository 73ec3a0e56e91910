// Grouped expert GEMMs in 8-bit integers (v_mfma_i32_32x32x32_i8), with a scale
// for each token (row of A) and each output channel (row of B):
//   g, u = a_scale[r] b_scale[c] sum_k A[r][k] B[c][k]
//   gate_up: act[r][i] = silu(g) u;   down: y[r][n] = the scaled product
//
// The sums are exact: int32 accumulators hold 131008 products of 128 * 128 (the
// entry points' limit on H and I).  They are converted to fp32 once (one
// rounding), multiplied by the row's scale, then the column's, and rounded to the
// output type once.
//
// Tiles, tile map, stages and K loops are those of the bf16 GEMMs (gemm_tile.h):
// a stage is 128 bytes of a row, here 128 values, and the int8 instruction
// takes as many bytes and as long as the bf16 one, so an int8 product streams half
// the bytes and takes half the matrix time of the bf16 product of the same sizes.
// H and I are multiples of 64, so a row may end in the middle of its last stage,
// whose second half is then cleared (clear_half).
//
// Measured: the 64-token layer of 256 experts (H = 7168, I = 2048) streams its
// weights at 6.8 TB/s (gate_up 954 us, down 483 us); 4096 tokens on them run at the
// chip's power limit, gate_up 1444 us (5.2 TB/s, 37% of the matrix pipe busy at 1.9
// GHz), down 908 us; 131072 rows of H = 2048, I = 768 reach 1.78 and 1.20 POP/s
// (463 and 343 us; a dense 8192^3 int8 product of the vendor library: 2.06).  A
// tile there spends 4 k cycles in the tile map, 46 k (gate_up, 16 stages) or 20 k
// (down, 6) in the K loop and 11 k in the epilogue, whose half is the vector ALU
// (exponential and reciprocal at a quarter of its rate).
#include <algorithm>
#include <type_traits>

#include "gemm_tile.h"

namespace moe {

namespace {

struct QuantArgs : TileArgs {
  void* C[2];            // [rows][ncols] (C[1]: chunk-1 rows when c_split)
  const float* a_scale;  // gate_up: one per row of A; down: one per joint row
  const float* b_scale;  // [E][rows of B]
};

// The scales of a tile: BM of its rows, then BN of its columns (gate_up: the
// gate columns, then the up columns).  Thread i fetches scale i before the K loop
// (one register, the latency hidden behind the loop) and leaves it in LDS after
// it, where the epilogue's lanes find the ones they need: fetched in the
// epilogue, a lane's 36 scales pushed the accumulators out of the registers.
template <bool kGateUp, int BM, int BN>
__device__ __forceinline__ float fetch_scale(const QuantArgs& a, const TileRows& tr, int nt,
                                             int i) {
  if (i < BM) {
    // rows past the tile are never stored
    const int v = tr.v0 + (i < tr.rows ? i : tr.rows - 1);
    if constexpr (!kGateUp) return a.a_scale[tr.joint_row(v)];
    int part;
    const int cr = tr.split_row(v, &part);
    const int32_t *g0 = a.gather[0], *g1 = a.gather[1];
    return a.a_scale[(part ? g1 : g0)[cr] / a.gather_k];
  }
  i -= BM;
  if (i >= BN) return 0.0f;
  const int e = __builtin_amdgcn_readfirstlane(tr.e);
  if constexpr (kGateUp) {
    const int q = i / (BN / 2), c = i % (BN / 2);
    return a.b_scale[((int64_t)e * 2 + q) * a.I + nt * (BN / 2) + c];
  } else {
    const int c = nt * BN + i;  // columns past C are never stored
    return a.b_scale[(int64_t)e * a.ncols + (c < a.ncols ? c : a.ncols - 1)];
  }
}

// Epilogue.  Lane l holds row l % 32 of each 32 x 32 block and its columns
// 8 (q / 4) + 4 (l / 32) + q % 4, q = 0..15, so a lane needs one row scale per
// block and four consecutive column scales per group of four accumulators.  The
// tile goes through the freed stage buffers, row-major, and leaves as 16-byte row
// segments.  (Stored from the registers instead, 32 bytes of a row at a time: the
// packed 16k down GEMM 352 -> 411 us, partial lines.)
template <bool kGateUp, bool kBf16, int FM, int FN, int BM, int BN, int WM, int WN, int NT>
__device__ __forceinline__ void store_tile_i8(const QuantArgs& a, const i32x16 (&acc)[FM][FN],
                                              const TileRows& tr, int nt, int row0, int nblk,
                                              int wn, int lane, char* smem,
                                              const float* scales) {
  typedef std::conditional_t<kBf16, uint16_t, float> out_t;
  constexpr int ES = sizeof(out_t), EV = 16 / ES;  // bytes of an element, elements of 16 bytes
  constexpr int CT = kGateUp ? BN / 2 : BN;        // tile columns of C
  constexpr int CPR = CT / EV;                     // 16-byte chunks per tile row
  static_assert(CPR >= 8, "chunk swizzle needs 8 chunks per row");
  // chunk ch of row r at slot ch ^ (r mod CPR): the 32 rows of one write fall in
  // distinct slots
  auto lds_at = [](int r, int c) {
    return r * (CT * ES) + (((c / EV) ^ (r & (CPR - 1))) << 4) + (c % EV) * ES;
  };
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  constexpr int FC = kGateUp ? FN / 2 : FN;  // 32-column blocks of C
  constexpr int CW = kGateUp ? WN / 2 : WN;  // columns of C per wave column
  const int cq = 4 * (lane >> 5), col0 = nt * CT;
  const float* row_scale = scales + row0 + (lane & 31);
  const float* col_scale = scales + BM;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if (i >= nblk || row0 + i * 32 >= tr.rows) break;
    const int r = row0 + i * 32 + (lane & 31);
    const float rs = row_scale[i * 32];
#pragma unroll
    for (int j = 0; j < FC; ++j)
#pragma unroll
      for (int g4 = 0; g4 < 4; ++g4) {
        const int c = wn * CW + j * 32 + 8 * g4 + cq;
        const float4 s0 = *(const float4*)(col_scale + c);
        const float cs[4] = {s0.x, s0.y, s0.z, s0.w};
        float v[4];
        if constexpr (kGateUp) {
          const float4 s1 = *(const float4*)(col_scale + CT + c);
          const float us[4] = {s1.x, s1.y, s1.z, s1.w};
#pragma unroll
          for (int t = 0; t < 4; ++t)
            v[t] = swiglu<kBf16>((float)acc[i][j][4 * g4 + t] * rs * cs[t],
                          (float)acc[i][j + FC][4 * g4 + t] * rs * us[t]);
        } else {
#pragma unroll
          for (int t = 0; t < 4; ++t) v[t] = (float)acc[i][j][4 * g4 + t] * rs * cs[t];
        }
        if constexpr (kBf16)
          *(bf16x4*)(smem + lds_at(r, c)) =
              bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
        else
          *(float4*)(smem + lds_at(r, c)) = make_float4(v[0], v[1], v[2], v[3]);
      }
  }
  __syncthreads();
  const out_t* const cbase[2] = {(const out_t*)a.C[0], (const out_t*)a.C[1]};
  for (int ch = threadIdx.x; ch < BM * CPR; ch += NT) {
    const int r = ch / CPR, c = (ch % CPR) * EV;
    if (r >= tr.rows || col0 + c >= a.ncols) continue;
    const u32x4 v = *(const u32x4*)(smem + lds_at(r, c));
    out_t* dst = (out_t*)row_ptr(cbase, a.c_split, tr, tr.v0 + r, a.ncols);
    // streamed (gate_up's act kept in the caches for the quantiser measured 4%
    // slower over the DeepSeek-V3-shaped layer)
    __builtin_nontemporal_store(v, (u32x4*)(dst + col0 + c));
  }
}

// As grouped_gemm_bf16: kLoop workgroups take tile after tile of their XCD's
// sequence, the others exactly one.
template <bool kGateUp, bool kBf16, int BM, int BN, int WAVES_M, int WAVES_N, int SB, int STAGES,
          bool kBuf, bool kLoop>
__global__ void __launch_bounds__(64 * WAVES_M * WAVES_N) grouped_gemm_i8(QuantArgs a) {
  constexpr int NW = WAVES_M * WAVES_N;
  constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  constexpr int FM = WM / 32, FN = WN / 32;
  using Loader = TileLoader<MmaI8, kGateUp, BM, BN, NW, WN, SB, kBuf>;
  constexpr bool kRoles = NW == 8;
  using RoleLoader = TileLoader<MmaI8, kGateUp, BM, BN, kRoles ? NW / 2 : NW, WN, SB, kBuf>;
  static_assert(WM % 32 == 0 && WN % 32 == 0, "wave tile");
  static_assert(!kGateUp || WN % 64 == 0, "gate/up halves");
  static_assert(STAGES >= 2, "pipeline depth");
  static_assert((STAGES - 1) * (Loader::LA + Loader::LB) <= 24, "wait_loads range");
  constexpr int kSmemBytes =
      cmax(kRoles ? 2 * Loader::A_BYTES + 3 * Loader::B_BYTES : STAGES * Loader::STAGE_BYTES,
           FM >= 4 ? cmax(3 * Loader::template small_stage<160>(),
                          cmax(3 * Loader::template small_stage<32>(),
                               3 * Loader::template small_stage<64>()))
                   : 0);
  __shared__ __attribute__((aligned(1024))) char smem[kSmemBytes];

  const int lane0 = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  const int xcd = blockIdx.x & 7, wg_per_xcd = gridDim.x >> 3;
  for (int q = blockIdx.x >> 3;; q += wg_per_xcd) {
    // an opaque copy of the lane per tile keeps lane-derived addresses from
    // staying live across the tile loop
    int lane = lane0;
    if constexpr (kLoop) asm volatile("" : "+v"(lane));
    MTileMap tm;
    tm.build(a.off0, a.off1, a.E, BM, BM >= 128 ? BM : 1);
    int mt, nt;
    if (!xcd_tile_at(tm, a.n_tiles, xcd, q, (32 + a.n_tiles - 1) / a.n_tiles, &mt, &nt)) break;
    const TileRows tr = tm.locate(a.off0, a.off1, BM, mt);

    static_assert(BM + BN <= 64 * NW, "a scale per thread");
    const float scale = fetch_scale<kGateUp, BM, BN>(a, tr, nt, wave * 64 + lane);

    i32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = i32x16{};

    const int KT = (int)((a.row_bytes + SB - 1) / SB);
    constexpr bool kSmallPath = FM >= 4 && WAVES_M == 2;
    // a panel that one tile alone reads is streamed non-temporally
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
        wide_k<FM, FN, WM, WN, BM, SB, STAGES, kNt, true, RoleLoader>(acc, ld, smem, KT, 0, lane,
                                                                      wm, wn, tr.rows);
      } else {
        Loader ld;
        ld.init(a, tr, nt, lane, wave);
        const int per_stage = ld.live_a + Loader::LB;
        wide_k<FM, FN, WM, WN, BM, SB, STAGES, kNt, false, Loader>(acc, ld, smem, KT, per_stage,
                                                                   lane, wm, wn, tr.rows);
      }
#undef MOE_K_SMALL
    };
    if (tr.single)
      run_k(std::true_type{});
    else
      run_k(std::false_type{});
    // the freed stage buffers hold the C tile, then the scales
    constexpr int kScales = BM * (kGateUp ? BN / 2 : BN) * (kBf16 ? 2 : 4);
    static_assert(kScales + (BM + BN) * 4 <= kSmemBytes, "C tile and scales fit the buffers");
    __syncthreads();  // every wave is done with the stage buffers
    float* scales = (float*)(smem + kScales);
    if (wave * 64 + lane < BM + BN) scales[wave * 64 + lane] = scale;
    __syncthreads();
    int band0 = wm * WM, nblk = FM;
    if constexpr (kSmallPath) {
      if (tr.rows <= 160) {
        const bool spread = tr.single != 0;
        const int f0 = compact_f0(tr.rows, spread);
        band0 = wm * f0 * 32;
        nblk = wm == 0 ? f0 : compact_f1(tr.rows, spread);
      }
    }
    store_tile_i8<kGateUp, kBf16, FM, FN, BM, BN, WM, WN, 64 * NW>(a, acc, tr, nt, band0, nblk, wn,
                                                                   lane, smem, scales);
    if constexpr (!kLoop) break;
    __syncthreads();  // the C tile has left LDS before the next tile's stage loads
  }
}

// The 256 x 256 tile (its loop for up to 160 rows included) or the 64 x 128 one, for
// bf16 output.  The large tile reads an expert's weights once for up to 256 rows;
// the small one starts and ends in less time, fills the chip with fewer columns,
// and wins while most experts fit its 64 rows (times in us, large / small):
//   E = 16, K = 4096 and 2048, 200 rows an expert: 80 / 136 and 45 / 67; 32: 64 / 60, 26 / 24
//   E = 128, K = 2048 and 768, 128 rows: 102 / 125 and 76 / 70; 32: 78 / 71, 56 / 45
//   E = 256, K = 7168 and 2048, 64 rows: 1302 / 1611 and 781 / 880; 8: 1103 / 1083, 628 / 586
//   E = 8, K = 2048 and 1408 (88 and 64 large tiles), 200 rows: 30 / 22 and 23 / 13
// So: at least 64 rows an expert on average, K of 2048 or more and a large tile for
// every CU.  From 4096 rows on always the large one: the counts are known only on
// the device, and when two of 256 experts get 8000 rows between them the small one
// takes about twice as long.  What that loses on even counts is a seventh where large
// tiles fill the chip, and up to half where few experts with few column tiles make less
// than one for every CU (E = 8 and 16 alike, gate_up / down, large against small):
//   H = 2048, I = 256:  4096 rows 29 / 13 against 15 / 12;  8192: 29 / 24 against 20 / 18;
//                      16384: 31 / 36 against 33 / 32
//   H = 512, I = 2048:  4096 rows 30 / 27 against 26 / 14;  8192: 45 / 28 against 44 / 20;
//                      16384: 76 / 30 against 81 / 32
bool prefer_wide(const QuantArgs& a, int64_t rows_bound, int n_tiles) {
  if (rows_bound >= 4096) return true;
  return rows_bound >= 64 * (int64_t)a.E && a.row_bytes >= 2048 &&
         (int64_t)a.E * n_tiles >= 256;
}

template <bool kGateUp, bool kBf16, int BM, int BN, int WM_, int WN_, bool kBuf>
hipError_t launch_instance(QuantArgs a, const Shape& s, int64_t rows_bound, hipStream_t st) {
  constexpr int threads = 64 * WM_ * WN_;
  a.n_tiles = kGateUp ? s.I / (BN / 2) : (s.H + BN - 1) / BN;
  const int64_t grid = xcd_grid(m_tiles_bound(rows_bound, s.E, BM), a.n_tiles);
  if (grid <= 0) return hipSuccess;
  if (grid > 0x7fffffff / threads) return hipErrorInvalidConfiguration;
  // few active experts out of many: the tile bound far exceeds what the rows can
  // fill, and the wide tile's workgroups take several tiles each (as in bf16)
  if constexpr (BM == 256 && kBuf) {
    const int64_t cap = 8 * std::max<int64_t>(128, 2 * ((rows_bound / BM + 7) / 8) * a.n_tiles);
    if (2 * cap < grid) {
      hipLaunchKernelGGL((grouped_gemm_i8<kGateUp, kBf16, BM, BN, WM_, WN_, 128, 2, kBuf, true>),
                         dim3((unsigned)cap), dim3(threads), 0, st, a);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((grouped_gemm_i8<kGateUp, kBf16, BM, BN, WM_, WN_, 128, 2, kBuf, false>),
                     dim3((unsigned)grid), dim3(threads), 0, st, a);
  return hipGetLastError();
}

template <bool kGateUp, bool kBuf>
hipError_t launch_kind(const QuantArgs& a, const Shape& s, int64_t rows_bound, hipStream_t st) {
  if (s.dtype != MOE_BF16)
    return launch_instance<kGateUp, false, 64, 128, 2, 2, kBuf>(a, s, rows_bound, st);
  // a 256-column gate_up tile holds 128 intermediate columns
  const bool wide_ok = !kGateUp || s.I % 128 == 0;
  const int n_tiles = kGateUp ? s.I / 128 : (s.H + 255) / 256;
  if (wide_ok && prefer_wide(a, rows_bound, n_tiles))
    return launch_instance<kGateUp, true, 256, 256, 2, 4, kBuf>(a, s, rows_bound, st);
  return launch_instance<kGateUp, true, 64, 128, 2, 2, kBuf>(a, s, rows_bound, st);
}

template <bool kGateUp>
hipError_t launch(const Shape& s, const GroupedIO& io, const float* a_scale, const void* B,
                  const float* b_scale, hipStream_t st) {
  if (io.rows_bound <= 0) return hipSuccess;
  QuantArgs a{};
  a.A[0] = a.A[1] = (const char*)io.a[0];
  a.C[0] = io.c[0];
  a.C[1] = io.c_split ? io.c[1] : io.c[0];
  a.off0 = io.off[0];
  a.off1 = io.off[1];
  a.c_split = io.c_split && io.off[1];
  a.gather[0] = io.gather[0];
  a.gather[1] = io.off[1] ? io.gather[1] : io.gather[0];
  a.gather_k = io.gather_k;
  a.B = (const char*)B;
  a.E = s.E;
  a.I = s.I;
  a.a_scale = a_scale;
  a.b_scale = b_scale;
  a.row_bytes = kGateUp ? s.H : s.I;
  a.ncols = kGateUp ? s.I : s.H;
  a.b_expert_bytes = (kGateUp ? (int64_t)2 * s.I : (int64_t)s.H) * a.row_bytes;
  a.a_base = a.A[0];
  // descriptor loads take 32-bit offsets: the A rows and an expert's weights each
  // have to lie within 4 GiB (2-byte elements are what rows_fit_4g counts)
  const bool buf = rows_fit_4g(a.A[0], a.A[0], kGateUp ? s.T : io.rows_bound, a.row_bytes / 2) &&
                   (uint64_t)a.b_expert_bytes < ((uint64_t)1 << 32);
  return buf ? launch_kind<kGateUp, true>(a, s, io.rows_bound, st)
             : launch_kind<kGateUp, false>(a, s, io.rows_bound, st);
}

}  // namespace

hipError_t launch_gate_up_i8(const Shape& s, const GroupedIO& io, const float* a_scale,
                             const void* w_gate_up, const float* w_scale, hipStream_t st) {
  return launch<true>(s, io, a_scale, w_gate_up, w_scale, st);
}

hipError_t launch_down_i8(const Shape& s, const GroupedIO& io, const float* a_scale,
                          const void* w_down, const float* w_scale, hipStream_t st) {
  return launch<false>(s, io, a_scale, w_down, w_scale, st);
}

}  // namespace moe
