// Grouped expert GEMMs with bf16 rows and packed 4-bit weights (fp4_layout.h):
//   gate_up: act[r][i] = silu(g) u,  g, u = x_r . W[e][i], x_r . W[e][I + i]
//   down   : y[r][n]   = act_r . W[e][n]
// A weight is an E2M1 number times a power of two, which bf16 holds exactly, so the
// products are those of the bf16 GEMMs with the weights written out: bf16 matrix
// instructions, fp32 sums over K in ascending order whatever the tile (the same bits
// from every variant), one rounding of the result.
//
// The weights stay in 4 bits until they are operands: a stage of 64 columns is copied
// to LDS as it lies in memory, a kilobyte for 32 weight rows, and a wave reads 16 bytes a
// lane of it and converts them (v_cvt_scalef32_pk_bf16_fp4: two values and their power
// of two in one instruction) right before the four matrix instructions that they feed.
// Lane 32 h + r holds columns 32 h .. 32 h + 31 of row r, so instruction kk multiplies
// columns 8 kk .. 8 kk + 7 of both halves; the fragments of the activations are read to
// match.  The powers of two of four stages lie in a dword a lane, copied to LDS with
// every fourth stage.
#include <algorithm>
#include <type_traits>

#include "fp4_layout.h"
#include "gemm_tile.h"

namespace moe {

namespace {

struct Fp4Args : GemmArgs {
  const char* scale;            // packed scales of B
  int64_t scale_expert_bytes;   // per expert
  int blocks;                   // 64-column blocks of a row: K / 64
  int quads;                    // scale dwords of a row
};

constexpr int kScaleUnits = 4;   // dwords of scales kept in LDS for a weight row
constexpr int kMaxStages = 12;   // stages that span at most that many units

template <bool kBuf>
struct Source {  // rows or blocks to copy from: a descriptor with offsets, or addresses
  rsrc_t desc;
  const char* base;
  __device__ __forceinline__ void init(const char* p) {
    base = p;
    if constexpr (kBuf) desc = raw_rsrc(p);
  }
  template <bool kNt>
  __device__ __forceinline__ void load16(char* dst, int64_t off, int koff) const {
    if constexpr (kBuf) {
      if constexpr (kNt)
        buffer_load_lds16_nt(desc, dst, (uint32_t)off, koff);
      else
        buffer_load_lds16(desc, dst, (uint32_t)off, koff);
    } else {
      __builtin_amdgcn_global_load_lds((const void*)(base + off + koff), (lds_void*)dst, 16, 0,
                                       kNt ? 2 : 0);
    }
  }
  __device__ __forceinline__ void load4(char* dst, int64_t off, int koff) const {
    if constexpr (kBuf)
      buffer_load_lds4(desc, dst, (uint32_t)off, koff);
    else
      __builtin_amdgcn_global_load_lds((const void*)(base + off + koff), (lds_void*)dst, 4, 0, 0);
  }
};

// The copies of one workgroup's stages: its rows of A in blocks of 8 (1 KB), dealt to the
// waves in turn, then NB blocks of B.
template <bool kGateUp, int BM, int NB, int FN, int NW, bool kBuf>
struct Fp4Loader {
  using G = StageGeom<128>;
  static constexpr int LA = BM / 8 / NW, LB = NB / NW;
  static_assert(LA * 8 * NW == BM && LB * NW == NB, "whole blocks for every wave");
  Source<kBuf> a, b, sc;
  int64_t a_off[LA], b_off[LB], s_off[LB];
  int wave, live_a;    // blocks of A that this wave copies
  int a_bytes, stage_bytes, stages;
  char *smem, *scales;

  __device__ __forceinline__ void init(const Fp4Args& g, const TileRows& tr, int nt, int lane,
                                       int wave_, char* smem_, int smem_bytes) {
    wave = wave_;
    scales = smem_;
    smem = smem_ + kScaleUnits * NB * kFp4ScaleBytes;
    const int nb = (tr.rows + 31) / 32;
    a_bytes = nb * 32 * G::ROW_BYTES;
    stage_bytes = a_bytes + NB * kFp4BlockBytes;
    stages = (smem_bytes - kScaleUnits * NB * kFp4ScaleBytes) / stage_bytes;
    stages = stages < kMaxStages ? stages : kMaxStages;
    const int e = __builtin_amdgcn_readfirstlane(tr.e);
    a.init(kBuf ? g.a_base : g.A[0]);
    b.init(g.B + (int64_t)e * g.b_expert_bytes);
    sc.init(g.scale + (int64_t)e * g.scale_expert_bytes);
    live_a = 0;
    int row[LA];
#pragma unroll
    for (int t = 0; t < LA; ++t) {
      row[t] = (t * NW + wave) * 8 + lane / G::CH;
      live_a += (t * NW + wave) * 8 < tr.rows ? 1 : 0;
    }
    int src[LA];
#pragma unroll
    for (int t = 0; t < LA; ++t) {
      const int v = tr.v0 + (row[t] < tr.rows ? row[t] : tr.rows - 1);
      if (g.gather[0]) {
        int part;
        const int cr = tr.split_row(v, &part);
        src[t] = (part ? g.gather[1] : g.gather[0])[cr];
      } else {
        src[t] = tr.joint_row(v);
      }
    }
#pragma unroll
    for (int t = 0; t < LA; ++t) {
      const int64_t r = g.gather[0] ? src[t] / g.gather_k : src[t];
      a_off[t] = r * g.row_bytes + ((lane % G::CH) ^ G::swz(row[t])) * 16;
    }
#pragma unroll
    for (int t = 0; t < LB; ++t) {
      const int j = t * NW + wave;  // tile block: 32 columns of the tile
      const int last = g.ncols / kFp4BlockRows - 1;
      int rb;
      if constexpr (kGateUp) {
        // a wave's FN blocks: gate for the first half, the matching up rows after
        const int q = j % FN / (FN / 2);
        rb = nt * (NB / 2) + j / FN * (FN / 2) + j % (FN / 2);
        rb = (rb < last ? rb : last) + q * (g.I / kFp4BlockRows);
      } else {
        rb = nt * NB + j;
        rb = rb < last ? rb : last;  // columns past C are never stored
      }
      b_off[t] = (int64_t)rb * g.blocks * kFp4BlockBytes + lane * 16;
      s_off[t] = (int64_t)rb * g.quads * kFp4ScaleBytes + lane * 4;
    }
  }

  // Stage kt into ring slot `slot`; every fourth with its unit of scales.
  template <bool kNt>
  __device__ __forceinline__ void issue(int kt, int slot) const {
    char* base = smem + slot * stage_bytes;
    if ((kt & 3) == 0) {
      char* s = scales + ((kt >> 2) & (kScaleUnits - 1)) * NB * kFp4ScaleBytes;
#pragma unroll
      for (int t = 0; t < LB; ++t)
        sc.load4(s + (t * NW + wave) * kFp4ScaleBytes, s_off[t], (kt >> 2) * kFp4ScaleBytes);
    }
#pragma unroll
    for (int t = 0; t < LB; ++t)
      b.template load16<kNt>(base + a_bytes + (t * NW + wave) * kFp4BlockBytes, b_off[t],
                             kt * kFp4BlockBytes);
#pragma unroll
    for (int t = 0; t < LA; ++t)
      if (t < live_a)
        a.template load16<false>(base + (t * NW + wave) * 1024, a_off[t], kt * G::ROW_BYTES);
  }
};

// Eight values of a lane as a bf16 fragment.
__device__ __forceinline__ bf16x8 unpack_fp4(uint32_t v, float power) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, power, 0);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, power, 1);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, power, 2);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, power, 3);
  return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
#else
  return bf16x8{};
#endif
}

// The K loop of a wave that holds F 32-row blocks of the tile from row0 on (F = 0: it only
// copies and joins the barriers).
template <int F, int FM, int FN, int NB, bool kNt, class Loader>
__device__ __forceinline__ void fp4_k_loop(f32x16 (&acc)[FM][FN], const Loader& ld, int KT,
                                           int lane, int wn, int row0) {
  using G = StageGeom<128>;
  static_assert(F <= FM, "band blocks");
  const int r = lane & 31, half = lane >> 5;
  const int per_stage = ld.live_a + Loader::LB, stages = ld.stages;
  for (int s = 0; s < stages - 1; ++s)
    if (s < KT) ld.template issue<kNt>(s, s);
  __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
  int slot = 0, next = stages - 1;  // of stage kt, and of stage kt + stages - 1
  for (int kt = 0; kt < KT; ++kt) {
    // stage kt has landed once only the newer stages' loads are pending
    const int newer = KT - 1 - kt < stages - 2 ? KT - 1 - kt : stages - 2;
    const int pending = newer * per_stage + (((kt + newer) >> 2) - (kt >> 2)) * Loader::LB;
    wait_loads(pending < 24 ? pending : 24);
    __builtin_amdgcn_s_barrier();
    const char* sa = ld.smem + slot * ld.stage_bytes + row0 * G::ROW_BYTES;
    if constexpr (F > 0) {
      const char* sb = ld.smem + slot * ld.stage_bytes + ld.a_bytes + wn * FN * kFp4BlockBytes;
      const char* ss = ld.scales + (((kt >> 2) & (kScaleUnits - 1)) * NB + wn * FN) * kFp4ScaleBytes;
      bf16x8 af[2][F], bf[2][FN];
      uint4 raw[FN];
      float power[FN];
      auto rows = [&](int kk, int b) __attribute__((always_inline)) {
        const int fo = r * G::ROW_BYTES + (((4 * half + kk) ^ G::swz(r)) << 4);
#pragma unroll
        for (int i = 0; i < F; ++i) af[b][i] = *(const bf16x8*)(sa + i * 32 * G::ROW_BYTES + fo);
      };
      auto cols = [&](int kk, int b) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const uint32_t v = kk == 0 ? raw[j].x : kk == 1 ? raw[j].y : kk == 2 ? raw[j].z : raw[j].w;
          bf[b][j] = unpack_fp4(v, power[j]);
        }
      };
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        raw[j] = *(const uint4*)(sb + j * kFp4BlockBytes + lane * 16);
        const uint32_t s = *(const uint32_t*)(ss + j * kFp4ScaleBytes + lane * 4);
        power[j] = __uint_as_float((s >> (8 * (kt & 3)) & 0xffu) << 23);
      }
      rows(0, 0);
      if (kt + stages - 1 < KT) ld.template issue<kNt>(kt + stages - 1, next);
      cols(0, 0);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (kk + 1 < 4) rows(kk + 1, (kk + 1) & 1);
        __builtin_amdgcn_sched_barrier(0);
        if (kk + 1 < 4) cols(kk + 1, (kk + 1) & 1);
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = MmaBf16::mma(bf[kk & 1][j], af[kk & 1][i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      if (kt + stages - 1 < KT) ld.template issue<kNt>(kt + stages - 1, next);
    }
    slot = slot + 1 == stages ? 0 : slot + 1;
    next = next + 1 == stages ? 0 : next + 1;
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);  // this stage's reads are complete
  }
}

template <bool kGateUp, int BM, int BN, int WAVES_M, int WAVES_N, int kSmem, bool kBuf>
__global__ void __launch_bounds__(64 * WAVES_M * WAVES_N) grouped_gemm_fp4(Fp4Args a) {
  constexpr int NW = WAVES_M * WAVES_N, NB = BN / 32;
  constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, FM = WM / 32, FN = WN / 32;
  using Loader = Fp4Loader<kGateUp, BM, NB, FN, NW, kBuf>;
  static_assert(!kGateUp || FN % 2 == 0, "gate/up halves");
  static_assert(BM * (kGateUp ? BN / 2 : BN) * 2 <= kSmem, "C tile fits the stage buffers");
  __shared__ __attribute__((aligned(1024))) char smem[kSmem];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  MTileMap tm;
  tm.build(a.off0, a.off1, a.E, BM, BM >= 128 ? BM : 1);
  int mt, nt;
  if (!xcd_tile_at(tm, a.n_tiles, blockIdx.x & 7, blockIdx.x >> 3,
                   (32 + a.n_tiles - 1) / a.n_tiles, &mt, &nt))
    return;
  const TileRows tr = tm.locate(a.off0, a.off1, BM, mt);
  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};
  // the tile's 32-row blocks are shared out evenly between the wave rows
  const int nb = (tr.rows + 31) / 32;
  const int f0 = WAVES_M == 1 ? nb : (nb + 1) / 2;
  const int f = wm == 0 ? f0 : nb - f0, row0 = wm == 0 ? 0 : f0 * 32;
  Loader ld;
  ld.init(a, tr, nt, lane, wave, smem, kSmem);
  auto run = [&](auto nt_tag) __attribute__((always_inline)) {
    constexpr bool kNt = decltype(nt_tag)::value;
    if (FM >= 4 && f == 4) {
      if constexpr (FM >= 4) fp4_k_loop<4, FM, FN, NB, kNt>(acc, ld, a.blocks, lane, wn, row0);
    } else if (FM >= 3 && f == 3) {
      if constexpr (FM >= 3) fp4_k_loop<3, FM, FN, NB, kNt>(acc, ld, a.blocks, lane, wn, row0);
    } else if (FM >= 2 && f == 2) {
      if constexpr (FM >= 2) fp4_k_loop<2, FM, FN, NB, kNt>(acc, ld, a.blocks, lane, wn, row0);
    } else if (f == 1) {
      fp4_k_loop<1, FM, FN, NB, kNt>(acc, ld, a.blocks, lane, wn, row0);
    } else {
      fp4_k_loop<0, FM, FN, NB, kNt>(acc, ld, a.blocks, lane, wn, row0);
    }
  };
  // the weights of a tile that holds all of its expert's rows are read by no other tile
  if (tr.single)
    run(std::true_type{});
  else
    run(std::false_type{});
  __syncthreads();  // every wave is done with the stage buffers
  store_tile_lds<kGateUp, 1, FM, FN, BM, BN, WM, WN, 64 * NW>(a, acc, tr, nt, row0, f, wn, lane,
                                                             smem);
}

template <bool kGateUp, int BM, int BN, int WAVES_M, int WAVES_N, int kSmem, bool kBuf>
hipError_t launch_instance(Fp4Args a, const Shape& s, int64_t rows_bound, hipStream_t st) {
  constexpr int threads = 64 * WAVES_M * WAVES_N, cols = kGateUp ? BN / 2 : BN;
  a.n_tiles = (a.ncols + cols - 1) / cols;
  const int64_t grid = xcd_grid(m_tiles_bound(rows_bound, s.E, BM), a.n_tiles);
  if (grid <= 0) return hipSuccess;
  if (grid > 0x7fffffff / threads) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((grouped_gemm_fp4<kGateUp, BM, BN, WAVES_M, WAVES_N, kSmem, kBuf>),
                     dim3((unsigned)grid), dim3(threads), 0, st, a);
  return hipGetLastError();
}

template <bool kGateUp, bool kBuf>
hipError_t launch_kind(const Fp4Args& a, const Shape& s, int64_t rows_bound, hipStream_t st) {
  if (rows_bound >= 4096)
    return launch_instance<kGateUp, 256, 256, 2, 4, 160 * 1024, kBuf>(a, s, rows_bound, st);
  return launch_instance<kGateUp, 32, 256, 1, 4, 80 * 1024, kBuf>(a, s, rows_bound, st);
}

template <bool kGateUp>
hipError_t launch(const Shape& s, const GroupedIO& io, const uint8_t* B, const uint8_t* scale,
                  hipStream_t st) {
  if (io.rows_bound <= 0) return hipSuccess;
  const int K = kGateUp ? s.H : s.I, rows = kGateUp ? 2 * s.I : s.H;  // of an expert's matrix
  Fp4Args a{};
  a.A[0] = a.A[1] = (const char*)io.a[0];
  a.C[0] = (uint16_t*)io.c[0];
  a.C[1] = (uint16_t*)(io.c_split ? io.c[1] : io.c[0]);
  a.off0 = io.off[0];
  a.off1 = io.off[1];
  a.c_split = io.c_split && io.off[1];
  a.gather[0] = io.gather[0];
  a.gather[1] = io.off[1] ? io.gather[1] : io.gather[0];
  a.gather_k = io.gather_k;
  a.B = (const char*)B;
  a.scale = (const char*)scale;
  a.E = s.E;
  a.I = s.I;
  a.row_bytes = (int64_t)K * 2;
  a.ncols = kGateUp ? s.I : s.H;
  a.blocks = K / kFp4BlockCols;
  a.quads = (int)fp4_scale_quads(K);
  a.b_expert_bytes = (int64_t)rows * K / 2;
  a.scale_expert_bytes = fp4_scale_bytes(rows, K);
  a.a_base = a.A[0];
  // descriptor loads take 32-bit offsets: the rows of A, and an expert's weights, each
  // have to lie within 4 GiB
  const bool buf = rows_fit_4g(a.A[0], a.A[0], kGateUp ? s.T : io.rows_bound, K) &&
                   (uint64_t)a.b_expert_bytes < ((uint64_t)1 << 32);
  return buf ? launch_kind<kGateUp, true>(a, s, io.rows_bound, st)
             : launch_kind<kGateUp, false>(a, s, io.rows_bound, st);
}

}  // namespace

hipError_t launch_gate_up_fp4(const Shape& s, const GroupedIO& io, const uint8_t* w_gate_up,
                              const uint8_t* w_scale, hipStream_t st) {
  return launch<true>(s, io, w_gate_up, w_scale, st);
}

hipError_t launch_down_fp4(const Shape& s, const GroupedIO& io, const uint8_t* w_down,
                           const uint8_t* w_scale, hipStream_t st) {
  return launch<false>(s, io, w_down, w_scale, st);
}

}  // namespace moe
