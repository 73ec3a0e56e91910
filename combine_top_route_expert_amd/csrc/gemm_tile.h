// Tile machinery of the grouped expert GEMMs (gemm_bf16.hip, gemm_i8.hip): the
// copies of A and B stages into LDS and the K loops around the matrix
// instruction.  Both kernels move K in stages of 128 bytes of a row (64 bf16 or
// 128 int8 values) and feed 16 bytes of a row per lane to a 32 x 32 matrix
// instruction of the same duration, so everything here counts in bytes; what
// differs is the instruction (an Mma type) and, for int8, the last stage of rows
// that end in its middle.  The reasons for the layout and the loops, and what
// they measured, are in gemm_bf16.hip.
#pragma once

#include <type_traits>

#include "moe_internal.h"

namespace moe {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

// v_mfma_f32_32x32x16_bf16 and v_mfma_i32_32x32x32_i8: both take 16 bytes of a
// row per lane (lane l: row l % 32, chunk l / 32 of the two that one
// instruction multiplies) and leave the same 32 x 32 accumulator layout.
// kHalfStage: rows are multiples of 64 bytes, so the last stage may hold only
// its first half (bf16 rows of H % 64 == 0 values always fill their stages).
// kRefill: k_loop keeps all STAGES in flight at the start of a step and refills a
// buffer at its end, behind a second barrier, instead of keeping STAGES - 1 and
// refilling at the start.  For int8 on the small tile, whose steps hold little
// matrix work: 2 rows per expert, gate_up 988 -> 963 and down 506 -> 485 us; 62 rows
// per expert 68 -> 61 and 40 -> 36 us.  (k_loop_small: 1520 -> 1590 us at 128
// rows per expert, where the waves issue no loads beside each other's MFMAs any more.)
struct MmaBf16 {
  typedef bf16x8 frag;
  typedef f32x16 acc;
  static constexpr bool kHalfStage = false;
  static constexpr bool kRefill = false;
  static __device__ __forceinline__ acc mma(frag b, frag a, acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, a, c, 0, 0, 0);
  }
};
struct MmaI8 {
  typedef i32x4 frag;
  typedef i32x16 acc;
  static constexpr bool kHalfStage = true;
  static constexpr bool kRefill = true;
  static __device__ __forceinline__ acc mma(frag b, frag a, acc c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(b, a, c, 0, 0, 0);
  }
};

// s_waitcnt immediates (gfx9 encoding: vmcnt[3:0] | expcnt[6:4] | lgkmcnt[11:8] | vmcnt[15:14])
constexpr int wait_vm(int v) { return (v & 0xF) | ((v >> 4) << 14) | (0x7 << 4) | (0xF << 8); }
constexpr int kWaitLgkm0 = 0xF | (0x3 << 14) | (0x7 << 4);

constexpr int cmax(int x, int y) { return x > y ? x : y; }

// Operands of one launch, in bytes.
struct TileArgs {
  const char* A[2];           // [rows][row_bytes] (A[1]: chunk-1 rows when a_split)
  const char* B;              // [E][b_rows][row_bytes]
  const int32_t* off0;        // E + 1 offsets of the (first) chunk
  const int32_t* off1;        // E + 1 offsets of the pair's second chunk, or null
  int a_split, c_split;
  int E, I, ncols, n_tiles;
  int64_t row_bytes;          // of a row of A and of B: K values
  int64_t b_expert_bytes;     // per expert in B
  const int32_t* gather[2];   // optional: A rows gathered from hidden_states (src_row slices)
  int gather_k;
  const char* a_base;         // descriptor loads: every A row lies within 4 GiB above it
};

// Address of virtual row v of the tile's expert on one side of the product.
template <class T>
__device__ __forceinline__ const T* row_ptr(const T* const (&base)[2], int split,
                                            const TileRows& tr, int v, int64_t ld) {
  // both read first: a choice between the array's elements kept it in scratch memory
  const T *b0 = base[0], *b1 = base[1];
  if (split) {
    int part;
    const int r = tr.split_row(v, &part);
    return (part ? b1 : b0) + (int64_t)r * ld;
  }
  return b0 + (int64_t)tr.joint_row(v) * ld;
}

// LDS layout of one stage: BM rows of A then BN rows of B, each row SB bytes
// of K (ROW_BYTES) holding CH 16-byte chunks; chunk c of row r sits at slot
// c ^ swz(r).  A 16-lane phase of a 16-byte fragment read covers 16
// consecutive rows at one chunk; rows r and r + RB share a position in a
// 256-byte bank line, so swz(r) = (r / RB) mod CH spreads the 16 rows over 16
// distinct 16-byte bank groups (measured: no bank conflicts).
template <int SB>
struct StageGeom {
  static constexpr int ROW_BYTES = SB;
  static constexpr int CH = SB / 16;              // 16-byte chunks per row
  static constexpr int RPB = 1024 / ROW_BYTES;     // rows per 1 KB direct-to-LDS block
  static constexpr int RB = 256 / ROW_BYTES;       // rows per 256-byte bank line
  static_assert(SB == 128, "stage depth");
  static __device__ __forceinline__ int swz(int r) { return (r / RB) & (CH - 1); }
  // Fragment of a 32-row block: lane l holds row l % 32 and 16-byte chunk
  // 2*kk + l/32 of the stage.
  static __device__ __forceinline__ int frag_offset(int lane, int kk) {
    const int r = lane & 31;
    const int chunk = 2 * kk + (lane >> 5);
    return r * ROW_BYTES + ((chunk ^ swz(r)) << 4);
  }
};

// Everything a workgroup needs to stream its tile's A and B stages into LDS.
//
// kBuf: the stages are copied with the buffer form of the direct-to-LDS load
// (a descriptor per operand, 32-bit byte offsets per lane) instead of the
// global form.  Same bytes, same LDS layout; but the global form is a FLAT
// instruction, and while one is outstanding the compiler cannot count LDS
// reads in order, so every wait for a fragment read drains all of them.  With
// descriptor loads the K loop waits only for the fragments it is about to use,
// and the next sub-step's reads overlap the current MFMAs.  The host picks the
// global form when the A rows do not fit one 4 GiB window.
template <class M, bool kGateUp, int BM, int BN, int NW, int WN, int SB, bool kBuf>
struct TileLoader {
  using Mma = M;
  using G = StageGeom<SB>;
  static constexpr int LA = BM / G::RPB / NW, LB = BN / G::RPB / NW;  // 1 KB loads per wave
  static constexpr int STAGE_BYTES = (BM + BN) * G::ROW_BYTES;
  static constexpr int kThreads = 64 * NW;  // of the waves that share the loads
  static_assert(LA * G::RPB * NW == BM && LB * G::RPB * NW == BN, "tile rows per wave");
  const char* a_src[LA];
  const char* b_src[LB];
  uint32_t a_off[LA], b_off[LB];  // kBuf: byte offsets from the descriptors' bases
  rsrc_t ra, rb;
  int wave, mrows;
  int live_a;  // A blocks of this wave that hold rows of the tile (the rest are skipped)
  // kHalfStage: the stage (or -1) whose second half lies past the rows' end.  Its
  // lanes of the upper four chunks read the chunk 64 bytes before instead (in
  // bounds; clear_half then clears those of A): half_off is 64 for the lanes
  // that hold an upper chunk in an even block of a wave's, 64 - half_off in an odd
  // one (the swizzle of rows eight apart differs in the chunk's upper bit).
  int half_kt;
  uint32_t half_off;
  static_assert(LA % 2 == 0 && LB % 2 == 0, "a wave's blocks start at an even one");
  __device__ __forceinline__ uint32_t back(int t, int kt) const {
    if constexpr (!M::kHalfStage) return 0;
    return kt == half_kt ? (t & 1 ? 64 - half_off : half_off) : 0;
  }

  __device__ __forceinline__ void init(const TileArgs& a, const TileRows& tr, int nt, int lane,
                                       int wave_) {
    wave = wave_;
    mrows = tr.rows;
    if constexpr (M::kHalfStage) {
      half_kt = a.row_bytes % SB ? (int)(a.row_bytes / SB) : -1;
      half_off = lane & 4 ? 64 : 0;  // slot bit 2, against the swizzle's 0 in even blocks
    }
    const int row_in_blk = lane / G::CH, slot = lane % G::CH;
    live_a = 0;
    int rr[LA], ch[LA];
#pragma unroll
    for (int t = 0; t < LA; ++t) {
      const int row = (wave * LA + t) * G::RPB + row_in_blk;
      ch[t] = slot ^ G::swz(row);
      rr[t] = row < mrows ? row : mrows - 1;
      live_a += (wave * LA + t) * G::RPB < mrows ? 1 : 0;
    }
    if (a.gather[0]) {
      // permute fused into the row addressing: chunk row -> token (the LA
      // lookups are issued together and waited for once)
      int src[LA];
#pragma unroll
      for (int t = 0; t < LA; ++t) {
        int part;
        const int cr = tr.split_row(tr.v0 + rr[t], &part);
        src[t] = (part ? a.gather[1] : a.gather[0])[cr];
      }
#pragma unroll
      for (int t = 0; t < LA; ++t)
        a_src[t] = a.A[0] + (int64_t)(src[t] / a.gather_k) * a.row_bytes + ch[t] * 16;
    } else {
#pragma unroll
      for (int t = 0; t < LA; ++t)
        a_src[t] = row_ptr(a.A, a.a_split, tr, tr.v0 + rr[t], a.row_bytes) + ch[t] * 16;
    }
    // the expert is the same for the whole workgroup: keep its base scalar
    const int e = __builtin_amdgcn_readfirstlane(tr.e);
    const char* Be = a.B + (int64_t)e * a.b_expert_bytes;
#pragma unroll
    for (int t = 0; t < LB; ++t) {
      const int col = (wave * LB + t) * G::RPB + row_in_blk;  // tile column = B row
      const int chunk = slot ^ G::swz(col);
      int brow;
      if constexpr (kGateUp) {
        // each wave's WN columns: gate for the first half, the matching up rows after
        const int cw = col / WN, w = col % WN;
        const int q = w / (WN / 2), c = w % (WN / 2);
        brow = q * a.I + nt * (BN / 2) + cw * (WN / 2) + c;
      } else {
        brow = nt * BN + col;
        if (brow > a.ncols - 1) brow = a.ncols - 1;
      }
      b_src[t] = Be + (int64_t)brow * a.row_bytes + chunk * 16;
    }
    if constexpr (kBuf) {
      ra = raw_rsrc(a.a_base);
      rb = raw_rsrc(Be);
#pragma unroll
      for (int t = 0; t < LA; ++t) a_off[t] = (uint32_t)(a_src[t] - a.a_base);
#pragma unroll
      for (int t = 0; t < LB; ++t) b_off[t] = (uint32_t)(b_src[t] - Be);
    }
  }

  // One 1 KB block: 64 lanes x 16 bytes of stage kt of their rows into dst.
  __device__ __forceinline__ void load_a(int t, int kt, char* dst) const {
    const int koff = kt * G::ROW_BYTES;
    if constexpr (kBuf)
      buffer_load_lds16(ra, dst, a_off[t] - back(t, kt), koff);
    else
      __builtin_amdgcn_global_load_lds((const void*)(a_src[t] + koff - back(t, kt)),
                                       (lds_void*)dst, 16, 0, 0);
  }
  // kNt: the weight panel is read by this tile only (its expert has one m-tile),
  // so its bytes are streamed with the non-temporal cache policy.
  template <bool kNt>
  __device__ __forceinline__ void load_b(int t, int kt, char* dst) const {
    const int koff = kt * G::ROW_BYTES;
    if constexpr (kBuf) {
      if constexpr (kNt)
        buffer_load_lds16_nt(rb, dst, b_off[t] - back(t, kt), koff);
      else
        buffer_load_lds16(rb, dst, b_off[t] - back(t, kt), koff);
    } else {
      __builtin_amdgcn_global_load_lds((const void*)(b_src[t] + koff - back(t, kt)),
                                       (lds_void*)dst, 16, 0, kNt ? 2 : 0);
    }
  }

  // Compact stage of a tile with at most SROWS rows: those rows of A (the
  // first blocks, which only the first waves hold) then the BN rows of B.
  template <int SROWS>
  static constexpr int small_a() { return SROWS * G::ROW_BYTES; }
  template <int SROWS>
  static constexpr int small_stage() { return small_a<SROWS>() + BN * G::ROW_BYTES; }
  template <int SROWS, bool kNt>
  __device__ __forceinline__ void issue_small(char* smem, int kt, int buf) const {
    char* base = smem + buf * small_stage<SROWS>();
#pragma unroll
    for (int t = 0; t < LA; ++t)
      if (t < live_a)  // blocks past the tile's (at most SROWS) rows are not live
        load_a(t, kt, base + (wave * LA + t) * 1024);
#pragma unroll
    for (int t = 0; t < LB; ++t)
      load_b<kNt>(t, kt, base + small_a<SROWS>() + (wave * LB + t) * 1024);
  }

  // Rings of the wide 256 x 256 kernel: two A stages, then three B stages.
  static constexpr int A_BYTES = BM * G::ROW_BYTES, B_BYTES = BN * G::ROW_BYTES;
  __device__ __forceinline__ void issue_a(char* smem, int kt, int abuf) const {
    char* base = smem + abuf * A_BYTES;
#pragma unroll
    for (int t = 0; t < LA; ++t)
      if (t < live_a) load_a(t, kt, base + (wave * LA + t) * 1024);
  }
  template <bool kNt>
  __device__ __forceinline__ void issue_b(char* smem, int kt, int bbuf) const {
    char* base = smem + 2 * A_BYTES + bbuf * B_BYTES;
#pragma unroll
    for (int t = 0; t < LB; ++t) load_b<kNt>(t, kt, base + (wave * LB + t) * 1024);
  }

  // Loads one stage.  A blocks of 1 KB that lie wholly past the tile's rows are
  // not loaded (their LDS rows feed only outputs that are never stored), so a
  // wave issues live_a + LB loads per stage.
  template <bool kNt>
  __device__ __forceinline__ void issue(char* smem, int kt, int buf) const {
    char* base = smem + buf * STAGE_BYTES;
#pragma unroll
    for (int t = 0; t < LA; ++t)
      if (t < live_a) load_a(t, kt, base + (wave * LA + t) * 1024);
#pragma unroll
    for (int t = 0; t < LB; ++t)
      load_b<kNt>(t, kt, base + BM * G::ROW_BYTES + (wave * LB + t) * 1024);
  }
};

// Waits until at most n of this wave's vector memory operations are pending
// (s_waitcnt takes an immediate, so n is dispatched over its possible values).
__device__ __forceinline__ void wait_loads(int n) {
#define MOE_WAIT_CASE(v)                    \
  case v:                                   \
    __builtin_amdgcn_s_waitcnt(wait_vm(v)); \
    return;
  switch (n) {
    MOE_WAIT_CASE(1) MOE_WAIT_CASE(2) MOE_WAIT_CASE(3) MOE_WAIT_CASE(4) MOE_WAIT_CASE(5)
    MOE_WAIT_CASE(6) MOE_WAIT_CASE(7) MOE_WAIT_CASE(8) MOE_WAIT_CASE(9) MOE_WAIT_CASE(10)
    MOE_WAIT_CASE(11) MOE_WAIT_CASE(12) MOE_WAIT_CASE(13) MOE_WAIT_CASE(14) MOE_WAIT_CASE(15)
    MOE_WAIT_CASE(16) MOE_WAIT_CASE(17) MOE_WAIT_CASE(18) MOE_WAIT_CASE(19) MOE_WAIT_CASE(20)
    MOE_WAIT_CASE(21) MOE_WAIT_CASE(22) MOE_WAIT_CASE(23) MOE_WAIT_CASE(24)
    default:  // n <= 0, or beyond the table: wait for every load
      __builtin_amdgcn_s_waitcnt(wait_vm(0));
      return;
  }
#undef MOE_WAIT_CASE
}

// MFMAs of one stage: the wave's F 32-row blocks at sa against its FN 32-column
// blocks at sb, the fragments of each 32-byte sub-step read right before its
// MFMAs.
template <int F, int SB, class Loader, int FM, int FN>
__device__ __forceinline__ void stage_mma(typename Loader::Mma::acc (&acc)[FM][FN], const char* sa,
                                          const char* sb, int lane) {
  using G = StageGeom<SB>;
  using Frag = typename Loader::Mma::frag;
  static_assert(F <= FM, "band blocks");
  if constexpr (F > 0) {
#pragma unroll
    for (int kk = 0; kk < SB / 32; ++kk) {
      const int fo = G::frag_offset(lane, kk);
      Frag af[F], bfr[FN];
#pragma unroll
      for (int i = 0; i < F; ++i) af[i] = *(const Frag*)(sa + i * 32 * G::ROW_BYTES + fo);
#pragma unroll
      for (int j = 0; j < FN; ++j) bfr[j] = *(const Frag*)(sb + j * 32 * G::ROW_BYTES + fo);
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = Loader::Mma::mma(bfr[j], af[i], acc[i][j]);
    }
  }
}

// kHalfStage: where stage kt holds only the first half of the rows' 128 bytes,
// clears the second half of its ROWS rows of A at sa (the upper four chunks, which
// hold a copy of the lower ones), so that they add nothing whatever B holds there.
// One loop for all stages, with this in front of a last half one: a second copy
// of the MFMAs for that stage cost the wide tile 67-107 spilled registers.
template <int ROWS, int NT, class Loader>
__device__ __forceinline__ void clear_half(const Loader& ld, char* sa, int kt, int tid) {
  if constexpr (Loader::Mma::kHalfStage) {
    using G = typename Loader::G;
    if (kt != ld.half_kt) return;
    for (int c = tid; c < ROWS * 4; c += NT) {
      const int r = c >> 2, chunk = 4 + (c & 3);
      *(i32x4*)(sa + r * G::ROW_BYTES + ((chunk ^ G::swz(r)) << 4)) = i32x4{};
    }
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
    __builtin_amdgcn_s_barrier();
  }
}

// The K loop of one wave.  F (<= FM) 32-row blocks of the wave's band take
// part in the MFMAs (F = 0: none); the wave still issues its share of every
// stage's loads and joins every barrier.  The loop body holds no branch, so
// the compiler schedules the fragment reads, MFMAs and the next stage's loads
// as one block.
template <int F, int FM, int FN, int WM, int WN, int BM, int SB, int STAGES, bool kNt, class Loader>
__device__ __forceinline__ void k_loop(typename Loader::Mma::acc (&acc)[FM][FN],
                                       const Loader& ld, char* smem, int KT, int per_stage,
                                       int lane, int wm, int wn) {
  using G = StageGeom<SB>;
  using Frag = typename Loader::Mma::frag;
  constexpr int KS = SB / 32;  // MFMA sub-steps per stage
  constexpr bool kRefill = Loader::Mma::kRefill;
  constexpr int kAhead = kRefill ? STAGES : STAGES - 1;  // stages in flight at a step's start
  // nothing of the lgkm class (scalar loads included) is pending on entry, so
  // the waits before each sub-step's MFMAs can count the LDS reads in order
  __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
  const int tid = ld.wave * 64 + lane;
  for (int kt = 0; kt < KT; ++kt) {
    // stage kt has landed once only the newer stages issued so far are pending
    const int newer = KT - 1 - kt < kAhead - 1 ? KT - 1 - kt : kAhead - 1;
    wait_loads(newer * per_stage);
    __builtin_amdgcn_s_barrier();
    char* sa = smem + (kt % STAGES) * Loader::STAGE_BYTES;
    const char* sb = sa + BM * G::ROW_BYTES;
    clear_half<BM, Loader::kThreads>(ld, sa, kt, tid);
    if constexpr (F > 0) {
      // fragments in two register sets: sub-step kk + 1 is read while the
      // MFMAs of sub-step kk run
      Frag af[2][F], bfr[2][FN];
      auto frag = [&](int kk, int b) __attribute__((always_inline)) {
        const int fo = G::frag_offset(lane, kk);
#pragma unroll
        for (int i = 0; i < F; ++i)
          af[b][i] = *(const Frag*)(sa + (wm * WM + i * 32) * G::ROW_BYTES + fo);
#pragma unroll
        for (int j = 0; j < FN; ++j)
          bfr[b][j] = *(const Frag*)(sb + (wn * WN + j * 32) * G::ROW_BYTES + fo);
      };
      frag(0, 0);  // ahead of the next stage's loads, so the first MFMAs start sooner
      if (!kRefill && kt + STAGES - 1 < KT)
        ld.template issue<kNt>(smem, kt + STAGES - 1, (kt + STAGES - 1) % STAGES);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        if (kk + 1 < KS) frag(kk + 1, (kk + 1) & 1);
        // keeps the compiler from sinking those reads below this sub-step's MFMAs
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = Loader::Mma::mma(bfr[kk & 1][j], af[kk & 1][i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      if (!kRefill && kt + STAGES - 1 < KT)
        ld.template issue<kNt>(smem, kt + STAGES - 1, (kt + STAGES - 1) % STAGES);
    }
    // this stage's LDS reads are complete before any wave refills its buffer
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
    if (kRefill && kt + STAGES < KT) {
      __builtin_amdgcn_s_barrier();
      ld.template issue<kNt>(smem, kt + STAGES, kt % STAGES);
    }
  }
}

// The K loop of the wide 256 x 256 kernel (two waves per SIMD).
// Each load instruction holds its wave in issue until the CU's texture unit
// takes it, at 16-20 cycles per 1 KB; with all eight waves issuing a 64 KB
// stage at the start of a K step, no wave reached its MFMAs for the first
// 800-1150 of about 3300 cycles.  So the two waves of a SIMD take different
// roles.  The second (wave row 1) issues the next step's rows of A at the
// start of the step; the first (wave row 0), which gets the matrix pipe first
// and used to wait about 1000 cycles at the barrier, starts its MFMAs at once
// and issues the weight rows of B two steps ahead once its MFMAs are issued.
// A stays double-buffered and B triple-buffered (2 x 32 + 3 x 32 KB).  Loader
// slot q = wave % 4 of a four-wave loader layout covers the same rows in
// either role.
template <int F, int FM, int FN, int WM, int WN, int BM, int SB, bool kNt, class Loader>
__device__ __forceinline__ void k_loop_roles(typename Loader::Mma::acc (&acc)[FM][FN],
                                             const Loader& ld, char* smem, int KT, int lane,
                                             int wm, int wn) {
  using G = StageGeom<SB>;
  using Frag = typename Loader::Mma::frag;
  constexpr int KS = SB / 32;
  const bool a_role = wm != 0;
  __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
  const int tid = (ld.wave + (a_role ? Loader::kThreads / 64 : 0)) * 64 + lane;
  for (int kt = 0; kt < KT; ++kt) {
    // an A wave's newest load is A(kt); a B wave may still have B(kt + 1)
    // pending behind B(kt)
    wait_loads(!a_role && kt + 1 < KT ? Loader::LB : 0);
    __builtin_amdgcn_s_barrier();
    char* sa = smem + (kt & 1) * Loader::A_BYTES;
    const char* sb = smem + 2 * Loader::A_BYTES + (kt % 3) * Loader::B_BYTES;
    clear_half<BM, 2 * Loader::kThreads>(ld, sa, kt, tid);  // both roles' waves
    if constexpr (F > 0) {
      Frag af[2][F], bfr[2][FN];
      auto frag = [&](int kk, int b) __attribute__((always_inline)) {
        const int fo = G::frag_offset(lane, kk);
#pragma unroll
        for (int i = 0; i < F; ++i)
          af[b][i] = *(const Frag*)(sa + (wm * WM + i * 32) * G::ROW_BYTES + fo);
#pragma unroll
        for (int j = 0; j < FN; ++j)
          bfr[b][j] = *(const Frag*)(sb + (wn * WN + j * 32) * G::ROW_BYTES + fo);
      };
      frag(0, 0);
      if (a_role && kt + 1 < KT) ld.issue_a(smem, kt + 1, (kt + 1) & 1);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        if (kk + 1 < KS) frag(kk + 1, (kk + 1) & 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = Loader::Mma::mma(bfr[kk & 1][j], af[kk & 1][i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (!a_role && kt + 2 < KT) ld.template issue_b<kNt>(smem, kt + 2, (kt + 2) % 3);
    } else {
      if (a_role && kt + 1 < KT) ld.issue_a(smem, kt + 1, (kt + 1) & 1);
      if (!a_role && kt + 2 < KT) ld.template issue_b<kNt>(smem, kt + 2, (kt + 2) % 3);
    }
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
  }
}

// K loop of a tile on the wide path: the first STAGES - 1 stages, then
// k_loop over the 32-row blocks of this wave's band that hold rows of the
// tile.  Blocks past them feed only outputs that are never stored, so a wide
// tile skips their MFMAs (a band of 1 or 2 live blocks runs the 1- or 2-block
// loop, 3 runs the full one).  A one-block band always runs its MFMAs: a
// wave-uniform branch there measured slower than the wasted work.
// (kRoles: the wide kernel's role split, k_loop_roles.)
template <int FM, int FN, int WM, int WN, int BM, int SB, int STAGES, bool kNt, bool kRoles,
          class Loader>
__device__ __forceinline__ void wide_k(typename Loader::Mma::acc (&acc)[FM][FN],
                                       const Loader& ld, char* smem, int KT, int per_stage,
                                       int lane, int wm, int wn, int rows) {
  if constexpr (kRoles) {
    // KT >= 1: H and I are positive multiples of 64 (checked at the boundary)
    if (wm != 0) {
      ld.issue_a(smem, 0, 0);
    } else {
      ld.template issue_b<kNt>(smem, 0, 0);
      if (1 < KT) ld.template issue_b<kNt>(smem, 1, 1);
    }
  } else {
#pragma unroll
    for (int s = 0; s < (Loader::Mma::kRefill ? STAGES : STAGES - 1); ++s)
      if (s < KT) ld.template issue<kNt>(smem, s, s);
  }
  const int band_rows = rows - wm * WM;
  const int fm_live = band_rows <= 0 ? 0 : (band_rows + 31) / 32;
#define MOE_K_LOOP(F)                                                                              \
  do {                                                                                             \
    if constexpr (kRoles)                                                                          \
      k_loop_roles<F, FM, FN, WM, WN, BM, SB, kNt, Loader>(acc, ld, smem, KT, lane, wm, wn);       \
    else                                                                                           \
      k_loop<F, FM, FN, WM, WN, BM, SB, STAGES, kNt, Loader>(acc, ld, smem, KT, per_stage, lane,   \
                                                             wm, wn);                              \
  } while (0)
  if constexpr (FM == 1) {
    MOE_K_LOOP(1);
  } else {
    if (fm_live > 2)
      MOE_K_LOOP(FM);
    else if (fm_live == 2)
      MOE_K_LOOP(2);
    else if (fm_live == 1)
      MOE_K_LOOP(1);
    else
      MOE_K_LOOP(0);
  }
#undef MOE_K_LOOP
}

// The K loop of a tile with at most SROWS (32, 64, 128 or 160) rows: such a
// tile (a small expert's only m-tile) is bound by streaming its B panel rather
// than by MFMAs, so it uses the compact stage layout and SSTAGES stages
// (SSTAGES - 1 in flight) to keep more weight bytes in flight.  The wave holds
// F 32-row blocks of the tile's rows starting at row0 (its band); a wave with
// F = 0 only loads and joins the barriers.  (Reading the next sub-step's
// fragments during the current MFMAs, as k_loop does, measured no faster here.)
template <int F, int SROWS, int SSTAGES, int FM, int FN, int WN, int SB, bool kNt, class Loader>
__device__ __forceinline__ void k_loop_small(typename Loader::Mma::acc (&acc)[FM][FN],
                                             const Loader& ld, char* smem, int KT, int per_stage,
                                             int lane, int wn, int row0) {
  constexpr int STAGE = Loader::template small_stage<SROWS>();
  constexpr int ROWB = StageGeom<SB>::ROW_BYTES;
  const int tid = ld.wave * 64 + lane;
#pragma unroll
  for (int s = 0; s < SSTAGES - 1; ++s)
    if (s < KT) ld.template issue_small<SROWS, kNt>(smem, s, s);
  for (int kt = 0; kt < KT; ++kt) {
    const int newer = KT - 1 - kt < SSTAGES - 2 ? KT - 1 - kt : SSTAGES - 2;
    wait_loads(newer * per_stage);
    __builtin_amdgcn_s_barrier();
    char* sa = smem + (kt % SSTAGES) * STAGE;
    clear_half<SROWS, Loader::kThreads>(ld, sa, kt, tid);
    if (kt + SSTAGES - 1 < KT)
      ld.template issue_small<SROWS, kNt>(smem, kt + SSTAGES - 1, (kt + SSTAGES - 1) % SSTAGES);
    stage_mma<F, SB, Loader>(acc, sa + row0 * ROWB,
                             sa + Loader::template small_a<SROWS>() + wn * WN * ROWB, lane);
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
  }
}

}  // namespace

}  // namespace moe
