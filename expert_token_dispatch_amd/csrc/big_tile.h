// The main loop of the large 16-bit tile, shared by the grouped products
// (grouped_gemm.hip) and the Newton-Schulz products (newton_schulz.hip).  How the tile is
// staged and scheduled stands at the top of grouped_gemm.hip.
#pragma once

#include <algorithm>

#include "ffn_common.h"

namespace moe {
namespace {
namespace big {

constexpr int BM = 256, BNE = 256, BK = 64, kStages = 2;

constexpr int kRowBytes = BK * 2;              // 128
constexpr int kXcds = 8;

// s_waitcnt on the vector-memory counter only (expcnt and lgkmcnt left at their maxima)
#define MOE_VMCNT(n) __builtin_amdgcn_s_waitcnt(((n) & 0xF) | (((n) >> 4) << 14) | (0x7 << 4) | (0xF << 8))
#define MOE_LGKMCNT0() __builtin_amdgcn_s_waitcnt(0xC07F)

// Tile shapes: regular 256 A rows x 256 B rows, wide 128 A rows x 512 B rows.  With
// NW = 4 waves (one per SIMD) a wave owns 128 A rows x 128 B rows (4 x 4 MFMA 32x32
// accumulators, waves 2 x 2, or 1 x 4 for the wide tile); with NW = 8 (two per SIMD)
// 128 A rows x 64 B rows (4 x 2 accumulators, waves 2 x 4, or 1 x 8).  NB = 16 / NW
// B fragments per wave.
template <bool WIDE, int NW>
struct Shape {
  static constexpr int kThreads = NW * 64;
  static constexpr int NB = 16 / NW;
  static constexpr int kA = WIDE ? BM / 2 : BM;          // A rows
  static constexpr int kB = WIDE ? 2 * BNE : BNE;        // B rows
  static constexpr int kStageA = kA * kRowBytes;
  static constexpr int kStageB = kB * kRowBytes;
  static constexpr int kStage = (kA + kB) * kRowBytes;   // 64 KB regular, 80 KB wide
  static constexpr int kLdA = kA / (8 * NW), kLdB = kB / (8 * NW);  // 1 KB direct loads per wave per stage
  static constexpr int kLd = kLdA + kLdB;
  __device__ static int wm(int wave) { return WIDE ? 0 : wave / (NW / 2); }
  __device__ static int wn(int wave) { return WIDE ? wave : wave % (NW / 2); }
};
constexpr size_t kLoopLdsMax = size_t(kStages) * Shape<true, 4>::kStage;  // 160 KB
// a regular tile's two A slots and three B slots fit in the same space
static_assert(2 * Shape<false, 4>::kStageA + 3 * Shape<false, 4>::kStageB <= int(kLoopLdsMax), "regular ring");

// The operands of one tile.  Each is stored one of two ways, with rows of ld elements:
//   A, AKM false: m-major, element (m, k) at A[m * lda + k]; the buffer holds a_rows rows
//      of m (rows past them read zero);
//   A, AKM true:  k-major, element (k, m) at A[k * lda + m]; a_rows rows of k;
//   B, BKN false: n-major, element (n, k) at B[n * ldb + k] (a linear layer's [out, in]);
//   B, BKN true:  k-major, element (k, n) at B[k * ldb + n] (the math form's [in, out]);
//      b_rows rows (of n or k) either way.
// Bg, and Bu for the up rows of gate/up; with kcat > 0 (one-matrix products only) the
// k steps from kcat on read Bu at step - kcat (a product over two matrices side by side
// along K, such as dg Wg + du Wu).  PAIR: they read A2 at step - kcat as well (the sum of
// two products, A Bg + A2 Bu).
struct Operands {
  const uint16_t* A;
  int a_rows, lda;
  const uint16_t* Bg;
  const uint16_t* Bu;
  int b_rows, ldb;
  const uint16_t* A2;
};

// The element type of the operands, 16 bits: one MFMA of the tile.
struct Bf16 {
  __device__ static f32x16_t mma(bf16x8_t b, bf16x8_t a, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, a, c, 0, 0, 0);
  }
};
struct F16 {
  typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
  __device__ static f32x16_t mma(bf16x8_t b, bf16x8_t a, f32x16_t c) {  // the registers hold float16
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, b), __builtin_bit_cast(f16x8_t, a), c, 0,
                                                  0, 0);
  }
};

// The main loop of one tile (or one K piece of it): rows [row0, ..) of A by B rows
// [n0, ..) over k steps [kb, kb + nks); then epi(acc) with the sums.  Every load of the
// wave has landed by then, but other waves may still read the last stage.
template <int NMAT, bool WIDE, int NW, bool BKN, bool AKM, class MM, bool PAIR, class Epi>
__device__ __forceinline__ void tile_loop(const Operands& op, int N, int kcat, int row0, int n0, int kb, int nks,
                                          char* lds, const Epi& epi) {
  const uint16_t* __restrict__ A = op.A;
  const uint16_t* __restrict__ Bg = op.Bg;
  const uint16_t* __restrict__ Bu = op.Bu;
  const int a_rows = op.a_rows, lda = op.lda, ldb = op.ldb;
  using S = Shape<WIDE, NW>;
  constexpr int NB = S::NB;
  // the wave index is uniform: keeping it in a scalar register makes every LDS
  // target of the direct loads scalar arithmetic
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = S::wm(wave), wn = S::wn(wave);

  // ---- direct loads: per stage kLdA 1 KB blocks of 8 A rows and kLdB of 8 B
  // rows per wave; wave w fills A blocks kLdA*w.. and B blocks kLdB*w.. .  Lane
  // i of block j writes row (first row of the wave) + 8j + i/8, physical chunk
  // i%8, which holds logical chunk (i%8) ^ ((row/2)%8); as the wave's first row
  // is a multiple of 16, that depends on i and the parity of j only.
  const int c_even = (lane & 7) ^ ((lane >> 4) & 7);
  const int c_odd = (lane & 7) ^ ((4 + (lane >> 4)) & 7);
  const int a_lrow = (S::kA / NW) * wave + (lane >> 3);
  // buffer resources over A (from the tile's first row when m-major) and over the whole
  // weight matrix (its extent is under 4 GiB); a read outside either returns zeros
  const int64_t a_span = AKM ? int64_t(a_rows) * lda : int64_t(a_rows - row0) * lda;
  const uint32_t a_bytes = uint32_t(min(a_span * 2, int64_t(0xFFFFFFFF)));
  const __amdgpu_buffer_rsrc_t a_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(AKM ? A : A + size_t(row0) * lda), 0, a_bytes, kRsrcFlags);
  const __amdgpu_buffer_rsrc_t a_rsrc2 = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(!PAIR ? A : (AKM ? op.A2 : op.A2 + size_t(row0) * lda)), 0, a_bytes, kRsrcFlags);
  // the first half of the waves loads gate rows (or the only matrix), the second half up rows;
  // b_rsrc2 is the second matrix of a product split along K
  const uint32_t b_bytes = uint32_t(min(int64_t(op.b_rows) * ldb * 2, int64_t(0xFFFFFFFF)));
  const __amdgpu_buffer_rsrc_t b_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(NMAT == 2 && wave >= NW / 2 ? Bu : Bg), 0, b_bytes, kRsrcFlags);
  const __amdgpu_buffer_rsrc_t b_rsrc2 = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(Bu), 0, b_bytes,
                                                                           kRsrcFlags);
  // Rows past the segment (A) or past N (B) feed only outputs that are never
  // stored, so they may read any valid row: A takes the rows that follow (up
  // to the last row of the buffer), B wraps around to the first rows.  Letting
  // them all repeat one row would send every lane of the padding to the same
  // 128 bytes, one L2 channel, on every step.
  // Each lane's byte offsets are fixed for the whole loop (A from the tile's
  // first row, B from the matrix); a step only moves the scalar offset by k0,
  // so a load costs no vector arithmetic.
  uint32_t a_vo[S::kLdA], b_vo[S::kLdB];
  if constexpr (!AKM) {
    const int a_lim = a_rows - 1 - row0;
#pragma unroll
    for (int j = 0; j < S::kLdA; ++j) {
      const int cc = (j & 1) ? c_odd : c_even;
      a_vo[j] = (uint32_t(min(a_lrow + 8 * j, a_lim)) * uint32_t(lda) + uint32_t(cc * 8)) * 2u;
    }
  } else {
    // k-major stage, laid out as the k-major B stage below: regions of 128 m columns,
    // 64 k rows of 256 bytes each, 64-byte units swizzled by row
#pragma unroll
    for (int j = 0; j < S::kLdA; ++j) {
      const int gb = S::kLdA * wave + j;
      const int krow = 4 * (gb & 15) + (lane >> 4);
      const int u = ((lane & 15) >> 2) ^ ((lane >> 4) & 3);
      // columns past the tile's rows read what follows (or zeros past the buffer): never stored
      a_vo[j] = (uint32_t(krow) * uint32_t(lda) + uint32_t(row0 + 128 * (gb >> 4) + 32 * u + 8 * (lane & 3))) * 2u;
    }
  }
  if constexpr (!BKN) {
    int b_lrow;
    if (NMAT == 2) b_lrow = ((S::kB / NW) * wave + (lane >> 3)) & (S::kB / 2 - 1);
    else b_lrow = (S::kB / NW) * wave + (lane >> 3);
#pragma unroll
    for (int j = 0; j < S::kLdB; ++j) {
      const int cc = (j & 1) ? c_odd : c_even;
      int r = n0 + b_lrow + 8 * j;
      if (r >= N) r %= N;
      b_vo[j] = (uint32_t(r) * uint32_t(ldb) + uint32_t(cc * 8)) * 2u;
    }
  } else {
    // k-major stage: the tile's B rows in regions of 128 columns (gate regions, then
    // up regions), each 64 k rows of 256 bytes; 64-byte unit u (32 columns) of k row
    // r sits at physical unit u ^ (r % 4), so the four rows a transposing read
    // touches per half wave fall in four different bank groups.  Block j of the wave
    // (1 KB: four k rows of one region) is global block kLdB*wave + j; its lane l
    // writes k row 4*(block % 16) + l/16, physical 16-byte chunk l % 16.
#pragma unroll
    for (int j = 0; j < S::kLdB; ++j) {
      const int gb = S::kLdB * wave + j;
      const int reg = gb >> 4, krow = 4 * (gb & 15) + (lane >> 4);
      const int u = ((lane & 15) >> 2) ^ ((lane >> 4) & 3);
      const int col = n0 + 128 * (NMAT == 2 ? reg % (S::kB / 256) : reg) + 32 * u + 8 * (lane & 3);
      // columns past N read what follows in memory (or zeros past the matrix): never stored
      b_vo[j] = (uint32_t(krow) * uint32_t(ldb) + uint32_t(col)) * 2u;
    }
  }
  // LDS stages.  A wide tile keeps two whole stages (A and B rows of a step together).
  // A regular tile keeps its A rows in two slots and its B rows in three (2 x 32 + 3 x
  // 32 KB): the weight rows, which miss L2 far more often than the activation rows,
  // are asked for two steps before they are used instead of one.  a_slot(s) is where
  // stage s's A rows start; b_slot(s) + kStageA is where its B rows start (the B
  // fragment offsets count from a whole stage's base).
  constexpr bool kRing3 = !WIDE;
  const auto a_slot = [&](int st) -> char* {
    return kRing3 ? lds + (st & 1) * S::kStageA : lds + (st % kStages) * S::kStage;
  };
  const auto b_slot = [&](int st) -> char* {
    return kRing3 ? lds + S::kStageA + (st % 3) * S::kStageB : lds + (st % kStages) * S::kStage;
  };
// loads q0..q1-1 of stage kt_, in the order A0 B0 A1 B1 ... (then the B rows
// past the last A block)
#define MOE_ISSUE(kt_, q0_, q1_)                                                                            \
  do {                                                                                                      \
    char* sa_ = a_slot(kt_) + (S::kLdA * wave) * 1024;                                                      \
    char* sb_ = b_slot(kt_) + S::kStageA + (S::kLdB * wave) * 1024;                                         \
    const int s_ = kb + (kt_);                                                                              \
    const bool sec_ = kcat > 0 && s_ >= kcat;                                                               \
    const uint32_t k0_ = uint32_t(PAIR && sec_ ? s_ - kcat : s_) * (AKM ? uint32_t(BK * 2) * uint32_t(lda) : uint32_t(BK * 2)); \
    const uint32_t kbo_ = uint32_t(sec_ ? s_ - kcat : s_) * (BKN ? uint32_t(BK * 2) * uint32_t(ldb) : uint32_t(BK * 2)); \
    _Pragma("unroll") for (int q = (q0_); q < (q1_); ++q) {                                                 \
      const int j_ = q < 2 * S::kLdA ? q / 2 : q - S::kLdA;                                                 \
      if (q < 2 * S::kLdA && q % 2 == 0)                                                                    \
        __builtin_amdgcn_raw_ptr_buffer_load_lds(PAIR && sec_ ? a_rsrc2 : a_rsrc, (lds_ptr_t)(sa_ + j_ * 1024), 16, a_vo[j_], k0_, 0, 0); \
      else                                                                                                  \
        __builtin_amdgcn_raw_ptr_buffer_load_lds(sec_ ? b_rsrc2 : b_rsrc, (lds_ptr_t)(sb_ + j_ * 1024), 16, b_vo[j_], \
                                                 kbo_, 0, 0);                                              \
    }                                                                                                       \
  } while (0)

#define MOE_ISSUE_A1(kt_, j_)                                                                               \
  do {                                                                                                      \
    char* sa_ = a_slot(kt_) + (S::kLdA * wave) * 1024;                                                      \
    const bool seca_ = PAIR && kb + (kt_) >= kcat;                                                          \
    const uint32_t k0_ = uint32_t(kb + (kt_) - (seca_ ? kcat : 0)) * (AKM ? uint32_t(BK * 2) * uint32_t(lda) : uint32_t(BK * 2)); \
    __builtin_amdgcn_raw_ptr_buffer_load_lds(PAIR && seca_ ? a_rsrc2 : a_rsrc, (lds_ptr_t)(sa_ + (j_) * 1024), 16, a_vo[j_], k0_, 0, 0);   \
  } while (0)
#define MOE_ISSUE_B1(kt_, j_)                                                                               \
  do {                                                                                                      \
    char* sb_ = b_slot(kt_) + S::kStageA + (S::kLdB * wave) * 1024;                                         \
    const int s_ = kb + (kt_);                                                                              \
    const bool sec_ = kcat > 0 && s_ >= kcat;                                                               \
    const uint32_t kbo_ = uint32_t(sec_ ? s_ - kcat : s_) * (BKN ? uint32_t(BK * 2) * uint32_t(ldb) : uint32_t(BK * 2)); \
    __builtin_amdgcn_raw_ptr_buffer_load_lds(sec_ ? b_rsrc2 : b_rsrc, (lds_ptr_t)(sb_ + (j_) * 1024), 16, b_vo[j_], \
                                             kbo_, 0, 0);                                                   \
  } while (0)
// all A loads (MOE_ISSUE_A) or all B loads (MOE_ISSUE_B) of stage kt_
#define MOE_ISSUE_A(kt_)                                                                                    \
  do {                                                                                                      \
    char* sa_ = a_slot(kt_) + (S::kLdA * wave) * 1024;                                                      \
    const bool seca_ = PAIR && kb + (kt_) >= kcat;                                                          \
    const uint32_t k0_ = uint32_t(kb + (kt_) - (seca_ ? kcat : 0)) * (AKM ? uint32_t(BK * 2) * uint32_t(lda) : uint32_t(BK * 2)); \
    _Pragma("unroll") for (int j_ = 0; j_ < S::kLdA; ++j_)                                                  \
      __builtin_amdgcn_raw_ptr_buffer_load_lds(PAIR && seca_ ? a_rsrc2 : a_rsrc, (lds_ptr_t)(sa_ + j_ * 1024), 16, a_vo[j_], k0_, 0, 0);  \
  } while (0)
#define MOE_ISSUE_B(kt_)                                                                                    \
  do {                                                                                                      \
    char* sb_ = b_slot(kt_) + S::kStageA + (S::kLdB * wave) * 1024;                                         \
    const int s_ = kb + (kt_);                                                                              \
    const bool sec_ = kcat > 0 && s_ >= kcat;                                                               \
    const uint32_t kbo_ = uint32_t(sec_ ? s_ - kcat : s_) * (BKN ? uint32_t(BK * 2) * uint32_t(ldb) : uint32_t(BK * 2)); \
    _Pragma("unroll") for (int j_ = 0; j_ < S::kLdB; ++j_)                                                  \
      __builtin_amdgcn_raw_ptr_buffer_load_lds(sec_ ? b_rsrc2 : b_rsrc, (lds_ptr_t)(sb_ + j_ * 1024), 16, b_vo[j_], \
                                               kbo_, 0, 0);                                                 \
  } while (0)

  f32x16_t acc[4][NB];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // ---- fragment addresses: A rows wm*128 + i*32 + (lane & 31); B rows of the
  // wave's four 32-column blocks (gate/up: two gate blocks, then the two up
  // blocks of the same columns) --------------------------------------------
  const int fr = lane & 31;
  const int sw = (fr >> 1) & 7;
  const int g = lane >> 5;
  int boffs[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int br = NMAT == 2 ? (j < NB / 2 ? wn * NB * 16 + j * 32 : S::kB / 2 + wn * NB * 16 + (j - NB / 2) * 32)
                             : wn * NB * 32 + j * 32;
    if constexpr (!BKN) {
      boffs[j] = S::kStageA + (br + fr) * kRowBytes;
    } else {
      // 32-column block br: region br / 128, unit (br % 128) / 32; lane group G = lane / 16
      // reads k rows 8 (G / 2) + i / 4 (i = lane % 16) and columns 16 (G % 2) + 4 (i % 4)
      const int G = lane >> 4, i = lane & 15, u = (br & 127) >> 5;
      boffs[j] = S::kStageA + (br >> 7) * 16384 + (8 * (G >> 1) + (i >> 2)) * 256 + 64 * (u ^ (i >> 2)) +
                 32 * (G & 1) + 8 * (i & 3);
    }
  }
  // A rows wm*128 + i*32: m-major, one row per lane; k-major, region wm, unit i
  int aoffs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (!AKM) {
      aoffs[i] = (wm * 128 + i * 32 + fr) * kRowBytes;
    } else {
      const int G = lane >> 4, il = lane & 15;
      aoffs[i] = wm * 16384 + (8 * (G >> 1) + (il >> 2)) * 256 + 64 * (i ^ (il >> 2)) + 32 * (G & 1) + 8 * (il & 3);
    }
  }
  bf16x8_t fa[2][4], fb[2][NB];
#define MOE_LOADF(buf_, sta_, stb_, kc_)                                                                  \
  do {                                                                                                    \
    const int co_ = ((2 * (kc_) + g) ^ sw) * 16;                                                          \
    _Pragma("unroll") for (int i = 0; i < 4; ++i)                                                         \
      fa[buf_][i] = AKM ? read_kn_frag((sta_) + aoffs[i] + (kc_) * 16 * 256)                               \
                        : *reinterpret_cast<const bf16x8_t*>((sta_) + aoffs[i] + co_);                     \
    _Pragma("unroll") for (int j = 0; j < NB; ++j)                                                        \
      fb[buf_][j] = BKN ? read_kn_frag((stb_) + boffs[j] + (kc_) * 16 * 256)                               \
                        : *reinterpret_cast<const bf16x8_t*>((stb_) + boffs[j] + co_);                     \
  } while (0)
#define MOE_MMA(buf_)                                                                                     \
  do {                                                                                                    \
    _Pragma("unroll") for (int i = 0; i < 4; ++i)                                                         \
      _Pragma("unroll") for (int j = 0; j < NB; ++j)                                                      \
        acc[i][j] = MM::mma(fb[buf_][j], fa[buf_][i], acc[i][j]);                                               \
  } while (0)
#define MOE_LOADF_Q(buf_, sta_, stb_, kc_, q_)                                                            \
  do {                                                                                                    \
    const int co_ = ((2 * (kc_) + g) ^ sw) * 16;                                                          \
    fa[buf_][q_] = AKM ? read_kn_frag((sta_) + aoffs[q_] + (kc_) * 16 * 256)                                \
                       : *reinterpret_cast<const bf16x8_t*>((sta_) + aoffs[q_] + co_);                      \
    if ((q_) < NB)                                                                                        \
      fb[buf_][(q_) % NB] = BKN ? read_kn_frag((stb_) + boffs[(q_) % NB] + (kc_) * 16 * 256)                \
                                : *reinterpret_cast<const bf16x8_t*>((stb_) + boffs[(q_) % NB] + co_);      \
  } while (0)
#define MOE_MMA_Q(buf_, q_)                                                                               \
  do {                                                                                                    \
    _Pragma("unroll") for (int j = 0; j < NB; ++j)                                                        \
      acc[q_][j] = MM::mma(fb[buf_][j], fa[buf_][q_], acc[q_][j]);                                             \
  } while (0)
// the order inside a quarter of a four-wave tile: its MFMAs with the fragment reads and the load
// between them (mixtral_like gate/up -1.6 to -2.4%; the same for the eight-wave tile was 2-4%
// slower, so it keeps the compiler's order inside each quarter)
#define MOE_QUARTER_ORDER()                                                                               \
  do {                                                                                                    \
    if constexpr (NB == 4 && !AKM && !BKN) {                                                              \
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                                  \
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                                                  \
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                                  \
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                                                  \
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                                  \
      __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);                                                  \
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                                  \
    }                                                                                                     \
  } while (0)
  // LDS reads per chunk (a k-major B fragment takes two transposing reads) and MFMAs per chunk
  constexpr int kDs = 4 * (AKM ? 2 : 1) + NB * (BKN ? 2 : 1), kMf = 4 * NB;
  // {MFMA, LDS read, MFMA} (or {MFMA, LDS read} when the reads outnumber half the
  // MFMAs): the next chunk's fragment reads spread over the whole group
#define MOE_PIPE_DS()                                                                                     \
  do {                                                                                                    \
    if constexpr (kMf >= 2 * kDs) {                                                                       \
      _Pragma("unroll") for (int p_ = 0; p_ < kDs; ++p_) {                                                \
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                                \
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                                                \
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                                \
      }                                                                                                   \
      if constexpr (kMf > 2 * kDs) __builtin_amdgcn_sched_group_barrier(0x008, kMf - 2 * kDs, 0);         \
    } else {                                                                                              \
      _Pragma("unroll") for (int p_ = 0; p_ < kDs; ++p_) {                                                \
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                                \
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                                                \
      }                                                                                                   \
      if constexpr (kMf > kDs) __builtin_amdgcn_sched_group_barrier(0x008, kMf - kDs, 0);                 \
    }                                                                                                     \
  } while (0)

  // The refill of a stage goes out in two halves: the first right after the
  // barrier that frees its slot (beside the last chunk of the stage before),
  // the second beside the first chunk of the stage in between.  Against one
  // burst of all kLd loads per step this halves the rate at which the 32 CUs
  // of an XCD hit L2 together, and the second half still has three chunks to
  // land before the barrier that waits for it.
  constexpr int kHalf = S::kLd / 2;
  static_assert(!kRing3 || (S::kLdA == kHalf && S::kLdB == kHalf), "a regular tile's A and B loads are the halves");
  // a chunk that also issues half a refill: its fragment reads first, then the loads
  // spread over its 4 * NB MFMAs
#define MOE_CHUNK_LOADS()                                                                                 \
  do {                                                                                                    \
    __builtin_amdgcn_sched_group_barrier(0x100, kDs, 0);                                                  \
    if constexpr (NB == 4) {                                                                              \
      _Pragma("unroll") for (int p_ = 0; p_ < 8; ++p_) {                                                  \
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);                                                \
        __builtin_amdgcn_sched_group_barrier(0x020, kHalf / 8, 0);                                        \
      }                                                                                                   \
      if constexpr (kHalf % 8 != 0) __builtin_amdgcn_sched_group_barrier(0x020, kHalf % 8, 0);           \
    } else {                                                                                              \
      _Pragma("unroll") for (int p_ = 0; p_ < kHalf; ++p_) {                                              \
        __builtin_amdgcn_sched_group_barrier(0x008, 4 * NB / kHalf, 0);                                   \
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);                                                \
      }                                                                                                   \
    }                                                                                                     \
  } while (0)
  // Load order (the vector-memory counter retires loads in issue order).  Wide tile:
  // stage 0, the first half of stage 1; each iteration kt then issues the second half of
  // stage kt+1 at its top and the first half of stage kt+2 after its barrier, and the
  // barrier waits for everything (stage kt+1).  Regular tile: A0 B0 B1 and the first
  // half of A1; iteration kt issues the second half of A(kt+1) in its chunk 0, B(kt+2)
  // in chunks 1 and 2, and the first half of A(kt+2) in chunk 3 (after its barrier), so
  // at the barrier only B(kt+2) may still be in flight.  One load per quarter chunk
  // keeps the texture addresser's queue from filling (with a chunk's loads issued
  // together it was full several times as often as the vendor library's; spreading
  // them: mixtral_like down −2 to −3%, gate/up −0.3%).  Near the end a stage past the
  // last repeats the last one (same bytes into the same slot).
  if constexpr (kRing3) {
    // within a chunk, per quarter: one row of MFMAs, the next chunk's fragments of that
    // quarter, at most one load; the fences pin the order
    constexpr int hA = S::kLdA / 2, hB = S::kLdB / 2;
    static_assert(hA <= 4 && hB <= 4 && 4 % hA == 0 && 4 % hB == 0, "loads per quarter");
    MOE_ISSUE_A(0);
    MOE_ISSUE_B(0);
    MOE_ISSUE_B(min(1, nks - 1));
    _Pragma("unroll") for (int j = 0; j < hA; ++j) MOE_ISSUE_A1(min(1, nks - 1), j);
    MOE_VMCNT(S::kLdB + hA);  // stage 0 landed
    block_barrier();
    MOE_LOADF(0, a_slot(0), b_slot(0), 0);
    for (int kt = 0; kt + 1 < nks; ++kt) {
      const char* sta = a_slot(kt);
      const char* stb = b_slot(kt);
      const int sa1 = min(kt + 1, nks - 1), s2 = min(kt + 2, nks - 1);
      __builtin_amdgcn_sched_barrier(0);
      // chunk 0 (fragments of chunk 1 into buffer 1)
      _Pragma("unroll") for (int q = 0; q < 4; ++q) {
        MOE_MMA_Q(0, q);
        MOE_LOADF_Q(1, sta, stb, 1, q);
        if (q % (4 / hA) == 4 / hA - 1) MOE_ISSUE_A1(sa1, hA + q / (4 / hA));
        MOE_QUARTER_ORDER();
        __builtin_amdgcn_sched_barrier(0);
      }
      // chunk 1
      _Pragma("unroll") for (int q = 0; q < 4; ++q) {
        MOE_MMA_Q(1, q);
        MOE_LOADF_Q(0, sta, stb, 2, q);
        if (q % (4 / hB) == 4 / hB - 1) MOE_ISSUE_B1(s2, q / (4 / hB));
        MOE_QUARTER_ORDER();
        __builtin_amdgcn_sched_barrier(0);
      }
      // chunk 2
      _Pragma("unroll") for (int q = 0; q < 4; ++q) {
        MOE_MMA_Q(0, q);
        MOE_LOADF_Q(1, sta, stb, 3, q);
        if (q % (4 / hB) == 4 / hB - 1) MOE_ISSUE_B1(s2, hB + q / (4 / hB));
        MOE_QUARTER_ORDER();
        __builtin_amdgcn_sched_barrier(0);
      }
      MOE_VMCNT(S::kLdB);  // all but B(kt+2)
      MOE_LGKMCNT0();
      block_barrier();
      __builtin_amdgcn_sched_barrier(0);
      // chunk 3 (fragments of the next stage's chunk 0 into buffer 0)
      {
        const char* nta = a_slot(kt + 1);
        const char* ntb = b_slot(kt + 1);
        _Pragma("unroll") for (int q = 0; q < 4; ++q) {
          MOE_MMA_Q(1, q);
          MOE_LOADF_Q(0, nta, ntb, 0, q);
          if (q % (4 / hA) == 4 / hA - 1) MOE_ISSUE_A1(s2, q / (4 / hA));
          MOE_QUARTER_ORDER();
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  } else {
    MOE_ISSUE(0, 0, S::kLd);
    if (nks > 1) {
      MOE_ISSUE(1, 0, kHalf);
      MOE_VMCNT(kHalf);  // stage 0 landed
    } else {
      MOE_VMCNT(0);
    }
    block_barrier();
    MOE_LOADF(0, a_slot(0), b_slot(0), 0);
    for (int kt = 0; kt + 1 < nks; ++kt) {
      const char* sta = a_slot(kt);
      const char* stb = b_slot(kt);
      MOE_LOADF(1, sta, stb, 1);
      MOE_ISSUE(min(kt + 1, nks - 1), kHalf, S::kLd);
      MOE_MMA(0);
      MOE_CHUNK_LOADS();
      __builtin_amdgcn_sched_barrier(0);
      MOE_LOADF(0, sta, stb, 2);
      MOE_MMA(1);
      MOE_LOADF(1, sta, stb, 3);
      MOE_MMA(0);
      MOE_PIPE_DS();
      MOE_PIPE_DS();
      __builtin_amdgcn_sched_barrier(0);
      MOE_VMCNT(0);
      MOE_LGKMCNT0();
      block_barrier();
      __builtin_amdgcn_sched_barrier(0);
      MOE_LOADF(0, a_slot(kt + 1), b_slot(kt + 1), 0);
      MOE_ISSUE(min(kt + 2, nks - 1), 0, kHalf);
      MOE_MMA(1);
      MOE_CHUNK_LOADS();
    }
  }
  {
    const char* sta = a_slot(nks - 1);
    const char* stb = b_slot(nks - 1);
    MOE_LOADF(1, sta, stb, 1);
    MOE_MMA(0);
    MOE_LOADF(0, sta, stb, 2);
    MOE_MMA(1);
    MOE_LOADF(1, sta, stb, 3);
    MOE_MMA(0);
    MOE_MMA(1);
  }
  MOE_VMCNT(0);  // the last refill repeated a stage; let it land before the block ends
#undef MOE_ISSUE
#undef MOE_ISSUE_A
#undef MOE_ISSUE_A1
#undef MOE_ISSUE_B1
#undef MOE_LOADF_Q
#undef MOE_MMA_Q
#undef MOE_QUARTER_ORDER
#undef MOE_ISSUE_B
#undef MOE_LOADF
#undef MOE_MMA
#undef MOE_PIPE_DS
#undef MOE_CHUNK_LOADS
  epi(acc);
}

}  // namespace big
}  // namespace
}  // namespace moe
