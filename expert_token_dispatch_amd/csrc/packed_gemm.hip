// The packed experts' feed-forward for segments past a few rows, on the 4-bit weights as
// they are.
//
// A block of four waves owns 128 token rows by 256 weight rows of one expert (gate/up: 128
// gate rows and the same up rows), a wave all the token rows by 64 weight rows: 4 x 2 MFMA
// 32x32 accumulators, 32-row blocks past the segment's end left out.  Two blocks share a
// CU, so that one's epilogue runs beside the other's products.  Where those tiles are too
// few for the card, a tile has 128 weight rows.
//
// A step is 64 k.  Token rows (128 bytes a step) come by direct global->LDS loads into three
// slots, two steps ahead.  Codes (32 bytes a step) too, or two steps at a time into two slots,
// one stage ahead, half as many loads (SP, steps of a stage of codes).  A lane takes 16 bytes
// of codes, 32 k under one scale, for its weight row; they become four fragments in registers
// (v_cvt_scalef32_pk_bf16_fp4, eight a fragment pair, beside eight MFMAs).  The MFMA sums
// over k in any order: fragment c of lane half g is k = 32 g + 8 c .. of the step in both
// operands.  The scale bytes come straight to registers, two steps (four bytes) a load.
//
// Many rows are bound by the MFMAs (16384 on 8 experts of 4096 x 14336: 5.0 ms, 1150 TFLOP/s),
// 64 an expert and fewer by the fetching of codes, 32 bytes a row and step (512 rows: 363 us).
//
// In LDS 16-byte piece c of token row r sits at piece c ^ (r / 2 % 8), piece c of weight row
// r at c ^ (r / 8 % 2), of two steps' four at c ^ (r / 4 % 4): the reads of 16 rows at one
// piece cover all banks.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "big_tile.h"
#include "kernels.h"
#include "packed.h"

namespace moe {
namespace {
namespace pk {

constexpr int BM = 128, BK = 64, kThreads = 256;
constexpr int kGroup = 4;  // n-tiles per group of the tile order
constexpr int kXcds = 8;

// BNR: weight rows of a tile, 256 or 128; SP: steps of a stage of codes, 1 or 2
template <int NMAT, int BNR, int SP>
struct Shape {
  static constexpr int NJ = BNR / 128;               // 32-row weight blocks of a wave
  static constexpr int kSlotsA = 3, kSlotsB = SP == 1 ? 3 : 2;
  static constexpr int kLdA = 4, kLdB = BNR * SP / 128;  // 1 KB loads per wave and stage: token rows, codes
  static constexpr int kStageA = BM * 128, kStageB = BNR * 32 * SP, kRing = kSlotsA * kStageA + kSlotsB * kStageB;
  static constexpr int kCols = BNR / NMAT;           // output columns
  static constexpr int kRS = kCols * 2 + 16;         // a row of the output tile in LDS
  static constexpr int kLds = kRing > BM * kRS ? kRing : BM * kRS;
  // gate/up: stage rows 0 .. kCols - 1 are gate rows, the others up rows.  Row l of a wave's
  // block j; with one block a wave holds 16 gate rows and the up rows beside them.
  __device__ static int turn(int r) { return SP == 1 ? (r >> 3) & 1 : (r >> 2) & 3; }  // of weight row r's pieces
  __device__ static int stage_row(int wave, int j, int l) {
    if (NMAT == 1) return wave * 32 * NJ + j * 32 + l;
    if (NJ == 2) return j * kCols + wave * 32 + l;
    return (l >> 4) * kCols + wave * 16 + (l & 15);
  }
};

// Tiles of the local experts are numbered one of two ways; every wave finds its own, 64
// experts at a time.
//   In order (many): over (expert, group of n-tiles, m-tile, n-tile in group), each XCD
//   a range, so that the blocks which run at once on an XCD share weight and token rows in L2.
//   By size (few tiles): full m-tiles of all experts, then the segments' tails of more
//   than half a tile, then the others, over (expert, m-tile, n-tile), dealt out singly: the
//   short ones fill the gaps at the end.
struct Tile {
  int expert, row0, rows, n;
};

// m-tiles of expert e in size class c (-1: all), and its first row of that class
__device__ __forceinline__ int m_tiles(const int32_t* __restrict__ offsets, int L, int e, int c, int& first) {
  first = offsets[min(e, L)];
  const int n = e < L ? offsets[e + 1] - first : 0, full = n / BM, tail = n % BM;
  if (c < 0) return full + (tail > 0);
  if (c == 0) return full;
  first += full * BM;
  return c == 1 ? tail > BM / 2 : tail > 0 && tail <= BM / 2;
}

__device__ __forceinline__ int total_tiles(const int32_t* __restrict__ offsets, int L, int NT) {
  int sum = 0, first;
  for (int e = threadIdx.x & 63; e < L; e += 64) sum += m_tiles(offsets, L, e, -1, first) * NT;
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
  return sum;
}

__device__ __forceinline__ Tile find_tile(const int32_t* __restrict__ offsets, int L, int NT, int t, bool by_size) {
  const int lane = threadIdx.x & 63;
  Tile r{-1, 0, 0, 0};
  for (int c = by_size ? 0 : -1; c < 3; ++c) {
    for (int base = 0; base < L; base += 64) {
      int first;
      const int mt = m_tiles(offsets, L, base + lane, c, first), mine = mt * NT;
      int incl = mine;
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d, 64);
        if (lane >= d) incl += o;
      }
      const uint64_t past = __ballot(incl > t);
      if (past) {
        const int l = __ffsll((unsigned long long)past) - 1;
        r.expert = base + l;
        t -= __shfl(incl - mine, l, 64);
        const int row = __shfl(first, l, 64), m = __shfl(mt, l, 64), end = offsets[r.expert + 1];
        if (by_size) {
          r.row0 = row + t / NT * BM;
          r.n = t % NT;
        } else {
          const int g = min(t / (m * kGroup), (NT - 1) / kGroup);
          t -= g * m * kGroup;
          const int w = min(kGroup, NT - g * kGroup);
          r.row0 = row + t / w * BM;
          r.n = g * kGroup + t % w;
        }
        r.rows = min(BM, end - r.row0);
        return r;
      }
      t -= __shfl(incl, 63, 64);
    }
  }
  return r;
}

template <int NMAT, int BNR, int SP>
__device__ __forceinline__ void body(const bf16_t* __restrict__ A, const int32_t* __restrict__ offsets,
                                     const uint8_t* __restrict__ q0, const uint8_t* __restrict__ s0,
                                     const uint8_t* __restrict__ q1, const uint8_t* __restrict__ s1,
                                     bf16_t* __restrict__ C, int L, int N, int K, bool by_size, char* lds) {
  using S = Shape<NMAT, BNR, SP>;
  constexpr int NJ = S::NJ;
  char* const lds_b = lds + S::kSlotsA * S::kStageA;
  const int NT = (N + S::kCols - 1) / S::kCols;
  const int total = __builtin_amdgcn_readfirstlane(total_tiles(offsets, L, NT));
  const int per = (total + kXcds - 1) / kXcds;
  const int xcd = blockIdx.x % kXcds, loc = blockIdx.x / kXcds, t = by_size ? int(blockIdx.x) : xcd * per + loc;
  if ((!by_size && loc >= per) || t >= total) return;
  const Tile tile = find_tile(offsets, L, NT, t, by_size);
  const int expert = __builtin_amdgcn_readfirstlane(tile.expert);
  const int row0 = __builtin_amdgcn_readfirstlane(tile.row0), rows = __builtin_amdgcn_readfirstlane(tile.rows);
  const int n0 = __builtin_amdgcn_readfirstlane(tile.n) * S::kCols;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int half = lane >> 5, fr = lane & 31;
  const int blocks = (rows + 31) / 32;  // 32-row blocks that have rows

  // ---- loads.  Token rows: this wave's 32 (four loads of eight rows); past the segment
  // they repeat its last row.  Codes: its quarter of the stage rows, 32 / SP a load; gate/up:
  // waves 0 and 1 gate rows, 2 and 3 up rows.  Rows past N repeat row N - 1.  Neither reaches an
  // output that is stored.
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<bf16_t*>(A + size_t(row0) * K), 0, uint32_t(rows) * uint32_t(K) * 2u, kRsrcFlags);
  const size_t eq = size_t(expert) * N * (K / 2), es = size_t(expert) * N * (K / 32);
  const bool second = NMAT == 2 && wave >= 2;
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>((second ? q1 : q0) + eq), 0,
                                                                      uint32_t(N) * uint32_t(K / 2), kRsrcFlags);
  uint32_t va[4], vb[S::kLdB];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = wave * 32 + 8 * j + (lane >> 3);
    va[j] = uint32_t(min(r, rows - 1)) * uint32_t(K) * 2u + uint32_t(((lane & 7) ^ ((r >> 1) & 7)) * 16);
  }
#pragma unroll
  for (int j = 0; j < S::kLdB; ++j) {
    const int r = wave * (BNR / 4) + 32 / SP * j + lane / (2 * SP);  // stage row
    const int row = min(n0 + r % S::kCols, N - 1);
    vb[j] = uint32_t(row) * uint32_t(K / 2) + uint32_t(((lane & (2 * SP - 1)) ^ S::turn(r)) * 16);
  }
  const int steps = (K + BK - 1) / BK;
  // K is a multiple of 32: the last step may be half a one; its token pieces past K read as
  // zero (an address behind the buffer), its codes may be whatever follows
  const bool cut = (K & 32) != 0;
  auto issue_a = [&](int s) {  // step min(s, steps - 1) into slot s
    const int st = min(s, steps - 1);
    char* slot = lds + (s % S::kSlotsA) * S::kStageA;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = (lane & 7) ^ (((wave * 32 + 8 * j + (lane >> 3)) >> 1) & 7);
      const uint32_t vo = cut && st == steps - 1 && c >= 4 ? 0xFFFFFFF0u : va[j];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(slot + (4 * wave + j) * 1024), 16, vo,
                                               uint32_t(st) * 128u, 0, 0);
    }
  };
  auto issue_b = [&](int stage) {  // steps SP stage .., or the last stage there is
    const int st = min(stage, (steps - 1) / SP);
    char* slot = lds_b + (stage % S::kSlotsB) * S::kStageB;
#pragma unroll
    for (int j = 0; j < S::kLdB; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr_t)(slot + (S::kLdB * wave + j) * 1024), 16, vb[j],
                                               uint32_t(st) * (32u * SP), 0, 0);
  };

  // ---- this lane's weight rows: stage row of block j, and its scales.  Four bytes are two
  // steps; where a row's bytes are no whole words the loads are unaligned, and at its end short.
  const uint8_t* sp[NJ];
  int br[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    br[j] = S::stage_row(wave, j, fr);
    const int row = min(n0 + br[j] % S::kCols, N - 1);
    sp[j] = (NMAT == 2 && br[j] >= S::kCols ? s1 : s0) + es + size_t(row) * (K / 32);
  }
  const int groups = K / 32;
  auto load_s = [&](int s, uint32_t (&v)[NJ]) {  // the scales of steps s and s + 1, s even
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      v[j] = 0;
      if (2 * s + 4 <= groups) {
        __builtin_memcpy(&v[j], sp[j] + 2 * s, 4);
      } else {
        for (int i = 0; i < 3; ++i)
          if (2 * s + i < groups) v[j] |= uint32_t(sp[j][2 * s + i]) << (8 * i);
      }
    }
  };

  f32x16_t acc[4][NJ];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  const int sw = (fr >> 1) & 7;
  uint32_t sc[NJ], sn[NJ];
  load_s(0, sc);
  issue_a(0);
  issue_b(0);
  issue_a(1);
  if (SP == 1) issue_b(1);
  // by the tile's row blocks, so that no branch stands among the products: the operands for
  // the next chunk are read and decoded between them
  const auto run = [&](auto blocks_t) {
    constexpr int MB = decltype(blocks_t)::value;
    for (int s = 0; s < steps; ++s) {
      // the step's loads have landed: behind them only the next step's token rows were issued,
      // and the codes that the last step asked for (and any scales, which only makes the
      // wait longer)
      if ((s & 1) == 0) {
        MOE_VMCNT(S::kLdA + (SP == 1 ? S::kLdB : 0));
      } else {
        MOE_VMCNT(S::kLdA + S::kLdB);
      }
      MOE_LGKMCNT0();
      block_barrier();
      // the scales first: loads return in order, and behind the refill they would make the
      // wave wait for it
      if ((s & 1) == 0) {
        load_s(s + 2 < steps ? s + 2 : 0, sn);
        asm volatile("" ::: "memory");
      }
      issue_a(s + 2);
      if (SP == 1)
        issue_b(s + 2);
      else if ((s & 1) == 0)
        issue_b(s / 2 + 1);
      const char* st = lds + (s % S::kSlotsA) * S::kStageA;
      const char* stb = lds_b + (s / SP % S::kSlotsB) * S::kStageB;
      const int first = s % SP * 2;  // of the lane's pieces of the stage
      u32x4_t w[NJ];
      float f[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        w[j] = *reinterpret_cast<const u32x4_t*>(stb + br[j] * 32 * SP + (((first + half) ^ S::turn(br[j])) * 16));
        f[j] = __uint_as_float(((sc[j] >> (16 * (s & 1) + 8 * half)) & 0xFFu) << 23);
      }
      const auto frag_a = [&](int i, int c) {
        return *reinterpret_cast<const bf16x8_t*>(st + (i * 32 + fr) * 128 + (((4 * half + c) ^ sw) * 16));
      };
      bf16x8_t fa[2][MB], fb[2][NJ];
#pragma unroll
      for (int i = 0; i < MB; ++i) fa[0][i] = frag_a(i, 0);
#pragma unroll
      for (int j = 0; j < NJ; ++j) fb[0][j] = decode_frag(w[j][0], f[j]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c < 3) {
#pragma unroll
          for (int i = 0; i < MB; ++i) fa[(c + 1) & 1][i] = frag_a(i, c + 1);
#pragma unroll
          for (int j = 0; j < NJ; ++j) fb[(c + 1) & 1][j] = decode_frag(w[j][c + 1], f[j]);
        }
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[c & 1][j], fa[c & 1][i], acc[i][j], 0, 0, 0);
        if (c < 3) {
#pragma unroll
          for (int i = 0; i < MB; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 4 * NJ / MB, 0);
            if constexpr (NJ == 2) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (s & 1) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) sc[j] = sn[j];
      }
    }
  };
  switch (blocks) {
    case 1: run(std::integral_constant<int, 1>{}); break;
    case 2: run(std::integral_constant<int, 2>{}); break;
    case 3: run(std::integral_constant<int, 3>{}); break;
    default: run(std::integral_constant<int, 4>{});
  }
  MOE_VMCNT(0);  // the last (repeated) loads land before the LDS is used again
  MOE_LGKMCNT0();
  block_barrier();

  // ---- epilogue: the products were (weight rows) x (token rows), so lane l holds token row
  // l % 32 and register 4q + u column 8q + 4 (l / 32) + u; the tile goes through LDS and
  // out in whole row pieces
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < blocks) {
#pragma unroll
      for (int j = 0; j < (NMAT == 2 ? 1 : NJ); ++j) {
#pragma unroll
        for (int q = 0; q < (NMAT == 2 && NJ == 1 ? 2 : 4); ++q) {
          float v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if constexpr (NMAT == 1)
              v[u] = acc[i][j][4 * q + u];
            else if constexpr (NJ == 2)
              v[u] = silu(acc[i][0][4 * q + u]) * acc[i][1][4 * q + u];
            else  // gate rows are the block's first 16, two q
              v[u] = silu(acc[i][0][4 * q + u]) * acc[i][0][4 * (q + 2) + u];
          }
          const int cl = wave * (S::kCols / 4) + j * 32 + 8 * q + 4 * half;
          *reinterpret_cast<uint2*>(lds + (i * 32 + fr) * S::kRS + cl * 2) =
              make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        }
      }
    }
  }
  MOE_LGKMCNT0();
  block_barrier();
  constexpr int kPieces = S::kCols / 8;
#pragma unroll
  for (int u = 0; u < BM * kPieces / kThreads; ++u) {
    const int id = tid + kThreads * u, r = id / kPieces, c = id % kPieces * 8;
    // N is a multiple of 8: a piece is inside or outside as a whole
    if (r < rows && n0 + c < N)
      *reinterpret_cast<u32x4_t*>(C + size_t(row0 + r) * N + n0 + c) =
          *reinterpret_cast<const u32x4_t*>(lds + r * S::kRS + c * 2);
  }
}

template <int NMAT, int BNR, int SP>
__global__ __launch_bounds__(kThreads, 2) void kernel(const bf16_t* __restrict__ A, const int32_t* __restrict__ offsets,
                                                      const uint8_t* __restrict__ q0, const uint8_t* __restrict__ s0,
                                                      const uint8_t* __restrict__ q1, const uint8_t* __restrict__ s1,
                                                      bf16_t* __restrict__ C, int L, int N, int K, int by_size) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  body<NMAT, BNR, SP>(A, offsets, q0, s0, q1, s1, C, L, N, K, by_size != 0, lds);
}

template <int NMAT, int BNR, int SP>
moe_status launch_bnr(const char* name, const bf16_t* A, const int32_t* offsets, const void* q0, const void* s0,
                      const void* q1, const void* s1, bf16_t* C, int L, int N, int K, int64_t max_pairs, bool by_size,
                      hipStream_t s) {
  using S = Shape<NMAT, BNR, SP>;
  auto kern = kernel<NMAT, BNR, SP>;
  const hipError_t e =
      hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
  if (e != hipSuccess) return set_error(MOE_ERR_HIP, "%s: LDS attribute: %s", name, hipGetErrorString(e));
  // at most this many tiles: every expert with rows may end in a partly filled one
  const int64_t m = max_pairs / BM + std::min<int64_t>(L, max_pairs);
  const int64_t tiles = m * ((N + S::kCols - 1) / S::kCols);
  const int64_t per = (tiles + kXcds - 1) / kXcds;
  MOE_LAUNCH(name, kern, dim3(unsigned(per * kXcds)), dim3(kThreads), S::kLds, s, A, offsets,
             static_cast<const uint8_t*>(q0), static_cast<const uint8_t*>(s0), static_cast<const uint8_t*>(q1),
             static_cast<const uint8_t*>(s1), C, L, N, K, by_size ? 1 : 0);
  return MOE_OK;
}

// Tiles of 256 weight rows, 128 where those would not give every CU one; by size while a CU
// gets fewer than four, in order from there (a prefill of 16384 pairs on 8 experts: in order
// -2%; 2047 pairs on 16 experts of very different load: by size -6%).  From there codes go two
// steps at a time, where rows begin at multiples of 64 bytes (the same prefill 5150 -> 4998
// us, 8192 pairs on 8 experts of 4096 x 4096 711 -> 696; with fewer tiles, 8192 pairs on 128
// experts, H 2048, I 768: 141 -> 154).  Tiles are counted from the most rows that the
// descriptor allows; where a rank holds part of the experts fewer arrive, and the choice is the
// one for more of them.
template <int NMAT>
moe_status launch(const char* name, const bf16_t* A, const int32_t* offsets, const void* q0, const void* s0,
                  const void* q1, const void* s1, bf16_t* C, int L, int N, int K, int64_t max_pairs, hipStream_t s) {
  const int64_t m = max_pairs / BM + std::min<int64_t>(L, max_pairs) / 2;
  const int64_t tiles = m * ((N + 256 / NMAT - 1) / (256 / NMAT));
#define MOE_PACKED_TILE(BNR_, SP_, BY_SIZE_) \
  launch_bnr<NMAT, BNR_, SP_>(name, A, offsets, q0, s0, q1, s1, C, L, N, K, max_pairs, BY_SIZE_, s)
  if (tiles >= 1024 && K % 128 == 0) return MOE_PACKED_TILE(256, 2, false);
  if (tiles >= 256) return MOE_PACKED_TILE(256, 1, tiles < 1024);
  return MOE_PACKED_TILE(128, 1, true);
#undef MOE_PACKED_TILE
}

}  // namespace pk
}  // namespace

bool packed_gemm_fits(const moe_layer_desc* d, int64_t max_pairs) {
  // an expert's codes and 128 token rows are addressed with 32-bit byte offsets, tiles counted in an int
  const int64_t H = d->hidden, I = d->intermediate;
  return d->dtype == MOE_BF16 && H * I / 2 < (int64_t(1) << 32) - 16 && std::max(H, I) * 256 < (int64_t(1) << 32) - 16 &&
         (max_pairs / pk::BM + d->local_count) * ((std::max(H, I) + 63) / 64) < (int64_t(1) << 30);
}

moe_status launch_packed_gemm(const PackedFfnArgs& a) {
  const moe_layer_desc* d = a.d;
  const int L = d->local_count, H = d->hidden, I = d->intermediate;
  const moe_packed_experts& p = *a.p;
  bf16_t* h = static_cast<bf16_t*>(a.h);
  const moe_status st = pk::launch<2>("ffn_gate_up", static_cast<const bf16_t*>(a.x_sorted), a.offsets, p.gate_codes,
                                      p.gate_scales, p.up_codes, p.up_scales, h, L, I, H, a.max_pairs, a.s);
  if (st != MOE_OK) return st;
  return pk::launch<1>("ffn_down", h, a.offsets, p.down_codes, p.down_scales, p.down_codes, p.down_scales,
                       static_cast<bf16_t*>(a.y_sorted), L, H, I, a.max_pairs, a.s);
}

}  // namespace moe
