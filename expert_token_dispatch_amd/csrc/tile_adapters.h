// The adapters' share of a tile of token rows by weight rows, for the products whose accumulators
// have the weight rows as the left operand (grouped_gemm.hip, adapted_gemm.hip).
#pragma once

#include "adapters.h"

namespace moe {
namespace {

// ---- adapters.  A tile's sums get the adapters' share before they are rounded: u's two parts
// by the adapter's B, for one adapter of the tile's rows after another (one or two in a prompt,
// whose requests follow each other).  Of every rank chunk of up to 32, the tile's rows of u
// go to LDS once and an adapter's rows of B (the tile's columns) after them, with the next
// adapter's already in flight; the products of all rows are formed apart and added where the row
// has the adapter, so that a row's sum, and what a broken adapter spoils, do not depend on the
// rows beside it.  LDS rows of 32 values and 16 bytes, so that 16 lanes' reads of 16 rows fall
// in different banks.
constexpr int kChunkRank = 32, kAdRow = kChunkRank * 2 + 16;
// the LDS it takes, from the tile's operands' (every load into them has landed)
template <class S, int NMAT>
constexpr int kTileAdapterLds = (NMAT * 2 * S::kA + S::kB) * kAdRow;

__device__ __forceinline__ f32x16_t mma32(bf16x8_t b, bf16x8_t a, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, a, c, 0, 0, 0);
}

// S: the tile's rows kA and kB (with NMAT = 2 half of kB gate, half up), kThreads, 32-column blocks a
// wave NB, and the wave's place wm, wn.  A wave has NA row blocks.

template <class S, int NMAT, int NA>
__device__ __forceinline__ void tile_adapters(const Adapters& ad, int expert, int row0, int rows, int n0, int N,
                                              char* lds, f32x16_t (&acc)[NA][S::NB]) {
  constexpr int NB = S::NB, kThreads = S::kThreads, kIds = S::kA / 64;
  constexpr int kBLoads = S::kB * (kChunkRank / 8) / kThreads;  // 16-byte pieces of a B chunk a thread
  constexpr int kPieces = kChunkRank / 8;           // of 16 bytes in a row
  char* su = lds;                                   // [NMAT][2][kA] rows of u and its low part
  char* sb = lds + NMAT * 2 * S::kA * kAdRow;       // [kB] rows of B
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int wm = S::wm(wave), wn = S::wn(wave), fr = lane & 31, g = lane >> 5;
  int id[kIds];     // rows lane, 64 + lane, ... of the tile: what the block has to do
  int mine_id[NA];  // row fr of the wave's row blocks
#pragma unroll
  for (int v = 0; v < kIds; ++v) id[v] = v * 64 + lane < rows ? ad.rid[row0 + v * 64 + lane] : -1;
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int r = wm * (32 * NA) + i * 32 + fr;
    mine_id[i] = r < rows ? ad.rid[row0 + r] : -1;
  }
  // the next adapter of the block's rows, in the order of their first rows; -1: none left
  auto next = [&](int (&left)[kIds]) {
    int cur = -1;
#pragma unroll
    for (int v = 0; v < kIds; ++v) {
      const uint64_t some = __ballot(left[v] >= 0);
      if (cur < 0 && some != 0) cur = __builtin_amdgcn_readlane(left[v], __builtin_ctzll(some));
    }
#pragma unroll
    for (int v = 0; v < kIds; ++v)
      if (left[v] == cur) left[v] = -1;
    return cur;
  };
  __builtin_amdgcn_s_waitcnt(0xC07F);
  block_barrier();  // every wave is done reading the last stage
  for (int c0 = 0; c0 < ad.rank; c0 += kChunkRank) {
    const int cr = min(kChunkRank, ad.rank - c0);  // a multiple of 8
    const int nkc = (cr + 15) / 16;                // k chunks of 16; the last one's upper half may be zeros
    const u32x4_t zero = {0, 0, 0, 0};
    int left[kIds];
#pragma unroll
    for (int v = 0; v < kIds; ++v) left[v] = id[v];
    int cur = next(left);
    if (cur < 0) return;  // no row of the tile has an adapter
    // load p of a thread: row (tid + p * kThreads) / kPieces of the tile's B rows, piece % kPieces of its chunk
    u32x4_t pb[kBLoads];
    auto load_b = [&](int a) {
#pragma unroll
      for (int p = 0; p < kBLoads; ++p) {
        const int v = tid + p * kThreads, br = v / kPieces, c = (v % kPieces) * 8;
        const int m = NMAT == 2 && br >= S::kB / 2 ? 1 : 0;
        const int col = min(n0 + br - m * (S::kB / 2), N - 1);
        pb[p] = c < cr && ad.u[m] != nullptr
                    ? *reinterpret_cast<const u32x4_t*>(adapter_b<bf16_t>(ad, m, a, expert, col, N) + c0 + c)
                    : zero;
      }
    };
    load_b(cur);
    if (c0 > 0) {
      __builtin_amdgcn_s_waitcnt(0xC07F);
      block_barrier();  // the chunk before has been read
    }
    for (int v = tid; v < NMAT * 2 * S::kA * kPieces; v += kThreads) {
      const int c = (v % kPieces) * 8, r = (v / kPieces) % S::kA, part = v / (kPieces * S::kA), m = part / 2;
      if (c >= nkc * 16 || r >= rows || ad.u[m] == nullptr) continue;
      const bf16_t* u = adapter_u<bf16_t>(ad, m, row0 + r) + (part % 2) * ad.lo + c0 + c;
      *reinterpret_cast<u32x4_t*>(su + (part * S::kA + r) * kAdRow + c * 2) =
          c < cr ? *reinterpret_cast<const u32x4_t*>(u) : zero;
    }
    for (bool first = true; cur >= 0; first = false) {
      if (!first) {
        __builtin_amdgcn_s_waitcnt(0xC07F);
        block_barrier();  // the adapter before has been read
      }
#pragma unroll
      for (int p = 0; p < kBLoads; ++p) {
        const int v = tid + p * kThreads;
        *reinterpret_cast<u32x4_t*>(sb + (v / kPieces) * kAdRow + (v % kPieces) * 16) = pb[p];
      }
      const int following = next(left);
      if (following >= 0) load_b(following);
      __builtin_amdgcn_s_waitcnt(0xC07F);
      block_barrier();
#pragma unroll
      for (int m = 0; m < NMAT; ++m) {
        if (ad.u[m] == nullptr) continue;
        constexpr int NJ = NB / NMAT;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          bf16x8_t fb[kChunkRank / 16];
          const char* br = sb + (m * (S::kB / 2) + (wn * NJ + j) * 32 + fr) * kAdRow + g * 16;
#pragma unroll
          for (int kc = 0; kc < kChunkRank / 16; ++kc)
            if (kc < nkc) fb[kc] = *reinterpret_cast<const bf16x8_t*>(br + kc * 32);
#pragma unroll
          for (int i = 0; i < NA; ++i) {
            const bool own = mine_id[i] == cur;
            if (__ballot(own) == 0) continue;
            const char* ur = su + (2 * m * S::kA + wm * (32 * NA) + i * 32 + fr) * kAdRow + g * 16;
            f32x16_t t;
#pragma unroll
            for (int r = 0; r < 16; ++r) t[r] = 0.0f;
#pragma unroll
            for (int kc = 0; kc < kChunkRank / 16; ++kc)
              if (kc < nkc) {
                t = mma32(fb[kc], *reinterpret_cast<const bf16x8_t*>(ur + kc * 32), t);
                t = mma32(fb[kc], *reinterpret_cast<const bf16x8_t*>(ur + S::kA * kAdRow + kc * 32), t);
              }
            // lane -> token row: the whole column of sums is one row's
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][m * NJ + j][r] = own ? acc[i][m * NJ + j][r] + t[r] : acc[i][m * NJ + j][r];
          }
        }
      }
      cur = following;
    }
  }
}

}  // namespace
}  // namespace moe
