// The adapters' share of a tile of token rows by weight rows, for the products whose accumulators
// have the weight rows as the left operand (grouped_gemm.hip, adapted_gemm.hip).
#pragma once

#include "adapters.h"

namespace moe {
namespace {

// ---- adapters.  A tile's sums get the adapters' share before they are rounded: u's two parts
// by the adapter's B, for one adapter of the tile's rows after another (one or two in a prompt,
// whose requests follow each other; all of them in a large decode batch).  Of every rank chunk of up
// to 32, the tile's rows of u go to LDS once and an adapter's rows of B (the tile's columns) after
// them by direct loads, three steps ahead; adapters of up to 16 ranks take half a chunk and go two a
// step.  u's rows of other adapters enter a product as zeros, which leave a row's sum as it is; where
// B holds infinities or NaN the sums of those rows are taken back instead, so that neither a row's
// sum nor what a broken adapter spoils depends on the rows beside it.
// 8177 rows of 19 adapters of rank 16 in random order on 25 experts of 384 x 3008, gate and up: 205 us
// against 256 with one adapter a step, its B through registers and its sums formed apart, and 82
// without adapters.  16384 rows in 8 requests, rank 64, 4096 x 14336 experts: gate and up 3.6 ms
// either way, 3.1 without.

// s_waitcnt's operand that waits until at most n loads are in flight
constexpr int vm_count(int n) { return (n & 0xF) | (n >> 4) << 14 | 0x7 << 4 | 0xF << 8; }

constexpr int kChunkRank = 32, kAdapterSlots = 4;
// the LDS it takes, from the tile's operands' (every load into them has landed)
template <class S, int NMAT>
constexpr int kTileAdapterLds = (NMAT * 2 * S::kA + kAdapterSlots * S::kB) * kChunkRank * 2;

__device__ __forceinline__ f32x16_t mma32(bf16x8_t b, bf16x8_t a, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, a, c, 0, 0, 0);
}

// S: the tile's rows kA and kB (with NMAT = 2 half of kB gate, half up), kThreads, 32-column blocks a
// wave NB, and the wave's place wm, wn.  A wave has NA row blocks.
template <class S, int NMAT, int NA>
__device__ __forceinline__ void tile_adapters(const Adapters& ad, int expert, int row0, int rows, int n0, int N,
                                              char* lds, f32x16_t (&acc)[NA][S::NB]) {
  constexpr int NB = S::NB, NJ = NB / NMAT, kWaves = S::kThreads / 64, kIds = S::kA / 64, KC = kChunkRank / 16;
  constexpr int kUPlane = S::kA * 32, kBPlane = S::kB * 32, kBSlot = KC * kBPlane;
  constexpr int kULoads = NMAT * 2 * KC * (S::kA / 32) / kWaves, kBLoads = KC * (S::kB / 32) / kWaves;  // a wave's
  constexpr uint32_t kOutside = 0xFFFFFFF0u;  // past every extent below: zeros, without a memory access
  char* su = lds;                            // planes [NMAT][2][KC] of kA rows of u and of its low part
  char* sb = lds + NMAT * 2 * KC * kUPlane;  // slots of planes [KC] of kB rows of B
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = S::wm(wave), wn = S::wn(wave), fr = lane & 31, g = lane >> 5;
  // a plane's row has two pieces of 16 bytes, which change places every eight rows: 16 rows' reads of one
  // piece fall in different banks
  const int in_row = ((lane & 1) ^ ((lane >> 4) & 1)) * 8;  // what this lane of a load brings
  const int at = fr * 32 + (g ^ ((fr >> 3) & 1)) * 16;  // what this lane of a product reads
  int id[kIds];     // rows lane, 64 + lane, ... of the tile: what the block has to do
  int mine_id[NA];  // row fr of the wave's row blocks
#pragma unroll
  for (int v = 0; v < kIds; ++v) id[v] = v * 64 + lane < rows ? ad.rid[row0 + v * 64 + lane] : -1;
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int r = wm * (32 * NA) + i * 32 + fr;
    mine_id[i] = r < rows ? ad.rid[row0 + r] : -1;
  }
  const bool two = ad.rank <= 16;  // an adapter takes half a chunk: two of them a step
  for (int c0 = 0; c0 < ad.rank; c0 += kChunkRank) {
    const int cr = min(kChunkRank, ad.rank - c0);  // a multiple of 8
    const int nkc = (cr + 15) / 16;                // planes; the last one's upper half may be zeros
    int left[kIds];
#pragma unroll
    for (int v = 0; v < kIds; ++v) left[v] = id[v];
    // the next adapter of the block's rows, in the order of their first rows; -2: none left
    auto next = [&]() {
      int cur = -2;
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
    int todo[kAdapterSlots][2];  // this step's adapter or two, and those of the steps whose loads are in flight
    auto step = [&](int (&of)[2]) {
      of[0] = next();
      of[1] = two ? next() : -2;
    };
    auto load_b = [&](const int (&of)[2], int slot) {
#pragma unroll
      for (int j = 0; j < kBLoads; ++j) {
        const int b = wave * kBLoads + j, kc = b / (S::kB / 32), r0 = b % (S::kB / 32) * 32;
        const int m = NMAT == 2 && r0 >= S::kB / 2 ? 1 : 0, a = two && kc > 0 ? of[1] : of[0];
        const int c = (two ? 0 : kc * 16) + in_row;
        const bool there = a >= 0 && ad.u[m] != nullptr;
        const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<bf16_t*>(adapter_b<bf16_t>(ad, m, there ? a : 0, expert, n0, N)), 0,
            there ? uint32_t(min(S::kB / NMAT, N - n0)) * uint32_t(ad.rank) * 2u : 0u, kRsrcFlags);
        const int r = r0 - m * (S::kB / 2) + (lane >> 1);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr_t)(sb + slot * kBSlot + kc * kBPlane + r0 * 32), 16,
                                                 c < cr ? uint32_t(r * ad.rank + c0 + c) * 2u : kOutside, 0, 0, 0);
      }
    };
    step(todo[0]);
    if (todo[0][0] < 0) return;  // no row of the tile has an adapter
    __builtin_amdgcn_s_waitcnt(0xC07F);
    block_barrier();  // every wave is done reading the last stage, or the chunk before
#pragma unroll
    for (int j = 0; j < kULoads; ++j) {
      const int b = wave * kULoads + j, plane = b / (S::kA / 32), r0 = b % (S::kA / 32) * 32;
      const int m = plane / (2 * KC), part = plane / KC % 2, kc = plane % KC, c = kc * 16 + in_row;
      const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<bf16_t*>(adapter_u<bf16_t>(ad, m, row0) + part * ad.lo), 0,
          ad.u[m] != nullptr ? uint32_t(rows) * uint32_t(ad.ldu) * 2u : 0u, kRsrcFlags);
      const int r = r0 + (lane >> 1);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr_t)(su + plane * kUPlane + r0 * 32), 16,
                                               c < cr && r < rows ? uint32_t(r * ad.ldu + c0 + c) * 2u : kOutside, 0,
                                               0, 0);
    }
    load_b(todo[0], 0);
#pragma unroll
    for (int d = 1; d < kAdapterSlots - 1; ++d) {
      step(todo[d]);
      load_b(todo[d], d);
    }
    for (int s = 0; todo[0][0] >= 0; ++s) {
      __builtin_amdgcn_s_waitcnt(vm_count(kBLoads * (kAdapterSlots - 2)));  // this wave's loads of step s have landed
      block_barrier();  // every wave's have, and the step before has been read
      step(todo[kAdapterSlots - 1]);
      load_b(todo[kAdapterSlots - 1], (s + kAdapterSlots - 1) % kAdapterSlots);  // into the slot of step s - 1
      const char* sbb = sb + s % kAdapterSlots * kBSlot;
#pragma unroll
      for (int m = 0; m < NMAT; ++m) {
        if (ad.u[m] == nullptr) continue;
        bf16x8_t fb[NJ][KC];
        u16x2_t most = {0, 0};  // the largest exponents of B's values
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int kc = 0; kc < KC; ++kc) {
            const u32x4_t b =
                *reinterpret_cast<const u32x4_t*>(sbb + kc * kBPlane + (m * (S::kB / 2) + (wn * NJ + j) * 32) * 32 + at);
            most = largest_exponents(most, b);
            fb[j][kc] = __builtin_bit_cast(bf16x8_t, b);
          }
        const bool finite = all_finite(most);
#pragma unroll
        for (int i = 0; i < NA; ++i) {
#pragma unroll
          for (int kc = 0; kc < KC; ++kc) {
            const bool own = mine_id[i] == (two ? todo[0][kc] : todo[0][0]);
            if (__ballot(own) == 0 || (!two && kc >= nkc)) continue;
            const char* ur = su + (m * 2 * KC + (two ? 0 : kc)) * kUPlane + (wm * NA + i) * 32 * 32 + at;
            u32x4_t hi = *reinterpret_cast<const u32x4_t*>(ur);
            u32x4_t lo = *reinterpret_cast<const u32x4_t*>(ur + KC * kUPlane);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              hi[r] = own ? hi[r] : 0;
              lo[r] = own ? lo[r] : 0;
            }
            const bf16x8_t uh = __builtin_bit_cast(bf16x8_t, hi), ul = __builtin_bit_cast(bf16x8_t, lo);
            if (finite) {
#pragma unroll
              for (int j = 0; j < NJ; ++j) acc[i][m * NJ + j] = mma32(fb[j][kc], uh, acc[i][m * NJ + j]);
#pragma unroll
              for (int j = 0; j < NJ; ++j) acc[i][m * NJ + j] = mma32(fb[j][kc], ul, acc[i][m * NJ + j]);
            } else {
#pragma unroll
              for (int j = 0; j < NJ; ++j) {
                const bf16x8_t fl = __builtin_bit_cast(bf16x8_t, finite_ones(__builtin_bit_cast(u32x4_t, fb[j][kc])));
                const f32x16_t t = mma32(fl, ul, mma32(fb[j][kc], uh, acc[i][m * NJ + j]));
                // lane -> token row: the whole column of sums is one row's
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][m * NJ + j][r] = own ? t[r] : acc[i][m * NJ + j][r];
              }
            }
          }
        }
      }
#pragma unroll
      for (int d = 0; d + 1 < kAdapterSlots; ++d) {
        todo[d][0] = todo[d + 1][0];
        todo[d][1] = todo[d + 1][1];
      }
    }
    __builtin_amdgcn_s_waitcnt(vm_count(0));  // the steps that were not there: zeros land before the LDS is used again
  }
}

}  // namespace
}  // namespace moe
