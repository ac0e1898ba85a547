// Low-rank adapters beside the experts' products: what a product's epilogue adds.
#pragma once

#include "common.h"
#include "kernels.h"

namespace moe {

// Row `row` of u (matrix m) and column `col` of N of adapter a's B, both rows of `rank` elements.
template <typename T>
__device__ __forceinline__ const T* adapter_u(const Adapters& ad, int m, int row) {
  return static_cast<const T*>(ad.u[m]) + size_t(row) * ad.ldu;
}
template <typename T>
__device__ __forceinline__ const T* adapter_b(const Adapters& ad, int m, int a, int expert, int col, int N) {
  return static_cast<const T*>(ad.b[m]) + ((size_t(a) * ad.experts + expert) * N + col) * ad.rank;
}

// ---- infinities and NaN in B (bfloat16).  u B^T is formed from u's two parts.  An infinity of B takes the
// sign of u, which is its high part's: the low part may be zero, or of the other sign, and would make
// the sum NaN.  So where a wave's fragments of B hold any, the low part's product is that of the finite ones.
typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));

// the largest exponents of a fragment's values and those before
__device__ __forceinline__ u16x2_t largest_exponents(u16x2_t most, const u32x4_t& b) {
#pragma unroll
  for (int r = 0; r < 4; ++r) most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2_t, b[r] & 0x7F807F80u));
  return most;
}
__device__ __forceinline__ bool all_finite(u16x2_t most) {  // in every lane
  return __ballot(most[0] == 0x7F80 || most[1] == 0x7F80) == 0;
}
__device__ __forceinline__ u32x4_t finite_ones(u32x4_t b) {  // zeros for the others
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    b[r] = (b[r] & 0x7F80u) == 0x7F80u ? b[r] & 0xFFFF0000u : b[r];
    b[r] = (b[r] & 0x7F800000u) == 0x7F800000u ? b[r] & 0xFFFFu : b[r];
  }
  return b;
}

// The y-th expert that has rows, -1 past the last.  The lanes look at four experts each: 256 cost one
// round of loads.
__device__ __forceinline__ int expert_with_rows(const int32_t* __restrict__ offsets, int L, int y) {
  const int lane = threadIdx.x & 63;
  for (int i0 = 0; i0 < L; i0 += 256) {
    int off[5];
#pragma unroll
    for (int j = 0; j < 5; ++j) off[j] = offsets[min(i0 + 4 * lane + j, L)];
    uint32_t has = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) has |= uint32_t(off[j + 1] > off[j]) << j;
    const int own = __popc(has);
    int upto = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d, 64);
      if (lane >= d) upto += v;
    }
    const uint64_t past = __ballot(upto > y);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      uint32_t bits = uint32_t(__builtin_amdgcn_readlane(int(has), l));
      for (int r = y - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(own, l)); r > 0; --r) bits &= bits - 1;
      return i0 + 4 * l + __builtin_ctz(bits);
    }
    y -= __builtin_amdgcn_readlane(upto, 63);
  }
  return -1;
}

}  // namespace moe
