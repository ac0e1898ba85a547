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
