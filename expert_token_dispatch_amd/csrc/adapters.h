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

}  // namespace moe
