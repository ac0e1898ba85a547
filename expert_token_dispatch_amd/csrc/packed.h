// What the kernels on 4-bit weights share.
#pragma once

#include "ffn_common.h"

namespace moe {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Eight e2m1 codes -> eight bf16, times the scale (a power of two: its exponent field counts).
__device__ __forceinline__ bf16x8_t decode_frag(uint32_t w, float s) {
  u32x4_t r;
  r[0] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
  r[1] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
  r[2] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
  r[3] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  return __builtin_bit_cast(bf16x8_t, r);
}

// The same to float32.
__device__ __forceinline__ void decode_f32(uint32_t w, float s, float* o) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1),
                   __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = v[i].x;
    o[2 * i + 1] = v[i].y;
  }
}

}  // namespace moe
