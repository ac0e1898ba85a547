// The packed experts' feed-forward for segments of a few rows (decode-sized batches).
//
// The product is bound by streaming the 4-bit weights, 17/32 byte each, so the work is
// split over weight rows and, inside a block, over K.  A wave owns two streams of 16
// weight rows: the gate and the up rows of 16 output columns, or two neighbouring groups
// of 16 output columns of the down product.  Of a block's four waves WK share one pair of
// streams, each a K range of its own (summed in LDS in a fixed order), and 4 / WK work on
// neighbouring columns.
//
// A step is 128 k: lane l reads 16 bytes (32 codes, one scale group) of row l % 16 at
// k group l / 16, so a wave instruction reads 16 rows x 64 bytes.  The MFMA sums over k in
// any order as long as both operands agree, so MFMA j of a step simply takes the lane's
// codes 8j .. 8j+7 (k = 32 (l / 16) + 8 j ..) and the token row's elements at the same k.
// The codes turn into bf16 with their scale applied by v_cvt_scalef32_pk_bf16_fp4, two a
// time, exactly; a step is 16 of them and four MFMAs 16x16x32 per stream and 16 rows.
// kBatch steps are loaded before the first is used; several waves a SIMD cover the rest.
#include <math.h>

#include <algorithm>

#include "ffn_common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kMaxRowBlocks = 4;
constexpr int kStep = 128;   // k of a step
constexpr int kBatch = 4;    // steps loaded ahead

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// eight codes -> eight bf16, times the scale
__device__ __forceinline__ bf16x8_t decode_frag(uint32_t w, float s) {
  u32x4_t r;
  r[0] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
  r[1] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
  r[2] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
  r[3] = __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  return __builtin_bit_cast(bf16x8_t, r);
}

// The `slot`-th expert that has rows (slots are at most the rows, experts may be many and
// mostly empty), or -1.  Every wave finds it for itself.
__device__ __forceinline__ int expert_of_slot(const int32_t* __restrict__ offsets, int L, int slot) {
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < L; base += 64) {
    const int e = base + lane;
    const bool has = e < L && offsets[e + 1] > offsets[e];
    const uint64_t m = __ballot(has);
    const int n = __popcll(m);
    if (slot < n) {
      const uint64_t hit = __ballot(has && __popcll(m & lanemask_lt()) == slot);
      return base + __ffsll((unsigned long long)hit) - 1;
    }
    slot -= n;
  }
  return -1;
}

template <int NMAT, int WK>
__global__ __launch_bounds__(kThreads) void packed_gemm_kernel(const bf16_t* __restrict__ A,
                                                               const int32_t* __restrict__ offsets,
                                                               const uint8_t* __restrict__ q0,
                                                               const uint8_t* __restrict__ s0,
                                                               const uint8_t* __restrict__ q1,
                                                               const uint8_t* __restrict__ s1, bf16_t* __restrict__ C,
                                                               int L, int N, int K) {
  constexpr int WN = 4 / WK;
  constexpr int kWaveCols = NMAT == 2 ? 16 : 32;
  const int expert = __builtin_amdgcn_readfirstlane(expert_of_slot(offsets, L, blockIdx.y));
  if (expert < 0) return;
  const int seg0 = offsets[expert], seg_n = offsets[expert + 1] - seg0;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wk = wave % WK, wn = wave / WK;
  const int col0 = (blockIdx.x * WN + wn) * kWaveCols;  // first output column of this wave
  const int lr = lane & 15, kg = lane >> 4;
  // rows past N repeat row N - 1 (never stored)
  const int r0 = min(col0 + lr, N - 1), r1 = NMAT == 2 ? r0 : min(col0 + 16 + lr, N - 1);
  const size_t row0 = size_t(expert) * N + r0, row1 = size_t(expert) * N + r1;
  const uint8_t* wq[2] = {q0 + row0 * (K / 2) + 16 * kg, (NMAT == 2 ? q1 : q0) + row1 * (K / 2) + 16 * kg};
  const uint8_t* ws[2] = {s0 + row0 * (K / 32) + kg, (NMAT == 2 ? s1 : s0) + row1 * (K / 32) + kg};
  // this wave's steps of K: the last one of all may be cut short (K is a multiple of 32)
  const int steps = (K + kStep - 1) / kStep;
  const int st0 = steps * wk / WK, st1 = steps * (wk + 1) / WK;

  __shared__ f32x4_t red[WK > 1 ? WN * (WK - 1) * 2 * kMaxRowBlocks * 64 : 1];

  for (int m0 = 0; m0 < seg_n; m0 += 16 * kMaxRowBlocks) {
    const int nrb = min(kMaxRowBlocks, (seg_n - m0 + 15) / 16);
    const bf16_t* arow[kMaxRowBlocks];
#pragma unroll
    for (int rb = 0; rb < kMaxRowBlocks; ++rb)
      arow[rb] = A + size_t(seg0 + min(m0 + rb * 16 + lr, seg_n - 1)) * K + 32 * kg;
    f32x4_t acc[2][kMaxRowBlocks];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int rb = 0; rb < kMaxRowBlocks; ++rb) acc[m][rb] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    for (int st = st0; st < st1; st += kBatch) {
      u32x4_t w[2][kBatch];
      uint32_t sb[2][kBatch];
      u32x4_t a0[kBatch][4];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int k0 = (st + u) * kStep;
        // a lane's 32 k are inside K as a whole or outside; outside both operands are zero
        const bool in = st + u < st1 && k0 + 32 * kg < K;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          w[m][u] = in ? *reinterpret_cast<const u32x4_t*>(wq[m] + k0 / 2) : u32x4_t{0, 0, 0, 0};
          sb[m][u] = in ? ws[m][k0 / 32] : 0u;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          a0[u][j] = in ? *reinterpret_cast<const u32x4_t*>(arow[0] + k0 + 8 * j) : u32x4_t{0, 0, 0, 0};
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (st + u < st1) {
          const int k0 = (st + u) * kStep;
          const bool in = k0 + 32 * kg < K;
          const float f0 = __uint_as_float(sb[0][u] << 23), f1 = __uint_as_float(sb[1][u] << 23);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bf16x8_t b0 = decode_frag(w[0][u][j], f0), b1 = decode_frag(w[1][u][j], f1);
#pragma unroll
            for (int rb = 0; rb < kMaxRowBlocks; ++rb) {
              if (rb < nrb) {
                u32x4_t av = a0[u][j];
                if (rb > 0) av = in ? *reinterpret_cast<const u32x4_t*>(arow[rb] + k0 + 8 * j) : u32x4_t{0, 0, 0, 0};
                const bf16x8_t a = __builtin_bit_cast(bf16x8_t, av);
                acc[0][rb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b0, acc[0][rb], 0, 0, 0);
                acc[1][rb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b1, acc[1][rb], 0, 0, 0);
              }
            }
          }
        }
      }
    }
    // the K ranges' sums, in the order of the ranges
    if constexpr (WK > 1) {
      f32x4_t* mine = red + wn * (WK - 1) * 2 * kMaxRowBlocks * 64;
      if (m0 > 0) __syncthreads();
      if (wk > 0) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int rb = 0; rb < kMaxRowBlocks; ++rb)
            if (rb < nrb) mine[(((wk - 1) * 2 + m) * kMaxRowBlocks + rb) * 64 + lane] = acc[m][rb];
      }
      __syncthreads();
      if (wk == 0) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int rb = 0; rb < kMaxRowBlocks; ++rb)
            if (rb < nrb)
              for (int k = 0; k < WK - 1; ++k) acc[m][rb] += mine[((k * 2 + m) * kMaxRowBlocks + rb) * 64 + lane];
      }
    }
    // lane -> weight row (column of the output) lane & 15, register i -> token row 4 (lane / 16) + i
    if (wk == 0) {
#pragma unroll
      for (int rb = 0; rb < kMaxRowBlocks; ++rb) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = m0 + rb * 16 + 4 * kg + i;
          if (rb < nrb && r < seg_n) {
            bf16_t* crow = C + size_t(seg0 + r) * N;
            if (NMAT == 2) {
              if (col0 + lr < N) crow[col0 + lr] = f32_to_bf16(silu(acc[0][rb][i]) * acc[1][rb][i]);
            } else {
#pragma unroll
              for (int s = 0; s < 2; ++s)
                if (col0 + 16 * s + lr < N) crow[col0 + 16 * s + lr] = f32_to_bf16(acc[s][rb][i]);
            }
          }
        }
      }
    }
  }
}

template <int NMAT, int WK>
moe_status launch_wk(const char* name, const bf16_t* A, const int32_t* offsets, const void* q0, const void* s0,
                     const void* q1, const void* s1, bf16_t* C, int L, int N, int K, int64_t max_pairs, hipStream_t s) {
  constexpr int cols = (NMAT == 2 ? 16 : 32) * (4 / WK);
  const dim3 grid(unsigned((N + cols - 1) / cols), unsigned(std::min<int64_t>(L, max_pairs)));
  MOE_LAUNCH(name, (packed_gemm_kernel<NMAT, WK>), grid, dim3(kThreads), 0, s, A, offsets,
             static_cast<const uint8_t*>(q0), static_cast<const uint8_t*>(s0), static_cast<const uint8_t*>(q1),
             static_cast<const uint8_t*>(s1), C, L, N, K);
  return MOE_OK;
}

// Waves along K: four from eight steps of 128 on (two steps or more each), else two.
template <int NMAT>
moe_status launch(const char* name, const bf16_t* A, const int32_t* offsets, const void* q0, const void* s0,
                  const void* q1, const void* s1, bf16_t* C, int L, int N, int K, int64_t max_pairs, hipStream_t s) {
  if (K >= 8 * kStep) return launch_wk<NMAT, 4>(name, A, offsets, q0, s0, q1, s1, C, L, N, K, max_pairs, s);
  return launch_wk<NMAT, 2>(name, A, offsets, q0, s0, q1, s1, C, L, N, K, max_pairs, s);
}

}  // namespace

bool packed_skinny_fits(const moe_layer_desc* d, int64_t max_pairs) {
  return d->dtype == MOE_BF16 && max_pairs <= int64_t(32) * d->local_count;
}

moe_status launch_packed_skinny(const PackedFfnArgs& a) {
  const moe_layer_desc* d = a.d;
  const int L = d->local_count, H = d->hidden, I = d->intermediate;
  const moe_packed_experts& p = *a.p;
  bf16_t* h = static_cast<bf16_t*>(a.h);
  const moe_status st = launch<2>("ffn_gate_up", static_cast<const bf16_t*>(a.x_sorted), a.offsets, p.gate_codes,
                                  p.gate_scales, p.up_codes, p.up_scales, h, L, I, H, a.max_pairs, a.s);
  if (st != MOE_OK) return st;
  return launch<1>("ffn_down", h, a.offsets, p.down_codes, p.down_scales, p.down_codes, p.down_scales,
                   static_cast<bf16_t*>(a.y_sorted), L, H, I, a.max_pairs, a.s);
}

}  // namespace moe
