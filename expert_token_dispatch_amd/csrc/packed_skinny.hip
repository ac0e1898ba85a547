// The packed experts' feed-forward for segments of a few rows (decode-sized batches).
//
// The product is bound by streaming the 4-bit weights, 17/32 byte each, so the work is
// split over weight rows and, where those are few, over K.  A wave owns two streams of 16
// weight rows: the gate and the up rows of 16 output columns, or two neighbouring groups
// of 16 output columns of the down product.  Of a block's four waves WK share one pair of
// streams, each every WK-th step of K (summed in LDS in a fixed order), and 4 / WK work on
// neighbouring columns.
//
// A step is 128 k: lane l reads 16 bytes (32 codes, one scale group) of row l % 16 at
// k group l / 16, so a wave instruction reads 16 rows x 64 bytes.  The MFMA sums over k in
// any order as long as both operands agree, so MFMA j of a step simply takes the lane's
// codes 8j .. 8j+7 (k = 32 (l / 16) + 8 j ..) and the token row's elements at the same k.
// The codes turn into bf16 with their scale applied by v_cvt_scalef32_pk_bf16_fp4, two at
// a time, exactly; a step is 16 of them and four MFMAs 16x16x32 per stream and 16 rows.  In
// float32 eight codes are eight MFMAs 16x16x4 instead, in the same places of k.
//
// Measured: 512 rows on 128 experts of H 2048, I 768 72 us, 4.5 TB/s of codes; one row on 8
// of them 13 us, two launches of load latency; float32, 64 rows on 8 experts of 512 x 256 12
// us (34 with the stacks unpacked first).
//
// A chunk of K is four steps of a wave, two where four waves share K, and half as many in
// float32.  The weights of so many steps are in flight in registers while one is multiplied.
// One load brings a row's scales of a chunk (lane group g holds step g's four bytes, handed
// round by a lane permute).  The token rows go through LDS, a chunk at a time, double
// buffered: read straight from memory, 64 bytes a lane and step, they would take the address
// units longer than the weights.
#include <math.h>

#include <algorithm>

#include "ffn_common.h"
#include "kernels.h"
#include "packed.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kStep = 128;   // k of a step

// The `slot`-th expert that has rows (slots are at most the rows, experts may be many and
// mostly empty) and its segment, or -1.  Every wave finds it for itself.
__device__ __forceinline__ int expert_of_slot(const int32_t* __restrict__ offsets, int L, int slot, int& seg0,
                                              int& seg_n) {
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < L; base += 64) {
    const int e = base + lane;
    const int o0 = offsets[min(e, L)], o1 = offsets[min(e + 1, L)];
    const uint64_t m = __ballot(o1 > o0);
    const int n = __popcll(m);
    if (slot < n) {
      const uint64_t hit = __ballot(o1 > o0 && __popcll(m & lanemask_lt()) == slot);
      const int l = __ffsll((unsigned long long)hit) - 1;
      seg0 = __builtin_amdgcn_readlane(o0, l);
      seg_n = __builtin_amdgcn_readlane(o1, l) - seg0;
      return base + l;
    }
    slot -= n;
  }
  return -1;
}

// k of a chunk, and a row's bytes of it in LDS.  16-byte piece c of row r sits at piece
// c ^ (r % 16), so the reads of 16 rows at one piece cover all banks.
template <typename T, int WK>
struct Chunk {
  // steps of a wave: a chunk's, and in flight
  static constexpr int kAhead = (WK == 4 ? 2 : 4) * 2 / int(sizeof(T));
  static constexpr int kSteps = WK * kAhead, kK = kSteps * kStep;
  static constexpr int kRowBytes = kK * int(sizeof(T)), kPieces = kRowBytes / 16;
  static constexpr int kStepBytes = kStep * int(sizeof(T)), kLanePieces = kStepBytes / 64;  // of a row's step, a lane's
};

// Eight codes under one scale times a token row's elements at their k, for every 16 rows:
// piece(rb, i) is the lane's i-th 16-byte piece of the eight.
template <int NRB, typename P>
__device__ __forceinline__ void multiply(bf16_t, const uint32_t (&w)[2], const float (&f)[2], const P& piece,
                                         f32x4_t (&acc)[2][NRB]) {
  const bf16x8_t v0 = decode_frag(w[0], f[0]), v1 = decode_frag(w[1], f[1]);
#pragma unroll
  for (int rb = 0; rb < NRB; ++rb) {
    const bf16x8_t a = *reinterpret_cast<const bf16x8_t*>(piece(rb, 0));
    acc[0][rb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, v0, acc[0][rb], 0, 0, 0);
    acc[1][rb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, v1, acc[1][rb], 0, 0, 0);
  }
}
template <int NRB, typename P>
__device__ __forceinline__ void multiply(float, const uint32_t (&w)[2], const float (&f)[2], const P& piece,
                                         f32x4_t (&acc)[2][NRB]) {
  float v[2][8];
#pragma unroll
  for (int m = 0; m < 2; ++m) decode_f32(w[m], f[m], v[m]);
#pragma unroll
  for (int rb = 0; rb < NRB; ++rb) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4_t a = *reinterpret_cast<const f32x4_t*>(piece(rb, i));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[0][rb] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], v[0][4 * i + e], acc[0][rb], 0, 0, 0);
        acc[1][rb] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], v[1][4 * i + e], acc[1][rb], 0, 0, 0);
      }
    }
  }
}

template <typename T, int NMAT, int WK, int NRB>
__global__ __launch_bounds__(kThreads) void packed_gemm_kernel(const T* __restrict__ A,
                                                               const int32_t* __restrict__ offsets,
                                                               const uint8_t* __restrict__ q0,
                                                               const uint8_t* __restrict__ s0,
                                                               const uint8_t* __restrict__ q1,
                                                               const uint8_t* __restrict__ s1, T* __restrict__ C,
                                                               int L, int N, int K) {
  using Ch = Chunk<T, WK>;
  constexpr int kAhead = Ch::kAhead;
  constexpr int WN = 4 / WK, kRows = 16 * NRB;
  constexpr int kWaveCols = NMAT == 2 ? 16 : 32;
  constexpr int kStage = kRows * Ch::kPieces / kThreads;  // 16-byte pieces of a chunk per thread
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  int seg0 = 0, seg_n = 0;
  const int expert = __builtin_amdgcn_readfirstlane(expert_of_slot(offsets, L, blockIdx.y, seg0, seg_n));
  if (expert < 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wk = wave % WK, wn = wave / WK;
  const int col0 = (blockIdx.x * WN + wn) * kWaveCols;  // first output column of this wave
  const int lr = lane & 15, kg = lane >> 4;
  // rows past N repeat row N - 1 (never stored)
  const int r0 = min(col0 + lr, N - 1), r1 = NMAT == 2 ? r0 : min(col0 + 16 + lr, N - 1);
  // codes by buffer loads over the expert's matrix: a byte offset per lane and stream, the
  // step in the scalar offset; what lies behind the matrix reads as zero
  const uint32_t qbytes = uint32_t(N) * uint32_t(K / 2);
  const size_t eq = size_t(expert) * N * (K / 2), es = size_t(expert) * N * (K / 32);
  const __amdgpu_buffer_rsrc_t rq[2] = {
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(q0 + eq), 0, qbytes, kRsrcFlags),
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>((NMAT == 2 ? q1 : q0) + eq), 0, qbytes, kRsrcFlags)};
  const uint32_t vq[2] = {uint32_t(r0) * uint32_t(K / 2) + 16u * kg, uint32_t(r1) * uint32_t(K / 2) + 16u * kg};
  const uint8_t* ws[2] = {s0 + es + size_t(r0) * (K / 32), (NMAT == 2 ? s1 : s0) + es + size_t(r1) * (K / 32)};
  const int chunks = (K + Ch::kK - 1) / Ch::kK;
  const int groups = K / 32;

  // this wave's u-th step of chunk c is step c * kSteps + u * WK + wk of K.  Behind the last
  // k of a row come the next row's codes: their scales are taken as 2^-127 and the token
  // rows are zero there, so they add nothing.
  u32x4_t w[kAhead][2];
  uint32_t sc[2];
  auto load_w = [&](int c, int u) {
    const int st = c * Ch::kSteps + u * WK + wk;
    if (st * kStep >= K) {  // no such step: zeros
      w[u][0] = w[u][1] = u32x4_t{0, 0, 0, 0};
      return;
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
      w[u][m] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rq[m], vq[m], uint32_t(st) * (kStep / 2), 0));
  };
  // lane group g: the four scale bytes of the wave's step g of the chunk
  auto load_s = [&](int c) {
    const int g0 = (c * Ch::kSteps + (kg % kAhead) * WK + wk) * (kStep / 32);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      uint32_t v = 0;
      if (g0 + 4 <= groups) {
        __builtin_memcpy(&v, ws[m] + g0, 4);
      } else {
        for (int i = 0; i < 3; ++i)
          if (g0 + i < groups) v |= uint32_t(ws[m][g0 + i]) << (8 * i);
      }
      sc[m] = v;
    }
  };

  // the lane's pieces of a token row's step: a quarter of it from piece kLanePieces kg on, turned by lr
  constexpr int kPer = Ch::kLanePieces / 4;  // pieces of eight elements
  int aoff[Ch::kLanePieces];
#pragma unroll
  for (int j = 0; j < Ch::kLanePieces; ++j)
    aoff[j] = lr * Ch::kRowBytes + wk * Ch::kStepBytes + (((Ch::kLanePieces * kg + j) ^ lr) * 16);
  constexpr int kWpr = Ch::kPieces / 64;                      // waves per row of a chunk being staged
  const int srow = wave / kWpr, spart = wave % kWpr;          // this wave stages rows srow, srow + 4 / kWpr, ..
  const int spiece = spart * 64 + lane;

  for (int m0 = 0; m0 < seg_n; m0 += kRows) {
    const int n = min(kRows, seg_n - m0);
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<T*>(A + size_t(seg0 + m0) * K), 0, uint32_t(n) * uint32_t(K) * uint32_t(sizeof(T)), kRsrcFlags);
    u32x4_t stage[kStage];
    auto load_a = [&](int c) {
      // lanes past the end of the row ask for what lies behind the buffer: zeros
      const uint32_t vo = c * Ch::kK + spiece * (16 / int(sizeof(T))) < K ? uint32_t(spiece) * 16u : 0xFFFFFFF0u;
#pragma unroll
      for (int i = 0; i < kStage; ++i) {
        const int r = srow + i * (4 / kWpr);
        if (r < n)
          stage[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                     ra, vo, uint32_t(r) * uint32_t(K) * uint32_t(sizeof(T)) + uint32_t(c) * Ch::kRowBytes, 0));
      }
    };
    auto store_a = [&](int c) {
      char* buf = lds + (c & 1) * kRows * Ch::kRowBytes;
#pragma unroll
      for (int i = 0; i < kStage; ++i) {
        const int r = srow + i * (4 / kWpr);
        if (r < n) *reinterpret_cast<u32x4_t*>(buf + r * Ch::kRowBytes + (spiece ^ (r & 15)) * 16) = stage[i];
      }
    };
    f32x4_t acc[2][NRB];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int rb = 0; rb < NRB; ++rb) acc[m][rb] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    load_a(0);
    load_s(0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load_w(0, u);
    if (m0 > 0) __syncthreads();  // the LDS of the rows before is read out
    store_a(0);
    __syncthreads();
    for (int c = 0; c < chunks; ++c) {
      const char* buf = lds + (c & 1) * kRows * Ch::kRowBytes;
      const bool more = c + 1 < chunks;
      const uint32_t sc0 = sc[0], sc1 = sc[1];
      if (more) {
        load_a(c + 1);
        load_s(c + 1);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        // the scales of step u sit in lane group u, byte kg
        const uint32_t b0 = uint32_t(__shfl(int(sc0), 16 * u + lr, 64)) >> (8 * kg);
        const uint32_t b1 = uint32_t(__shfl(int(sc1), 16 * u + lr, 64)) >> (8 * kg);
        const float f[2] = {__uint_as_float((b0 & 0xFFu) << 23), __uint_as_float((b1 & 0xFFu) << 23)};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // rows past n hold what the LDS held: they reach only outputs that are never stored
          const uint32_t codes[2] = {w[u][0][j], w[u][1][j]};
          multiply<NRB>(T{}, codes, f, [&](int rb, int i) {
            return buf + aoff[j * kPer + i] + rb * 16 * Ch::kRowBytes + u * WK * Ch::kStepBytes;
          }, acc);
        }
        if (more) load_w(c + 1, u);
        __builtin_amdgcn_sched_barrier(0);  // a step's reads stay in the step: registers
      }
      if (more) {
        store_a(c + 1);
        __syncthreads();
      }
    }
    // the waves' sums of one pair of streams, in the order of the waves
    if constexpr (WK > 1) {
      __syncthreads();
      f32x4_t* mine = reinterpret_cast<f32x4_t*>(lds) + wn * (WK - 1) * 2 * NRB * 64;
      if (wk > 0) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int rb = 0; rb < NRB; ++rb) mine[(((wk - 1) * 2 + m) * NRB + rb) * 64 + lane] = acc[m][rb];
      }
      __syncthreads();
      if (wk == 0) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
            for (int k = 0; k < WK - 1; ++k) acc[m][rb] += mine[((k * 2 + m) * NRB + rb) * 64 + lane];
      }
    }
    // lane -> weight row (column of the output) lane & 15, register i -> token row 4 (lane / 16) + i
    if (wk == 0) {
#pragma unroll
      for (int rb = 0; rb < NRB; ++rb) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = rb * 16 + 4 * kg + i;
          if (r < n) {
            T* crow = C + size_t(seg0 + m0 + r) * N;
            if (NMAT == 2) {
              if (col0 + lr < N) crow[col0 + lr] = Elem<T>::from_f32(silu(acc[0][rb][i]) * acc[1][rb][i]);
            } else {
#pragma unroll
              for (int s = 0; s < 2; ++s)
                if (col0 + 16 * s + lr < N) crow[col0 + 16 * s + lr] = Elem<T>::from_f32(acc[s][rb][i]);
            }
          }
        }
      }
    }
  }
}

template <typename T, int NMAT, int WK, int NRB>
moe_status launch_wk(const char* name, const T* A, const int32_t* offsets, const void* q0, const void* s0,
                     const void* q1, const void* s1, T* C, int L, int N, int K, int64_t max_pairs, hipStream_t s) {
  constexpr int cols = (NMAT == 2 ? 16 : 32) * (4 / WK);
  const dim3 grid(unsigned((N + cols - 1) / cols), unsigned(std::min<int64_t>(L, max_pairs)));
  auto kern = packed_gemm_kernel<T, NMAT, WK, NRB>;
  constexpr int kBuf = 16 * NRB * Chunk<T, WK>::kRowBytes;
  constexpr int kRed = 4 * 2 * NRB * 1024;  // an upper bound of the waves' sums
  static_assert(kRed <= kBuf, "the sums fit in one buffer");
  static_assert(2 * kBuf <= 64 * 1024, "the dynamic LDS that a launch may have without an attribute");
  const int lds = K > Chunk<T, WK>::kK ? 2 * kBuf : kBuf;
  MOE_LAUNCH(name, kern, grid, dim3(kThreads), lds, s, A, offsets, static_cast<const uint8_t*>(q0),
             static_cast<const uint8_t*>(s0), static_cast<const uint8_t*>(q1), static_cast<const uint8_t*>(s1), C, L, N,
             K);
  return MOE_OK;
}

// Waves along K: as many as it takes for two blocks a CU, given the experts that can have
// rows, while every wave keeps two steps.  As in the choice of the kernel, rows are the
// most that the descriptor allows (T * top_k without a capacity): a rank that holds part of
// the experts is sent fewer.
template <typename T, int NMAT>
moe_status launch(const char* name, const T* A, const int32_t* offsets, const void* q0, const void* s0,
                  const void* q1, const void* s1, T* C, int L, int N, int K, int64_t max_pairs, hipStream_t s) {
  constexpr int kCols = NMAT == 2 ? 64 : 128;
  const int64_t blocks = (N + kCols - 1) / kCols * std::min<int64_t>(L, max_pairs);
  const int steps = (K + kStep - 1) / kStep;
  const bool many = max_pairs > 8 * int64_t(L);
#define MOE_PACKED(WK_, NRB_) \
  launch_wk<T, NMAT, WK_, NRB_>(name, A, offsets, q0, s0, q1, s1, C, L, N, K, max_pairs, s)
  if (many) return MOE_PACKED(1, 2);
  if (blocks < 256 && steps >= 8) return MOE_PACKED(4, 1);
  if (blocks < 512 && steps >= 4) return MOE_PACKED(2, 1);
  return MOE_PACKED(1, 1);
#undef MOE_PACKED
}

}  // namespace

bool packed_skinny_fits(const moe_layer_desc* d, int64_t max_pairs) {
  // Up to 32 rows an expert on average, one pass of the kernel: past that the tiles of packed_gemm.hip
  // win (16 experts, H = I = 2880, 1024 rows: 112 us here, 95 there), in float32 the unpacked
  // products (8 experts, 1024 x 1024, 512 rows: 92 and 89 us; one expert: 686 and 68).
  // An expert's codes and 32 of its rows are addressed with 32-bit byte offsets.
  const int64_t H = d->hidden, I = d->intermediate;
  return max_pairs <= int64_t(32) * d->local_count && H * I / 2 < (int64_t(1) << 32) - 16 &&
         std::max(H, I) * 32 * int64_t(dtype_bytes(d->dtype)) < (int64_t(1) << 32) - 16;
}

namespace {
template <typename T>
moe_status run(const PackedFfnArgs& a) {
  const moe_layer_desc* d = a.d;
  const int L = d->local_count, H = d->hidden, I = d->intermediate;
  const moe_packed_experts& p = *a.p;
  T* h = static_cast<T*>(a.h);
  const moe_status st = launch<T, 2>("ffn_gate_up", static_cast<const T*>(a.x_sorted), a.offsets, p.gate_codes,
                                     p.gate_scales, p.up_codes, p.up_scales, h, L, I, H, a.max_pairs, a.s);
  if (st != MOE_OK) return st;
  return launch<T, 1>("ffn_down", h, a.offsets, p.down_codes, p.down_scales, p.down_codes, p.down_scales,
                      static_cast<T*>(a.y_sorted), L, H, I, a.max_pairs, a.s);
}
}  // namespace

moe_status launch_packed_skinny(const PackedFfnArgs& a) {
  return a.d->dtype == MOE_BF16 ? run<bf16_t>(a) : run<float>(a);
}

}  // namespace moe
