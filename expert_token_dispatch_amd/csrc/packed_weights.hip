// Expert weights in 4 bits: packing a stack, and unpacking it.
//
// A stack of `count` matrices, each `out` x `in`, is held as codes
// [count, out, in / 2] (two 4-bit e2m1 codes a byte, the lower input in the low
// half) and scales [count, out, in / 32] (one e8m0 byte per 32 inputs of one
// output), whatever layout the weights themselves have.  A code's value is
// +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}, a scale byte b stands for 2^(b - 127), so a
// weight is value * 2^(b - 127): at most two significant bits, exact in bf16 and
// float32.  Per group of 32: b = clamp(floor(log2 max|w|) - 2 + 127, 0, 254), and
// each w / 2^(b - 127) goes to the nearest code, ties to the even one, +-6 at most.
// A group that holds a NaN or an infinity gets b = 255, and its weights are NaN.
//
// gfx950 converts between packed fp4 and float32 or bf16 pairs with the power-of-two
// scale applied (v_cvt_scalef32_pk_*): it takes the scale operand's exponent field
// as the e8m0 byte, so a byte is used as `byte << 23` (0 is 2^-127, 255 gives NaN),
// rounds to nearest even and saturates at 6 (both checked on the GPU).
//
// Both directions are bound by HBM: (dt + 17/32) bytes per weight each (16 x 2880 x 2880 in
// bfloat16, stored [in, out]: packed in 85 us, 4.0 TB/s, unpacked in 71 us, 4.7 TB/s).
#include <stdint.h>

#include "common.h"
#include "kernels.h"
#include "packed.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 32;

// Eight consecutive inputs of one output, as float32.
__device__ __forceinline__ void load8(const bf16_t* p, float* f) {
  unpack16(*reinterpret_cast<const uint4*>(p), bf16_t{}, f);
}
__device__ __forceinline__ void load8(const float* p, float* f) {
  unpack16(reinterpret_cast<const uint4*>(p)[0], float{}, f);
  unpack16(reinterpret_cast<const uint4*>(p)[1], float{}, f + 4);
}

// The four lanes of a group hold eight weights each: its scale byte.  The largest
// magnitude's exponent field is the largest of the fields, and NaN and infinity
// have the largest field of all.
__device__ __forceinline__ uint32_t group_scale(const float* f) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7F800000u);
  m = max(m, uint32_t(__shfl_xor(int(m), 1, 64)));
  m = max(m, uint32_t(__shfl_xor(int(m), 2, 64)));
  const uint32_t ef = m >> 23;
  return ef == 255 ? 255u : (ef > 2 ? ef - 2 : 0u);
}

__device__ __forceinline__ uint32_t encode8(const float* f, uint32_t byte) {
  const float s = __uint_as_float(byte << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[0], f[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2], f[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4], f[5], s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6], f[7], s, 3);
  return w;
}

__device__ __forceinline__ void decode8(uint32_t w, uint32_t byte, bf16_t* o) {
  *reinterpret_cast<bf16x8_t*>(o) = decode_frag(w, __uint_as_float(byte << 23));
}
__device__ __forceinline__ void decode8(uint32_t w, uint32_t byte, float* o) {
  decode_f32(w, __uint_as_float(byte << 23), o);
}

// Weights stored [out, in]: the stack is one run of units of eight weights, a lane
// each (16 or 32 bytes of weights, four of codes), a group to four neighbours.
// units is a multiple of four, so the lanes of a group leave the loop together.
template <typename T>
__global__ __launch_bounds__(kThreads) void pack_rows_kernel(const T* __restrict__ w, uint32_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scales, int64_t units) {
  const int64_t step = int64_t(gridDim.x) * kThreads;
  for (int64_t u = int64_t(blockIdx.x) * kThreads + threadIdx.x; u < units; u += step) {
    float f[8];
    load8(w + u * 8, f);
    const uint32_t byte = group_scale(f);
    codes[u] = encode8(f, byte);
    if ((u & 3) == 0) scales[u >> 2] = uint8_t(byte);
  }
}

template <typename T>
__device__ __forceinline__ void unpack_rows(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                            T* __restrict__ w, int64_t units) {
  const int64_t step = int64_t(gridDim.x) * kThreads;
  for (int64_t u = int64_t(blockIdx.x) * kThreads + threadIdx.x; u < units; u += step) {
    __attribute__((aligned(16))) T o[8];
    decode8(codes[u], scales[u >> 2], o);
#pragma unroll
    for (int i = 0; i < int(sizeof(o) / 16); ++i)
      reinterpret_cast<uint4*>(w + u * 8)[i] = reinterpret_cast<const uint4*>(o)[i];
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void unpack_rows_kernel(const uint32_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, T* __restrict__ w,
                                                               int64_t units) {
  unpack_rows(codes, scales, w, units);
}

// Weights stored [in, out]: a block turns a tile of kTI inputs x kTO outputs round in
// LDS, so that the weights move in whole pieces of an input's row and the codes in
// whole pieces of an output's.  Rows of the LDS tile are one element longer than the
// tile (odd in 4-byte words for float32, 33 words for bf16), so reading down a column
// passes over the banks.
constexpr int kTI = 128, kTO = 64;

template <typename T>
struct Tile {
  static constexpr int kLd = kTO + (sizeof(T) == 2 ? 2 : 1);
  static constexpr int kVec = 16 / int(sizeof(T));  // elements of a 16-byte piece
};

template <typename T>
__global__ __launch_bounds__(kThreads) void pack_cols_kernel(const T* __restrict__ w, uint32_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scales, int out, int in) {
  using S = Tile<T>;
  __shared__ T t[kTI * S::kLd];
  const int i0 = blockIdx.x * kTI, o0 = blockIdx.y * kTO;
  const size_t m = blockIdx.z;
  const T* wm = w + m * size_t(in) * out;
  constexpr int kPieces = kTO / S::kVec;
  for (int p = threadIdx.x; p < kTI * kPieces; p += kThreads) {
    const int i = p / kPieces, o = (p % kPieces) * S::kVec;
    T v[S::kVec] = {};
    if (i0 + i < in && o0 + o < out)  // out is a multiple of 8: a piece is inside or outside as a whole
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(wm + size_t(i0 + i) * out + o0 + o);
#pragma unroll
    for (int k = 0; k < S::kVec; ++k) t[i * S::kLd + o + k] = v[k];
  }
  __syncthreads();
  constexpr int kUnits = kTI / 8;  // units of eight inputs, 16 neighbouring lanes to an output
  for (int p = threadIdx.x; p < kTO * kUnits; p += kThreads) {
    const int o = p / kUnits, i = (p % kUnits) * 8;
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = Elem<T>::to_f32(t[(i + k) * S::kLd + o]);
    const uint32_t byte = group_scale(f);
    if (i0 + i < in && o0 + o < out) {  // in is a multiple of 32: a group is inside or outside as a whole
      const size_t row = m * out + o0 + o;
      codes[(row * in + i0 + i) / 8] = encode8(f, byte);
      if ((p & 3) == 0) scales[(row * in + i0 + i) / kGroup] = uint8_t(byte);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void unpack_cols_kernel(const uint32_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, T* __restrict__ w,
                                                               int out, int in) {
  using S = Tile<T>;
  __shared__ T t[kTI * S::kLd];
  const int i0 = blockIdx.x * kTI, o0 = blockIdx.y * kTO;
  const size_t m = blockIdx.z;
  constexpr int kUnits = kTI / 8;
  for (int p = threadIdx.x; p < kTO * kUnits; p += kThreads) {
    const int o = p / kUnits, i = (p % kUnits) * 8;
    if (i0 + i < in && o0 + o < out) {
      const size_t at = (m * out + o0 + o) * in + i0 + i;
      __attribute__((aligned(16))) T v[8];
      decode8(codes[at / 8], scales[at / kGroup], v);
#pragma unroll
      for (int k = 0; k < 8; ++k) t[(i + k) * S::kLd + o] = v[k];
    }
  }
  __syncthreads();
  T* wm = w + m * size_t(in) * out;
  constexpr int kPieces = kTO / S::kVec;
  for (int p = threadIdx.x; p < kTI * kPieces; p += kThreads) {
    const int i = p / kPieces, o = (p % kPieces) * S::kVec;
    if (i0 + i < in && o0 + o < out) {
      __attribute__((aligned(16))) T v[S::kVec];
#pragma unroll
      for (int k = 0; k < S::kVec; ++k) v[k] = t[i * S::kLd + o + k];
      *reinterpret_cast<uint4*>(wm + size_t(i0 + i) * out + o0 + o) = *reinterpret_cast<const uint4*>(v);
    }
  }
}

// Three stacks stored [out, in] in one launch (y: which).
struct Unpack3 {
  const uint32_t* codes[3];
  const uint8_t* scales[3];
  void* w[3];
};
template <typename T>
__global__ __launch_bounds__(kThreads) void unpack3_rows_kernel(Unpack3 a, int64_t units) {
  const int i = blockIdx.y;
  unpack_rows(a.codes[i], a.scales[i], static_cast<T*>(a.w[i]), units);
}

unsigned row_blocks(int64_t units) {
  const int64_t b = (units + kThreads - 1) / kThreads;
  return unsigned(b < 16384 ? b : 16384);
}

template <typename T>
moe_status launch_pack_t(const char* name, const PackArgs& a) {
  const int64_t units = int64_t(a.count) * a.out * a.in / 8;
  const T* w = static_cast<const T*>(a.w);
  if (a.layout == MOE_WEIGHTS_OUT_IN) {
    MOE_LAUNCH(name, pack_rows_kernel<T>, dim3(row_blocks(units)), dim3(kThreads), 0, a.s, w,
               static_cast<uint32_t*>(a.codes), static_cast<uint8_t*>(a.scales), units);
  } else {
    MOE_LAUNCH(name, pack_cols_kernel<T>, dim3((a.in + kTI - 1) / kTI, (a.out + kTO - 1) / kTO, a.count),
               dim3(kThreads), 0, a.s, w, static_cast<uint32_t*>(a.codes), static_cast<uint8_t*>(a.scales), a.out, a.in);
  }
  return MOE_OK;
}

template <typename T>
moe_status launch_unpack_t(const char* name, const PackArgs& a) {
  const int64_t units = int64_t(a.count) * a.out * a.in / 8;
  T* w = static_cast<T*>(a.w);
  if (a.layout == MOE_WEIGHTS_OUT_IN) {
    MOE_LAUNCH(name, unpack_rows_kernel<T>, dim3(row_blocks(units)), dim3(kThreads), 0, a.s,
               static_cast<const uint32_t*>(a.codes), static_cast<const uint8_t*>(a.scales), w, units);
  } else {
    MOE_LAUNCH(name, unpack_cols_kernel<T>, dim3((a.in + kTI - 1) / kTI, (a.out + kTO - 1) / kTO, a.count),
               dim3(kThreads), 0, a.s, static_cast<const uint32_t*>(a.codes), static_cast<const uint8_t*>(a.scales), w,
               a.out, a.in);
  }
  return MOE_OK;
}

}  // namespace

moe_status launch_pack(const char* name, const PackArgs& a) {
  return a.dtype == MOE_BF16 ? launch_pack_t<bf16_t>(name, a) : launch_pack_t<float>(name, a);
}
moe_status launch_unpack(const char* name, const PackArgs& a) {
  return a.dtype == MOE_BF16 ? launch_unpack_t<bf16_t>(name, a) : launch_unpack_t<float>(name, a);
}

// ---- the experts' feed-forward on packed weights -------------------------------------
// The products read the codes themselves (packed_skinny.hip for both types, packed_gemm.hip
// for bf16).  For more float32 rows, and experts too large for those kernels' 32-bit offsets, the three
// stacks are unpacked into the workspace and the products run on them: the unpacked
// stacks hold the same values as the codes, so nothing is rounded on the way.
namespace {
size_t stack_bytes(const moe_layer_desc* d) {
  return align_up(size_t(d->local_count) * d->hidden * d->intermediate * dtype_bytes(d->dtype), 256);
}
}  // namespace

size_t packed_ffn_scratch_bytes(const moe_layer_desc* d, int64_t max_pairs) {
  if (packed_skinny_fits(d, max_pairs) || packed_gemm_fits(d, max_pairs)) return 0;
  return 3 * stack_bytes(d) + align_up(ffn_scratch_bytes(d, max_pairs), 256);
}

moe_status launch_packed_ffn(const PackedFfnArgs& a) {
  if (a.max_pairs <= 0) return MOE_OK;
  if (packed_skinny_fits(a.d, a.max_pairs)) return launch_packed_skinny(a);
  if (packed_gemm_fits(a.d, a.max_pairs)) return launch_packed_gemm(a);
  const moe_layer_desc* d = a.d;
  char* base = static_cast<char*>(a.scratch);
  void* w[3];
  for (int i = 0; i < 3; ++i) w[i] = base + size_t(i) * stack_bytes(d);
  const moe_packed_experts& p = *a.p;
  Unpack3 u{};
  const void* codes[3] = {p.gate_codes, p.up_codes, p.down_codes};
  const void* scales[3] = {p.gate_scales, p.up_scales, p.down_scales};
  for (int i = 0; i < 3; ++i) {
    u.codes[i] = static_cast<const uint32_t*>(codes[i]);
    u.scales[i] = static_cast<const uint8_t*>(scales[i]);
    u.w[i] = w[i];
  }
  const int64_t units = int64_t(d->local_count) * d->hidden * d->intermediate / 8;
  if (d->dtype == MOE_BF16) {
    MOE_LAUNCH("ffn_unpack", unpack3_rows_kernel<bf16_t>, dim3(row_blocks(units), 3), dim3(kThreads), 0, a.s, u, units);
  } else {
    MOE_LAUNCH("ffn_unpack", unpack3_rows_kernel<float>, dim3(row_blocks(units), 3), dim3(kThreads), 0, a.s, u, units);
  }
  moe_layer_desc dl = *d;
  dl.weight_layout = MOE_WEIGHTS_OUT_IN;  // the unpacked stacks' layout, whatever the layer's own
  FfnArgs f{&dl, a.x_sorted, a.offsets, w[0], w[1], w[2], a.y_sorted, a.h, base + 3 * stack_bytes(d), a.max_pairs, a.s};
  return launch_grouped_ffn(f);
}

}  // namespace moe
