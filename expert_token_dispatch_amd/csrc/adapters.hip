// Low-rank adapters of many requests beside the experts' projections, the first product:
//   u[q, r] = s_a * sum_k x[q, k] A[a, e, r, k]
// for sorted row q of expert e whose token has adapter a.  The second product, u B^T, is added
// by the epilogues of the experts' own products.
//
// A block takes 16 RB rows of one expert and finds the adapters among them (ids come in any
// order; tokens of one request follow each other in a prompt and are strangers in a decode
// batch).  For one adapter after another it multiplies all its rows by that adapter's A and
// keeps the rows that are its own: a row costs no more than its block's adapters, and an
// adapter's A is read once a block.  A non-finite value in one request's adapter reaches no
// other request.  The eight waves split K, 16-byte vectors straight from memory into MFMA
// fragments, and their sums meet in LDS in a fixed order.
#include <algorithm>

#include "adapters.h"
#include "kernels.h"

namespace moe {
namespace {

struct ShrinkP {
  const void* x;            // [P_max, K]
  const int32_t* offsets;   // [L + 1]
  const int32_t* pairs;     // sorted_pairs, or NULL: rid holds the rows' adapters already
  const int32_t* ids;       // [T] adapter of every token
  int32_t* rid;             // [P_max] adapter of every row, -1: none
  const float* scale;       // [count] or NULL
  const void* a[2];         // [count, L, rank, K] of up to two matrices
  void* u;                  // [P_max, ldu]: matrix m's columns start at m * rank
  int ldu, rank, count, mats, L, K, top_k;
};

constexpr int kWaves = 8;

template <typename T> struct Mma16;
template <> struct Mma16<bf16_t> {  // 16 bytes a lane are 32 k of 16 rows
  static constexpr int kStep = 32;
  __device__ static f32x4_t mma(const u32x4_t& a, const u32x4_t& b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                   0, 0);
  }
};
template <> struct Mma16<float> {  // 16 k, in four products of one k of each lane group
  static constexpr int kStep = 16;
  __device__ static f32x4_t mma(const u32x4_t& a, const u32x4_t& b, f32x4_t c) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[i]), __uint_as_float(b[i]), c, 0, 0, 0);
    return c;
  }
};

// NG groups of 16 of the mats * rank columns a block (blockIdx.z / slots); of its rows' adapters it
// takes every slots-th (blockIdx.z % slots).
template <typename T, int RB, int NG>
__global__ __launch_bounds__(kWaves * 64) void shrink_kernel(ShrinkP p, int slots) {
  constexpr int E = Elem<T>::kPerVec, kStep = Mma16<T>::kStep;
  constexpr int kSteps = RB * NG <= 2 ? 4 : 2;  // steps of K loaded together
  __shared__ float red[kWaves][16][NG * 16];
  const int e = blockIdx.x, seg0 = p.offsets[e], n = p.offsets[e + 1] - seg0;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int slot = blockIdx.z % slots, c0 = (blockIdx.z / slots) * NG * 16, cols = p.mats * p.rank;
  const T* x = static_cast<const T*>(p.x);
  for (int m0 = blockIdx.y * 16 * RB; m0 < n; m0 += gridDim.y * 16 * RB) {
    // the adapters of the rows, one a lane (RB <= 4), the same in every wave
    int id = -1;
    if (lane < 16 * RB && m0 + lane < n) {
      const int q = seg0 + m0 + lane;
      if (p.pairs != nullptr) {
        id = p.ids[p.pairs[q] / p.top_k];
        if (id < 0 || id >= p.count) id = -1;
        if (wave == 0 && blockIdx.z == 0) p.rid[q] = id;
      } else {
        id = p.rid[q];
      }
    }
    uint64_t todo = p.mats > 0 ? __ballot(id >= 0) : 0;  // gate and up without adapters: the ids alone
    for (int seen = 0; todo != 0; ++seen) {
      const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
      const uint64_t mine = __ballot(id == cur);
      todo &= ~mine;
      if (seen % slots != slot) continue;
      const T* arow[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int c = min(c0 + g * 16 + (lane & 15), cols - 1);  // columns past the last repeat it, never stored
        const int m = c >= p.rank ? 1 : 0;
        arow[g] = static_cast<const T*>(p.a[m]) + ((size_t(cur) * p.L + e) * p.rank + (c - m * p.rank)) * p.K;
      }
      const T* xrow[RB];
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) xrow[rb] = x + size_t(seg0 + min(m0 + rb * 16 + (lane & 15), n - 1)) * p.K;
      f32x4_t acc[RB][NG];
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int g = 0; g < NG; ++g) acc[rb][g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      for (int k0 = wave * kSteps * kStep; k0 < p.K; k0 += kWaves * kSteps * kStep) {
        u32x4_t xv[kSteps][RB], av[kSteps][NG];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const int k = k0 + s * kStep + (lane >> 4) * E;  // K is a multiple of 8: a vector is in or out as a whole
#pragma unroll
          for (int rb = 0; rb < RB; ++rb)
            xv[s][rb] = k < p.K ? *reinterpret_cast<const u32x4_t*>(xrow[rb] + k) : u32x4_t{0, 0, 0, 0};
#pragma unroll
          for (int g = 0; g < NG; ++g)
            av[s][g] = k < p.K ? *reinterpret_cast<const u32x4_t*>(arow[g] + k) : u32x4_t{0, 0, 0, 0};
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int g = 0; g < NG; ++g) acc[rb][g] = Mma16<T>::mma(xv[s][rb], av[s][g], acc[rb][g]);
      }
      const float sc = p.scale != nullptr ? p.scale[cur] : 1.0f;
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        if (((mine >> (16 * rb)) & 0xFFFF) == 0) continue;
        __syncthreads();  // the sums before these have been read
        // lane -> column lane % 16 of the group, register i -> row 4 (lane / 16) + i
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) red[wave][4 * (lane >> 4) + i][g * 16 + (lane & 15)] = acc[rb][g][i];
        __syncthreads();
        for (int v = threadIdx.x; v < 16 * NG * 16; v += kWaves * 64) {
          const int r = v / (NG * 16), c = v % (NG * 16);
          if (!((mine >> (16 * rb + r)) & 1) || c0 + c >= cols) continue;
          float s = 0.0f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) s += red[w][r][c];
          static_cast<T*>(p.u)[size_t(seg0 + m0 + rb * 16 + r) * p.ldu + c0 + c] = Elem<T>::from_f32(sc * s);
        }
      }
    }
  }
}

template <typename T, int RB>
moe_status launch_rb(const char* name, const ShrinkP& p, int64_t max_pairs, hipStream_t s) {
  const int groups = std::max(1, (p.mats * p.rank + 15) / 16);
  // row blocks of an expert with four times its share; a larger one's blocks take more than one
  const int64_t ny = std::min<int64_t>((max_pairs + 16 * RB - 1) / (16 * RB), 4 * max_pairs / (16 * RB * p.L) + 1);
  const int slots = RB == 1 ? std::min(p.count, 4) : 1;
#define MOE_SHRINK(NG_)                                                                                          \
  MOE_LAUNCH(name, (shrink_kernel<T, RB, NG_>), dim3(unsigned(p.L), unsigned(ny), unsigned((groups + NG_ - 1) / NG_ * slots)), \
             dim3(kWaves * 64), 0, s, p, slots)
  if (groups <= 1) MOE_SHRINK(1);
  else if (groups <= 2) MOE_SHRINK(2);
  else if (groups <= 4) MOE_SHRINK(4);
  else MOE_SHRINK(8);
#undef MOE_SHRINK
  return MOE_OK;
}

// Blocks of 64 rows, which read an adapter's A a quarter as often, where they still fill the card.
template <typename T>
moe_status launch_t(const char* name, const ShrinkP& p, int64_t max_pairs, hipStream_t s) {
  return max_pairs >= 64 * 128 ? launch_rb<T, 4>(name, p, max_pairs, s) : launch_rb<T, 1>(name, p, max_pairs, s);
}

int mats_of(const moe_adapters* a, bool down) {
  return down ? (a->down_a != nullptr ? 1 : 0) : (a->gate_a != nullptr ? 1 : 0) + (a->up_a != nullptr ? 1 : 0);
}

}  // namespace

AdapterScratch carve_adapter_scratch(const moe_layer_desc* d, const moe_adapters* a, int64_t max_pairs, void* base) {
  AdapterScratch w{};
  const size_t dt = dtype_bytes(d->dtype);
  char* p = static_cast<char*>(base);
  size_t o = 0;
  auto take = [&](size_t bytes) -> void* {
    void* r = p ? p + o : nullptr;
    o += align_up(bytes, 256);
    return r;
  };
  w.rid = static_cast<int32_t*>(take(size_t(max_pairs) * 4));
  w.u_gu = take(size_t(max_pairs) * mats_of(a, false) * a->rank * dt);
  w.u_down = take(size_t(max_pairs) * mats_of(a, true) * a->rank * dt);
  w.bytes = o;
  return w;
}

Adapters gate_up_adapters(const moe_layer_desc* d, const moe_adapters* a, const AdapterScratch& w) {
  const size_t dt = dtype_bytes(d->dtype);
  const int mats = mats_of(a, false);
  char* u = static_cast<char*>(w.u_gu);
  Adapters r{};
  r.rid = w.rid;
  r.u[0] = a->gate_a != nullptr ? u : nullptr;
  r.u[1] = a->up_a != nullptr ? u + (mats - 1) * a->rank * dt : nullptr;
  r.b[0] = a->gate_b;
  r.b[1] = a->up_b;
  r.ldu = mats * a->rank;
  r.rank = a->rank;
  r.experts = d->local_count;
  return r;
}

Adapters down_adapters(const moe_layer_desc* d, const moe_adapters* a, const AdapterScratch& w) {
  Adapters r{};
  r.rid = w.rid;
  r.u[0] = a->down_a != nullptr ? w.u_down : nullptr;
  r.b[0] = a->down_b;
  r.ldu = r.rank = a->rank;
  r.experts = d->local_count;
  return r;
}

moe_status launch_adapter_shrink(const AdaptedFfnArgs& a, bool down) {
  const moe_layer_desc* d = a.f.d;
  ShrinkP p{};
  p.x = down ? a.f.h : a.f.x_sorted;
  p.offsets = a.f.offsets;
  p.pairs = down ? nullptr : a.sorted_pairs;
  p.ids = a.adapter_ids;
  p.rid = a.w.rid;
  p.scale = a.ad->scale;
  p.mats = mats_of(a.ad, down);
  p.rank = a.ad->rank;
  p.count = a.ad->count;
  p.L = d->local_count;
  p.K = down ? d->intermediate : d->hidden;
  p.top_k = d->top_k;
  p.ldu = p.mats * p.rank;
  if (down) {
    if (p.mats == 0) return MOE_OK;
    p.a[0] = a.ad->down_a;
    p.u = a.w.u_down;
  } else {
    p.a[0] = a.ad->gate_a != nullptr ? a.ad->gate_a : a.ad->up_a;
    p.a[1] = a.ad->up_a;
    p.u = a.w.u_gu;
  }
  const char* name = down ? "adapter_shrink_down" : "adapter_shrink";
  return d->dtype == MOE_BF16 ? launch_t<bf16_t>(name, p, a.f.max_pairs, a.f.s)
                              : launch_t<float>(name, p, a.f.max_pairs, a.f.s);
}

moe_status launch_adapted_ffn(const AdaptedFfnArgs& a) {
  if (a.f.max_pairs <= 0) return MOE_OK;
  const moe_status st = launch_adapter_shrink(a, false);
  if (st != MOE_OK) return st;
  return launch_adapted_products(a);
}

}  // namespace moe
