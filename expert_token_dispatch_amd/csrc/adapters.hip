// Low-rank adapters of many requests beside the experts' projections, the first product:
//   u[q, r] = s_a * sum_k x[q, k] A[a, e, r, k]
// for sorted row q of expert e whose token has adapter a.  The second product, u B^T, is added
// by the epilogues of the experts' own products.
//
// A block takes 16 RB rows of one expert and finds the adapters among them (ids come in any
// order; tokens of one request follow each other in a prompt and are strangers in a decode
// batch).  For one adapter after another it multiplies the rows that have it by its A; the rows
// that have not are not loaded.  A non-finite value in one request's adapter reaches no other
// request, and a row's sums do not depend on its neighbours.
//
// What bounds it: in a decode batch reading each adapter's A once, in a prompt reading x (h for
// the down product) once more than the experts' own products do.  Both operands come by direct
// global -> LDS loads, whole lines of a row at a time, into a ring of stages: fragments loaded
// straight from memory have a lane per row, sixteen lines a quarter wave, and kept the
// texture unit four times as long (16384 pairs, rank 64, 4096 x 14336 experts: 180 and 380 us).
// The waves split a stage's k (and the rows), and their sums meet in LDS in a fixed order.
#include <math.h>

#include <algorithm>

#include "adapters.h"
#include "ffn_common.h"
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
  void* u;                  // [P_max, ldu]: matrix m's columns start at m * rank, their low parts lo behind
  int ldu, lo, rank, count, mats, L, K, top_k;
};

constexpr int kWaves = 4;

#define MOE_VMCNT(n) __builtin_amdgcn_s_waitcnt(((n) & 0xF) | (((n) >> 4) << 14) | (0x7 << 4) | (0xF << 8))

// Stages of RB row blocks of x and NG column groups (16 rows of A each), WK x 64 bytes of k a row:
// one MFMA step for each of the WK waves along k, the others split the rows.
template <int RB, int NG>
struct Ring {
  static constexpr int WK = RB == 1 ? 4 : 2, WM = kWaves / WK, MB = RB / WM;  // MB: row blocks of a wave
  static constexpr int kRowBytes = WK * 64, kRows = 16 * (RB + NG), kPerLoad = 1024 / kRowBytes;  // rows of a 1 KB load
  static constexpr int kLoads = (kRows / kPerLoad + kWaves - 1) / kWaves;                         // a wave's, per stage
  static constexpr int kStage = kLoads * kWaves * 1024;
  static constexpr int kSums = WK * 16 * RB * 16 * NG * 4;
  static constexpr int kSlots = kStage <= 8 * 1024 ? 8 : kStage <= 12 * 1024 ? 6 : kStage <= 20 * 1024 ? 4 : 3;
  static constexpr int kLds = kSlots * kStage > kSums ? kSlots * kStage : kSums;
};

// The expert of row block g and the block's first row within it; expert -1 past the last.  The
// lanes hold four experts each, so 256 experts cost one round of loads.
struct RowBlock {
  int expert, m0;
};
__device__ __forceinline__ RowBlock find_rows(const int32_t* __restrict__ offsets, int L, int rows, int g) {
  const int lane = threadIdx.x & 63;
  for (int i0 = 0; i0 < L; i0 += 256) {
    int off[5], t[4];
#pragma unroll
    for (int j = 0; j < 5; ++j) off[j] = offsets[min(i0 + 4 * lane + j, L)];
    int own = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) own += t[j] = (off[j + 1] - off[j] + rows - 1) / rows;  // past L: no rows
    int upto = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d, 64);
      if (lane >= d) upto += v;
    }
    const uint64_t past = __ballot(upto > g);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      int r = g - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(own, l)), e = i0 + 4 * l;
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const int tj = __builtin_amdgcn_readlane(t[j], l);
        if (e == i0 + 4 * l + j && r >= tj) {
          r -= tj;
          ++e;
        }
      }
      return {e, r * rows};
    }
    g -= __builtin_amdgcn_readlane(upto, 63);
  }
  return {-1, 0};
}

// NG groups of 16 of the mats * rank columns a block (blockIdx.z / slots); of its rows' adapters it
// takes every slots-th (blockIdx.z % slots).
template <typename T, int RB, int NG>
__device__ __forceinline__ void shrink_body(const ShrinkP& p, int slots, char* lds) {
  using S = Ring<RB, NG>;
  // in a prompt an XCD's blocks (every eighth) are neighbours, whose adapters are often the same
  const int per_xcd = (gridDim.x + 7) / 8, b = blockIdx.x;
  const RowBlock at_rows = find_rows(p.offsets, p.L, 16 * RB, RB > 1 ? b % 8 * per_xcd + b / 8 : b);
  const int e = at_rows.expert, m0 = at_rows.m0;
  if (e < 0) return;
  const int seg0 = p.offsets[e], n = p.offsets[e + 1] - seg0;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wk = wave % S::WK, wm = wave / S::WK;
  const int slot = blockIdx.z % slots, c0 = (blockIdx.z / slots) * NG * 16, cols = p.mats * p.rank;
  const uint32_t row_bytes = uint32_t(p.K) * sizeof(T);  // a multiple of 16
  const int nk = int((row_bytes + S::kRowBytes - 1) / S::kRowBytes);
  constexpr uint32_t kOutside = 0xFFFFFFF0u;  // past every extent below: reads zero, without a memory access
  constexpr int CPR = S::kRowBytes / 16;      // 16-byte chunks of a stage's row
  // chunk c of row r sits at chunk c ^ swizzle(r): 16 rows' reads of one chunk fall in different banks
  auto swizzle = [](int r) { return CPR == 8 ? (r >> 1) & 7 : r & 15; };
  // the adapters of the rows, one a lane (RB <= 2), the same in every wave
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
  const __amdgpu_buffer_rsrc_t x_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<T*>(static_cast<const T*>(p.x) + size_t(seg0 + m0) * p.K), 0, uint32_t(16 * RB) * row_bytes, kRsrcFlags);
  for (int seen = 0; todo != 0; ++seen) {
    const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    const uint64_t mine = __ballot(id == cur);
    todo &= ~mine;
    if (seen % slots != slot) continue;
    // this lane's place in each of the wave's loads: row of the stage (x, then A), chunk, byte offset
    __amdgpu_buffer_rsrc_t rsrc[S::kLoads];
    uint32_t at[S::kLoads], in_row[S::kLoads];
#pragma unroll
    for (int j = 0; j < S::kLoads; ++j) {
      const int b = S::kLoads * wave + j, r0 = b * S::kPerLoad, r = r0 + lane / CPR;
      in_row[j] = uint32_t((lane % CPR) ^ swizzle(r)) * 16u;
      if (r0 < 16 * RB) {
        rsrc[j] = x_rsrc;
        at[j] = (mine >> r) & 1 ? uint32_t(r) * row_bytes : kOutside;
      } else {
        const int col0 = c0 + r0 - 16 * RB, c = col0 + lane / CPR;  // the rank is a multiple of 8: one matrix a load
        const int m = col0 >= p.rank ? 1 : 0;
        rsrc[j] = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<T*>(static_cast<const T*>(p.a[m]) + (size_t(cur) * p.L + e) * p.rank * p.K), 0,
            uint32_t(p.rank) * row_bytes, kRsrcFlags);
        at[j] = c < cols && r < S::kRows ? uint32_t(c - m * p.rank) * row_bytes : kOutside;
      }
    }
    auto issue = [&](int s) {  // stage min(s, nk - 1) into slot s
      char* dst = lds + (s % S::kSlots) * S::kStage + S::kLoads * wave * 1024;
      const uint32_t k0 = uint32_t(min(s, nk - 1)) * S::kRowBytes;
#pragma unroll
      for (int j = 0; j < S::kLoads; ++j) {
        const uint32_t k = k0 + in_row[j];
        const uint32_t vo = at[j] != kOutside && k < row_bytes ? at[j] + k : kOutside;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc[j], (lds_ptr_t)(dst + j * 1024), 16, vo, 0, 0, 0);
      }
    };
    f32x4_t acc[S::MB][NG];
#pragma unroll
    for (int rb = 0; rb < S::MB; ++rb)
#pragma unroll
      for (int g = 0; g < NG; ++g) acc[rb][g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // fragments: row lane % 16 of a block, chunk 4 wk + lane / 16
    const int chunk = 4 * wk + (lane >> 4);
    int xo[S::MB], ao[NG];
#pragma unroll
    for (int rb = 0; rb < S::MB; ++rb) {
      const int r = (wm * S::MB + rb) * 16 + (lane & 15);
      xo[rb] = r * S::kRowBytes + (chunk ^ swizzle(r)) * 16;
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int r = 16 * RB + g * 16 + (lane & 15);
      ao[g] = r * S::kRowBytes + (chunk ^ swizzle(r)) * 16;
    }
    __syncthreads();  // the sums of the adapter before have been read
#pragma unroll
    for (int s = 0; s < S::kSlots - 1; ++s) issue(s);
    for (int s = 0; s < nk; ++s) {
      MOE_VMCNT(S::kLoads * (S::kSlots - 2));   // this wave's loads of stage s have landed
      __builtin_amdgcn_s_waitcnt(0xC07F);       // and its reads of stage s - 1 (lgkmcnt)
      block_barrier();                          // as every wave's have
      issue(s + S::kSlots - 1);                 // into the slot of stage s - 1
      const char* st = lds + (s % S::kSlots) * S::kStage;
      u32x4_t xv[S::MB], av[NG];
#pragma unroll
      for (int rb = 0; rb < S::MB; ++rb) xv[rb] = *reinterpret_cast<const u32x4_t*>(st + xo[rb]);
#pragma unroll
      for (int g = 0; g < NG; ++g) av[g] = *reinterpret_cast<const u32x4_t*>(st + ao[g]);
#pragma unroll
      for (int rb = 0; rb < S::MB; ++rb)
#pragma unroll
        for (int g = 0; g < NG; ++g) acc[rb][g] = Mma16<T>::mma(xv[rb], av[g], acc[rb][g]);
    }
    MOE_VMCNT(0);     // the last (repeated) loads land before the sums take their place
    __syncthreads();  // in every wave
    // lane -> column lane % 16 of the group, register i -> row 4 (lane / 16) + i
    float* red = reinterpret_cast<float*>(lds);  // [WK][16 RB][16 NG]
#pragma unroll
    for (int rb = 0; rb < S::MB; ++rb)
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          red[((wk * RB + wm * S::MB + rb) * 16 + 4 * (lane >> 4) + i) * (NG * 16) + g * 16 + (lane & 15)] = acc[rb][g][i];
    __syncthreads();
    const float sc = p.scale != nullptr ? p.scale[cur] : 1.0f;
    for (int v = threadIdx.x; v < 16 * RB * 16 * NG; v += kWaves * 64) {
      const int r = v / (NG * 16), c = v % (NG * 16);
      if (!((mine >> r) & 1) || c0 + c >= cols) continue;
      float a = red[v];
#pragma unroll
      for (int w = 1; w < S::WK; ++w) a += red[v + w * (16 * RB * 16 * NG)];
      T* u = static_cast<T*>(p.u) + size_t(seg0 + m0 + r) * p.ldu + c0 + c;
      const T hi = Elem<T>::from_f32(sc * a);
      u[0] = hi;
      if constexpr (sizeof(T) == 2) {
        // what hi leaves; nothing behind an infinity, which an inf - inf would make NaN
        const float left = sc * a - Elem<T>::to_f32(hi);
        u[p.lo] = Elem<T>::from_f32(fabsf(left) < INFINITY ? left : 0.0f);
      }
    }
  }
}
#undef MOE_VMCNT

template <typename T, int RB, int NG>
__global__ __launch_bounds__(kWaves * 64) void shrink_kernel(ShrinkP p, int slots) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  shrink_body<T, RB, NG>(p, slots, lds);
}

template <typename T, int RB, int NG>
moe_status launch_ng(const char* name, const ShrinkP& p, const dim3& grid, int slots, hipStream_t s) {
  auto kern = shrink_kernel<T, RB, NG>;
  constexpr int lds = Ring<RB, NG>::kLds;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return set_error(MOE_ERR_HIP, "%s: LDS attribute: %s", name, hipGetErrorString(e));
  MOE_LAUNCH(name, kern, grid, dim3(kWaves * 64), lds, s, p, slots);
  return MOE_OK;
}

template <typename T, int RB>
moe_status launch_rb(const char* name, const ShrinkP& p, int64_t max_pairs, int groups, hipStream_t s) {
  const int64_t blocks = (max_pairs + 16 * RB - 1) / (16 * RB) + p.L;  // at most; a multiple of 8 for the XCDs
  // four blocks share the adapters of their rows, which are many in a decode batch (16384 mixed rows of
  // 60 adapters, rank 16, gate and up of 4096 x 14336 experts: 601 -> 428 us; eight 410, but one of 512 rows
  // 19 -> 20), and run side by side in a prompt (one: 114 and 244 us of the case below)
  const int slots = std::min(p.count, 4);
  const auto grid = [&](int ng) {
    return dim3(unsigned((blocks + 7) / 8 * 8), 1, unsigned((groups + ng - 1) / ng * slots));
  };
  // a few rows: their columns over more blocks
  if constexpr (RB == 1)
    if (groups <= 1 || max_pairs <= 64) return launch_ng<T, RB, 1>(name, p, grid(1), slots, s);
  if (groups <= 2) return launch_ng<T, RB, 2>(name, p, grid(2), slots, s);
  if (groups <= 4) return launch_ng<T, RB, 4>(name, p, grid(4), slots, s);
  return launch_ng<T, RB, 8>(name, p, grid(8), slots, s);
}

// Blocks of 32 rows, which read an adapter's A half as often, where they fill the card twice (16384
// pairs in 8 requests, rank 64, 4096 x 14336 experts: 100 and 195 us; 16 rows 167 and 229) and an
// adapter has more than 16 columns (with those alone, mixed rows of 60 adapters 1075 us, 16 rows 922).
template <typename T>
moe_status launch_t(const char* name, const ShrinkP& p, int64_t max_pairs, hipStream_t s) {
  const int groups = std::max(1, (p.mats * p.rank + 15) / 16);
  return groups > 1 && max_pairs >= 32 * 256 ? launch_rb<T, 2>(name, p, max_pairs, groups, s)
                                             : launch_rb<T, 1>(name, p, max_pairs, groups, s);
}

int mats_of(const moe_adapters* a, bool down) {
  return down ? (a->down_a != nullptr ? 1 : 0) : (a->gate_a != nullptr ? 1 : 0) + (a->up_a != nullptr ? 1 : 0);
}

}  // namespace

AdapterScratch carve_adapter_scratch(const moe_layer_desc* d, const moe_adapters* a, int64_t max_pairs, void* base) {
  AdapterScratch w{};
  char* p = static_cast<char*>(base);
  size_t o = 0;
  auto take = [&](size_t bytes) -> void* {
    void* r = p ? p + o : nullptr;
    o += align_up(bytes, 256);
    return r;
  };
  w.rid = static_cast<int32_t*>(take(size_t(max_pairs) * 4));
  w.u_gu = take(size_t(max_pairs) * mats_of(a, false) * a->rank * 4);  // float32, or two bfloat16
  w.u_down = take(size_t(max_pairs) * mats_of(a, true) * a->rank * 4);
  w.ffn = take(adapted_ffn_scratch_bytes(d, max_pairs));
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
  r.lo = d->dtype == MOE_BF16 ? mats * a->rank : 0;
  r.ldu = mats * a->rank + r.lo;
  r.rank = a->rank;
  r.experts = d->local_count;
  return r;
}

Adapters down_adapters(const moe_layer_desc* d, const moe_adapters* a, const AdapterScratch& w) {
  Adapters r{};
  r.rid = w.rid;
  r.u[0] = a->down_a != nullptr ? w.u_down : nullptr;
  r.b[0] = a->down_b;
  r.rank = a->rank;
  r.lo = d->dtype == MOE_BF16 ? a->rank : 0;
  r.ldu = a->rank + r.lo;
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
  p.lo = d->dtype == MOE_BF16 ? p.mats * p.rank : 0;
  p.ldu = p.mats * p.rank + p.lo;
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
