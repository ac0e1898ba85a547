// The experts' bfloat16 products with adapters for segments of tens to hundreds of rows, and for
// widths off the large tile's grid (Ultralytics glossary "Expert Parallelism", "How tokens move
// between GPUs", step 3: each GPU runs its local experts on what it received).
//
// A block of eight waves owns 128 token rows by 256 weight rows of one expert (128 gate rows and
// the same up rows for the gate/up product), each wave 64 x 64 as 2 x 2 MFMA 32x32 blocks; where those
// do not fill the card, four waves own 64 by 128.
// At these sizes a product is bound by reading the weights: at up to 128 rows an expert each weight
// is read once and every CU has a tile, where the large tile's 256 x 256 or 128 x 512 ones are too few
// or read half-empty blocks of rows.  K advances 64 at a time through a ring of three 48 KB (six 24 KB)
// stages, filled by direct global -> LDS loads two (five) steps ahead; vectors past the end of a row
// of K, rows past the segment and weight rows past N are not loaded and read as zeros, so any
// multiple of 8 is a width.
#include <algorithm>
#include <atomic>

#include "adapters.h"
#include "ffn_common.h"
#include "kernels.h"
#include "tile_adapters.h"

namespace moe {
namespace {
namespace mid {

// Tiles of kA token rows by kB weight rows; waves of 32 NA x 64.
template <int KA>
struct Shape {
  static constexpr int kA = KA, kB = 2 * KA, kWaves = KA / 16, kThreads = 64 * kWaves;
  static constexpr int NB = 2, kWaveCols = kB / 64, NA = kA / (32 * (kWaves / kWaveCols));
  static constexpr int kRowBytes = 128;                           // 64 k
  static constexpr int kStage = (kA + kB) * kRowBytes;            // 48 KB, 24 KB
  static constexpr int kLoads = kStage / 1024 / kWaves;           // 1 KB loads of a wave per stage
  static constexpr int kSlots = 144 * 1024 / kStage, kLds = kSlots * kStage;
  __device__ static int wm(int wave) { return wave / kWaveCols; }
  __device__ static int wn(int wave) { return wave % kWaveCols; }
};
constexpr int kXcds = 8;

#define MOE_VMCNT(n) __builtin_amdgcn_s_waitcnt(((n) & 0xF) | (((n) >> 4) << 14) | (0x7 << 4) | (0xF << 8))

// ---- which tile, and which part of its K, a block has.  Tiles run over (expert, column tile, row
// tile), so that the row tiles that read the same weights run together, and each XCD (every
// eighth block) takes a contiguous share of them in rounds of cpx, its CUs.  The r tiles of a round
// that does not fill them are cut along K into s pieces, as many as the round has room for; a
// piece leaves its float32 sums in the workspace and fixup_kernel adds the pieces in order.  (288
// tiles of 45 stages on 256 CUs: 1.25 instead of 2 rounds.)
constexpr int kMaxCut = 8, kMinStages = 4;  // pieces of a tile, stages of a piece
constexpr int kMaxParts = 32;               // pieces of an XCD, a round of its CUs at most

struct Plan {
  int base, F, r, s, units;
};
__device__ __forceinline__ Plan plan_of(int total, int xcd, int cpx, int nk) {
  Plan p;
  const int q = total / kXcds, rest = total % kXcds, mine = q + (xcd < rest ? 1 : 0);
  p.base = xcd * q + min(xcd, rest);
  p.F = mine / cpx;
  p.r = mine - p.F * cpx;
  p.s = p.r == 0 ? 1 : max(1, min(min(cpx / p.r, kMaxCut), nk / kMinStages));
  p.units = p.F * cpx + p.r * p.s;
  return p;
}

struct Tile {
  int expert, row0, rows, nt;  // nt: which of the product's NT column tiles
};

// The tiles of the experts, four a lane: 256 experts cost one round of loads.
template <int KA>
struct Tiles {
  const int32_t* __restrict__ offsets;
  int L, NT;
  int off[5], own, upto;  // of the lane's experts of the last scan: tiles, and tiles up to and with them

  __device__ __forceinline__ int scan(int i0) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < 5; ++j) off[j] = offsets[min(i0 + 4 * lane + j, L)];
    own = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) own += (off[j + 1] - off[j] + KA - 1) / KA * NT;
    upto = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d, 64);
      if (lane >= d) upto += v;
    }
    return __builtin_amdgcn_readlane(upto, 63);
  }
  __device__ __forceinline__ int total() {
    int n = 0;
    for (int i0 = 0; i0 < L; i0 += 256) n += scan(i0);
    return n;
  }
  // tile t < total(), after it
  __device__ __forceinline__ Tile find(int t) {
    for (int i0 = 0; i0 < L; i0 += 256) {
      if (L > 256) scan(i0);  // else the lanes hold it
      const uint64_t past = __ballot(upto > t);
      if (past != 0) {
        const int l = __builtin_ctzll(past);
        int r = t - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(own, l)), e = 0, seg0 = 0, n = 1;
        bool done = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int o0 = __builtin_amdgcn_readlane(off[j], l), o1 = __builtin_amdgcn_readlane(off[j + 1], l);
          const int tj = (o1 - o0 + KA - 1) / KA * NT;
          if (!done && r < tj) {
            done = true;
            e = i0 + 4 * l + j;
            seg0 = o0;
            n = o1 - o0;
          }
          if (!done) r -= tj;
        }
        const int mt = (n + KA - 1) / KA, m = r % mt;
        return {e, seg0 + m * KA, min(KA, n - m * KA), r / mt};
      }
      t -= __builtin_amdgcn_readlane(upto, 63);
    }
    return {0, 0, 0, 0};  // not reached
  }
};

// A piece's sums, thread-major: float4 number v of thread t at v * kThreads + t.
template <int KA>
__device__ __forceinline__ f32x4_t* part_of(float* parts, int slot) {
  return reinterpret_cast<f32x4_t*>(parts + size_t(slot) * (Shape<KA>::kA * Shape<KA>::kB));
}

template <int NMAT, int KA>
__device__ __forceinline__ void body(const bf16_t* A, const int32_t* __restrict__ offsets, const bf16_t* B0,
                                     const bf16_t* B1, bf16_t* __restrict__ C, int L, int N, int K, int cpx, float* parts,
                                     const Adapters& ad, char* lds) {
  using S = Shape<KA>;
  constexpr int kLoads = S::kLoads, kSlots = S::kSlots, kRowBytes = S::kRowBytes, kStage = S::kStage, NA = S::NA;
  static_assert(kTileAdapterLds<S, NMAT> <= S::kLds, "the adapters' LDS");
  constexpr int ON = S::kB / NMAT;  // columns of the output
  const uint32_t row_bytes = uint32_t(K) * 2u;  // a multiple of 16
  const int nk = int((row_bytes + kRowBytes - 1) / kRowBytes);
  Tiles<KA> tiles{offsets, L, (N + ON - 1) / ON};
  const int xcd = blockIdx.x % kXcds, u = blockIdx.x / kXcds;
  const Plan plan = plan_of(tiles.total(), xcd, cpx, nk);
  if (u >= plan.units) return;
  int t = u, part = 0, nparts = 1;
  if (u >= plan.F * cpx) {
    nparts = plan.s;
    t = plan.F * cpx + (u - plan.F * cpx) / nparts;
    part = (u - plan.F * cpx) % nparts;
  }
  const Tile tl = tiles.find(plan.base + t);
  const int kb = part * nk / nparts, nks = (part + 1) * nk / nparts - kb;  // the piece's stages
  const int n0 = tl.nt * ON;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = S::wm(wave), wn = S::wn(wave), fr = lane & 31, g = lane >> 5;
  constexpr uint32_t kOutside = 0xFFFFFFF0u;  // past every extent below: reads zero, without a memory access

  // ---- this lane's place in each of the wave's loads (8 rows of a stage, A's then B's; chunk c of
  // row r sits at chunk c ^ (r / 2) % 8).  Every buffer is the tile's own rows.
  const int cols = min(ON, N - n0);
  const auto rsrc_of = [&](const bf16_t* p, int rows) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<bf16_t*>(p), 0, uint32_t(rows) * row_bytes, kRsrcFlags);
  };
  const size_t boff = (size_t(tl.expert) * N + n0) * K;
  const __amdgpu_buffer_rsrc_t ra = rsrc_of(A + size_t(tl.row0) * K, tl.rows);
  const __amdgpu_buffer_rsrc_t rb0 = rsrc_of(B0 + boff, cols), rb1 = rsrc_of((NMAT == 2 ? B1 : B0) + boff, cols);
  __amdgpu_buffer_rsrc_t rsrc[kLoads];
  uint32_t at[kLoads], in_row[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int r0 = (kLoads * wave + j) * 8, r = r0 + (lane >> 3);
    const bool is_a = r0 < S::kA, second = NMAT == 2 && r0 >= S::kA + ON;
    const int mrow = is_a ? r : r - S::kA - (second ? ON : 0);
    rsrc[j] = is_a ? ra : second ? rb1 : rb0;
    at[j] = mrow < (is_a ? tl.rows : cols) ? uint32_t(mrow) * row_bytes : kOutside;
    in_row[j] = uint32_t((lane & 7) ^ ((r >> 1) & 7)) * 16u;
  }
  auto issue = [&](int s) {  // the piece's stage min(s, nks - 1) into slot s
    char* dst = lds + (s % kSlots) * kStage + kLoads * wave * 1024;
    const uint32_t k0 = uint32_t(kb + min(s, nks - 1)) * kRowBytes;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const uint32_t k = k0 + in_row[j];
      const uint32_t vo = at[j] != kOutside && k < row_bytes ? at[j] + k : kOutside;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc[j], (lds_ptr_t)(dst + j * 1024), 16, vo, 0, 0, 0);
    }
  };

  f32x16_t acc[NA][2];
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  // fragments: row fr of a 32-row block, chunk 2 kc + g
  int ao[NA], bo[2];
  const int sw = (fr >> 1) & 7;  // the blocks start at multiples of 16 rows
#pragma unroll
  for (int i = 0; i < NA; ++i) ao[i] = ((wm * NA + i) * 32 + fr) * kRowBytes;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int br = NMAT == 2 ? j * ON + wn * 32 + fr : wn * 64 + j * 32 + fr;
    bo[j] = (S::kA + br) * kRowBytes;
  }
#pragma unroll
  for (int s = 0; s < kSlots - 1; ++s) issue(s);
  for (int s = 0; s < nks; ++s) {
    MOE_VMCNT(kLoads * (kSlots - 2));    // this wave's loads of stage s have landed
    __builtin_amdgcn_s_waitcnt(0xC07F);  // and its reads of stage s - 1 (lgkmcnt)
    block_barrier();                     // as every wave's have
    issue(s + kSlots - 1);               // into the slot of stage s - 1
    const char* st = lds + (s % kSlots) * kStage;
#pragma unroll
    for (int kc = 0; kc < 4; ++kc) {
      const int co = ((2 * kc + g) ^ sw) * 16;
      bf16x8_t fa[NA], fb[2];
#pragma unroll
      for (int i = 0; i < NA; ++i) fa[i] = *reinterpret_cast<const bf16x8_t*>(st + ao[i] + co);
#pragma unroll
      for (int j = 0; j < 2; ++j) fb[j] = *reinterpret_cast<const bf16x8_t*>(st + bo[j] + co);
#pragma unroll
      for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mma32(fb[j], fa[i], acc[i][j]);
    }
  }
  MOE_VMCNT(0);  // the last (repeated) loads land before the LDS holds anything else
  if (part == 0) tile_adapters<S, NMAT, NA>(ad, tl.expert, tl.row0, tl.rows, n0, N, lds, acc);
  if (nparts > 1) {
    f32x4_t* dst = part_of<KA>(parts, xcd * kMaxParts + u - plan.F * cpx);
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          dst[((i * 2 + j) * 4 + q) * S::kThreads + tid] =
              f32x4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    return;
  }
  __builtin_amdgcn_s_waitcnt(0xC07F);
  block_barrier();  // every wave is done with the LDS

  // ---- epilogue: lane -> token row fr, register 4q + u -> column 8q + 4g + u.  The tile goes through LDS
  // as bfloat16 and out in whole pieces of 16 bytes.
  constexpr int RS = ON * 2 + 16, CPR = ON / 8;
  static_assert(S::kA * RS <= S::kLds, "the tile in the ring's LDS");
#pragma unroll
  for (int i = 0; i < NA; ++i) {
#pragma unroll
    for (int j = 0; j < 2 / NMAT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          v[u] = NMAT == 2 ? silu(acc[i][0][4 * q + u]) * acc[i][1][4 * q + u] : acc[i][j][4 * q + u];
        const int cl = wn * (32 * (2 / NMAT)) + j * 32 + 8 * q + 4 * g;
        *reinterpret_cast<uint2*>(lds + ((wm * NA + i) * 32 + fr) * RS + cl * 2) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      }
  }
  __builtin_amdgcn_s_waitcnt(0xC07F);
  block_barrier();
#pragma unroll
  for (int p = 0; p < S::kA * CPR / S::kThreads; ++p) {
    const int id = tid + S::kThreads * p, r = id / CPR, c = id % CPR;
    // N is a multiple of 8: a piece is wholly inside or wholly past column N
    if (r < tl.rows && n0 + c * 8 < N)
      *reinterpret_cast<u32x4_t*>(C + size_t(tl.row0 + r) * N + n0 + c * 8) =
          *reinterpret_cast<const u32x4_t*>(lds + r * RS + c * 16);
  }
}
#undef MOE_VMCNT

template <int NMAT, int KA>
__global__ __launch_bounds__(Shape<KA>::kThreads) void gemm_kernel(const bf16_t* A, const int32_t* offsets,
                                                                   const bf16_t* B0, const bf16_t* B1, bf16_t* C, int L,
                                                                   int N, int K, int cpx, float* parts, Adapters ad) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  body<NMAT, KA>(A, offsets, B0, B1, C, L, N, K, cpx, parts, ad, lds);
}

// Adds the pieces of the cut tiles in order and writes the tiles.  A block takes one row block's
// and, in the plain product, one column block's float4s of a thread: kFixBlocks blocks a tile.
template <int NMAT, int KA>
constexpr int kFixBlocks = Shape<KA>::NA * 2 / NMAT;

template <int NMAT, int KA>
__global__ __launch_bounds__(Shape<KA>::kThreads) void fixup_kernel(const int32_t* offsets, bf16_t* __restrict__ C, int L,
                                                                    int N, int K, int cpx, const float* parts) {
  using S = Shape<KA>;
  constexpr int ON = S::kB / NMAT;
  const int sub = blockIdx.x % kFixBlocks<NMAT, KA>, cut = blockIdx.x / kFixBlocks<NMAT, KA>;
  const int xcd = cut % kXcds, w = cut / kXcds;
  Tiles<KA> tiles{offsets, L, (N + ON - 1) / ON};
  const Plan plan = plan_of(tiles.total(), xcd, cpx, (K * 2 + S::kRowBytes - 1) / S::kRowBytes);
  if (w >= plan.r || plan.s == 1) return;
  const Tile tl = tiles.find(plan.base + plan.F * cpx + w);
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, fr = lane & 31, g = lane >> 5;
  const int i = sub / (2 / NMAT), j = NMAT == 2 ? 0 : sub % 2;
  const size_t stride = size_t(S::kA) * S::kB / 4;  // float4s a piece
  const f32x4_t* src = part_of<KA>(const_cast<float*>(parts), xcd * kMaxParts + w * plan.s) + (i * 2 + j) * 4 * S::kThreads + tid;
  f32x4_t a[4], b[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    a[q] = src[q * S::kThreads];
    b[q] = NMAT == 2 ? src[(4 + q) * S::kThreads] : a[q];
  }
  for (int p = 1; p < plan.s; ++p)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      a[q] += src[size_t(p) * stride + q * S::kThreads];
      if (NMAT == 2) b[q] += src[size_t(p) * stride + (4 + q) * S::kThreads];
    }
  const int r = (S::wm(wave) * S::NA + i) * 32 + fr;
  if (r >= tl.rows) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int col = tl.nt * ON + S::wn(wave) * (32 * (2 / NMAT)) + j * 32 + 8 * q + 4 * g;
    float v[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = NMAT == 2 ? silu(a[q][x]) * b[q][x] : a[q][x];
    if (col < N)  // N is a multiple of 8
      *reinterpret_cast<uint2*>(C + size_t(tl.row0 + r) * N + col) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
}

// CUs of an XCD, on the current device (32 where they cannot be asked for).
int cus_per_xcd() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 32;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < kXcds) n = 256;
    n = std::min(n / kXcds, kMaxParts);
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Tiles that max_pairs rows of L experts can have: row tiles at most one an expert more than full ones.
template <int KA, int NMAT>
int64_t most_tiles(int64_t max_pairs, int L, int N) {
  constexpr int ON = 2 * KA / NMAT;
  return ((max_pairs + KA - 1) / KA + L) * ((N + ON - 1) / ON);
}

template <int NMAT, int KA>
moe_status launch(const char* name, const char* fix_name, const void* A, const int32_t* offsets, const void* B0,
                  const void* B1, void* C, int L, int N, int K, int64_t max_pairs, float* parts, hipStream_t s,
                  const Adapters& ad) {
  using S = Shape<KA>;
  auto kern = gemm_kernel<NMAT, KA>;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
  if (e != hipSuccess) return set_error(MOE_ERR_HIP, "%s: LDS attribute: %s", name, hipGetErrorString(e));
  const int cpx = cus_per_xcd();
  // an XCD's share of the tiles is rounded up; pieces add less than a round
  const int64_t share = (most_tiles<KA, NMAT>(max_pairs, L, N) + kXcds - 1) / kXcds;
  const int64_t units = share + cpx;
  MOE_LAUNCH(name, kern, dim3(unsigned(units * kXcds)), dim3(S::kThreads), S::kLds, s, static_cast<const bf16_t*>(A), offsets,
             static_cast<const bf16_t*>(B0), static_cast<const bf16_t*>(B1), static_cast<bf16_t*>(C), L, N, K, cpx, parts, ad);
  const int nk = int((int64_t(K) * 2 + S::kRowBytes - 1) / S::kRowBytes);
  if (nk < 2 * kMinStages) return MOE_OK;  // nothing is cut
  const int64_t cuts = std::min<int64_t>(share, cpx / 2);  // a round of more than half the CUs is not cut
  MOE_LAUNCH(fix_name, (fixup_kernel<NMAT, KA>), dim3(unsigned(cuts * kXcds * kFixBlocks<NMAT, KA>)), dim3(S::kThreads), 0, s,
             offsets, static_cast<bf16_t*>(C), L, N, K, cpx, static_cast<const float*>(parts));
  return MOE_OK;
}

// 64 x 128 tiles while they take a round of the card (half of the experts' last row tiles counted).
// Small against large, rank 16, us: 33 rows on each of 8 experts of 1000 x 2008, 60 instead of 74, and on
// 16 of 1024 x 1024 56 instead of 71; 127 there, 96 instead of 73; 127 on one of 4096 x 2048 57 instead of
// 70, 600 there 104 instead of 84.
template <int NMAT>
bool small_tiles(int64_t max_pairs, int L, int N) {
  constexpr int ON = 128 / NMAT;
  return (max_pairs / 64 + (L + 1) / 2) * ((N + ON - 1) / ON) <= 300;
}

template <int NMAT>
moe_status launch(const char* name, const char* fix_name, const void* A, const int32_t* offsets, const void* B0,
                  const void* B1, void* C, int L, int N, int K, int64_t max_pairs, float* parts, hipStream_t s,
                  const Adapters& ad) {
  return small_tiles<NMAT>(max_pairs, L, N)
             ? launch<NMAT, 64>(name, fix_name, A, offsets, B0, B1, C, L, N, K, max_pairs, parts, s, ad)
             : launch<NMAT, 128>(name, fix_name, A, offsets, B0, B1, C, L, N, K, max_pairs, parts, s, ad);
}

}  // namespace mid
}  // namespace

size_t mid_adapted_scratch_bytes() {
  return size_t(mid::kXcds) * mid::kMaxParts * mid::Shape<128>::kA * mid::Shape<128>::kB * sizeof(float);
}

bool mid_adapted_fits(const moe_layer_desc* d, int64_t max_pairs) {
  const int64_t tiles = mid::most_tiles<64, 2>(max_pairs, d->local_count, std::max(d->hidden, d->intermediate));
  // fewer than 2^32 threads, whichever tiles they are
  return d->dtype == MOE_BF16 && d->weight_layout == MOE_WEIGHTS_OUT_IN && tiles < (int64_t(1) << 24) - 1024;
}

moe_status launch_mid_adapted(const AdaptedFfnArgs& a) {
  const FfnArgs& f = a.f;
  const moe_layer_desc* d = f.d;
  const int L = d->local_count, H = d->hidden, I = d->intermediate;
  float* parts = static_cast<float*>(f.scratch);
  moe_status st = mid::launch<2>("ffn_gate_up", "ffn_gate_up_fixup", f.x_sorted, f.offsets, f.w_gate, f.w_up, f.h, L, I, H,
                                 f.max_pairs, parts, f.s, gate_up_adapters(d, a.ad, a.w));
  if (st != MOE_OK) return st;
  st = launch_adapter_shrink(a, true);
  if (st != MOE_OK) return st;
  return mid::launch<1>("ffn_down", "ffn_down_fixup", f.h, f.offsets, f.w_down, f.w_down, f.y_sorted, L, H, I,
                        f.max_pairs, parts, f.s, down_adapters(d, a.ad, a.w));
}

}  // namespace moe
