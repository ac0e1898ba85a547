// Stage 3, the skinny grouped-GEMM kernel for decode-sized batches (a few token
// rows per expert): Ultralytics glossary "Expert Parallelism", "How tokens move
// between GPUs", step 3 (each GPU runs its local experts on what it received).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "adapters.h"
#include "ffn_common.h"
#include "kernels.h"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// Skinny kernel for segments of a few rows (decode-sized batches).
//
// With a handful of rows per expert the product is bound by streaming the
// expert weights from HBM, so the work is split over weight rows: one block
// of four waves owns one expert and 64 consecutive output columns (each wave
// 16 weight rows, or 16 gate + 16 up rows).  A wave multiplies up to 64 of the
// expert's token rows at a time (four MFMA 16x16x32 row blocks) and streams
// its weight rows straight from HBM into registers, eight k-steps of 32 in
// flight per matrix (16-byte loads; two consecutive steps cover a 128-byte
// line of each weight row).  The token rows come through the caches.  An
// expert that received no rows returns before touching its weights.
namespace skinny {

constexpr int kThreads = 256, kMaxRowBlocks = 4;
// k of one step: 64 bytes of a row
template <typename T>
constexpr int kStep = 64 / int(sizeof(T));

bool supported(int K) { return K % 32 == 0; }

// KS = 4, for a few rows with adapters whose active experts do not fill the card: the waves share
// their columns and split K, so a block covers a quarter of the columns and there are four times
// as many; their sums meet in LDS in wave order, and wave w finishes row block w.
//
// Each wave streams two sets of 16 weight rows: for gate/up the gate and the
// up rows of the same 16 output columns, for down two adjacent groups of 16
// output columns.  So a block (four waves) covers 64 gate/up columns or 128
// down columns.  The k loop is double-buffered in registers: the loads of the
// next four 32-k steps are in flight while the MFMAs of the current four run.
template <int NMAT>
constexpr int cols_per_block() { return NMAT == 2 ? 64 : 128; }

// Adds the adapters' share to the sums of one row block (16 rows from row0, n of them there, id: the
// adapter of row lane % 16) and the wave's two streams of 16 columns; layout of the sums: lane ->
// column lane & 15, register i -> row 4 (lane / 16) + i.  A decode batch's rows have adapters of
// their own, so four adapters are in flight together; each one's products take all the rows and
// are added to its own.
template <typename T, int NMAT>
__device__ __forceinline__ void add_adapters(const Adapters& ad, int expert, int row0, int n, int id, int col0, int N,
                                             f32x4_t& acc0, f32x4_t& acc1) {
  constexpr int kFlight = 4, E = Elem<T>::kPerVec;
  const int lane = threadIdx.x & 63, r16 = lane & 15, kg = (lane >> 4) * E;
  uint32_t todo = uint32_t(__ballot(id >= 0)) & 0xFFFF;
  const int row = row0 + min(r16, n - 1);
  const int col[2] = {min(col0 + r16, N - 1), min(NMAT == 2 ? col0 + r16 : col0 + 16 + r16, N - 1)};
  while (todo != 0) {
    uint32_t mine[kFlight];
    const T* b[kFlight][2];
    f32x4_t t[kFlight][2];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      // past the last adapter its products are repeated, for no row
      const int cur = todo != 0 || f == 0 ? __builtin_amdgcn_readlane(id, __builtin_ctz(todo)) : -1;
      mine[f] = cur >= 0 ? uint32_t(__ballot(id == cur)) & 0xFFFF : 0;
      todo &= ~mine[f];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int m = NMAT == 2 ? s : 0;
        b[f][s] = cur >= 0 && ad.u[m] != nullptr ? adapter_b<T>(ad, m, cur, expert, col[s], N) : f > 0 ? b[0][s] : nullptr;
        t[f][s] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
    }
    for (int c0 = 0; c0 < ad.rank; c0 += kStep<T>) {
      const int c = c0 + kg;
      const u32x4_t zero = {0, 0, 0, 0};
      u32x4_t uf[NMAT], ul[NMAT], bf[kFlight][2];
#pragma unroll
      for (int m = 0; m < NMAT; ++m) {
        const bool in = c < ad.rank && ad.u[m] != nullptr;  // a vector at a time, as the rank is
        const T* u = adapter_u<T>(ad, m, row);
        uf[m] = in ? *reinterpret_cast<const u32x4_t*>(u + c) : zero;
        ul[m] = zero;
        if constexpr (sizeof(T) == 2) ul[m] = in ? *reinterpret_cast<const u32x4_t*>(u + ad.lo + c) : zero;
#pragma unroll
        for (int f = 0; f < kFlight; ++f)
#pragma unroll
          for (int s = 0; s < 2; ++s)
            if (NMAT == 1 || s == m) bf[f][s] = in ? *reinterpret_cast<const u32x4_t*>(b[f][s] + c) : zero;
      }
#pragma unroll
      for (int f = 0; f < kFlight; ++f)
#pragma unroll
        for (int s = 0; s < 2; ++s) t[f][s] = Mma16<T>::mma(uf[NMAT == 2 ? s : 0], bf[f][s], t[f][s]);
      if constexpr (sizeof(T) == 2) {
        u16x2_t most = {0, 0};
#pragma unroll
        for (int f = 0; f < kFlight; ++f)
#pragma unroll
          for (int s = 0; s < 2; ++s) most = largest_exponents(most, bf[f][s]);
        if (!all_finite(most))
#pragma unroll
          for (int f = 0; f < kFlight; ++f)
#pragma unroll
            for (int s = 0; s < 2; ++s) bf[f][s] = finite_ones(bf[f][s]);
#pragma unroll
        for (int f = 0; f < kFlight; ++f)
#pragma unroll
          for (int s = 0; s < 2; ++s) t[f][s] = Mma16<T>::mma(ul[NMAT == 2 ? s : 0], bf[f][s], t[f][s]);
      }
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool own = (mine[f] >> (4 * (lane >> 4) + i)) & 1;
        acc0[i] = own ? acc0[i] + t[f][0][i] : acc0[i];
        acc1[i] = own ? acc1[i] + t[f][1][i] : acc1[i];
      }
  }
}

// SAVE (gate/up of the training forward): the gate and up pre-activations go to Gs, Us too.
// BKN: the weights are k-major (element (k, n) at B[k * N + n]): each lane then loads
// 16 bytes of one k row (a 32 x 16 block of a stream per step is 32 rows of 32 bytes),
// the wave parks the block in its own 1 KB of LDS and reads the fragments back with
// transposing reads, so the MFMAs see the same operands as with n-major weights.
// AD: Adapters, whose share is added to the sums, or NoAdapters.
template <typename T, int NMAT, bool SAVE, bool BKN, class AD, int KS>
__global__ __launch_bounds__(kThreads) void gemm_kernel(const T* __restrict__ A, const int32_t* __restrict__ offsets,
                                                        const T* __restrict__ B0, const T* __restrict__ B1,
                                                        T* __restrict__ C, int N, int K, T* __restrict__ Gs,
                                                        T* __restrict__ Us, AD ad) {
  constexpr int kWaveCols = NMAT == 2 ? 16 : 32;
  constexpr int kPipe = 4, KK = kStep<T>, E = Elem<T>::kPerVec;
  static_assert(!BKN || sizeof(T) == 2, "the transposing reads move 16-bit elements");
  int expert = blockIdx.y;
  if constexpr (std::is_same<AD, Adapters>::value) {
    expert = expert_with_rows(offsets, ad.experts, blockIdx.y);
    if (expert < 0) return;
  }
  const int seg0 = offsets[expert];
  const int seg_n = offsets[expert + 1] - seg0;
  if (seg_n <= 0) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  // first output column of this wave; with KS > 1 the block's waves have the same
  const int col0 = KS > 1 ? int(blockIdx.x) * kWaveCols : int(blockIdx.x) * cols_per_block<NMAT>() + wave * kWaveCols;
  if (col0 >= N) return;
  const int kb = KS > 1 ? KK * ((K / KK) * wave / KS) : 0;              // this wave's k
  const int ke = KS > 1 ? KK * ((K / KK) * (wave + 1) / KS) : KK * (K / KK);
  const size_t boff = size_t(expert) * N * K;
  const int kg = (lane >> 4) * E;  // the lane's k values within a step (8 in bf16)
  const T* bs0;
  const T* bs1;
  size_t kstride;  // elements between consecutive k of a lane's stream
  if constexpr (!BKN) {
    // stream 0 / 1 weight row of this lane (rows past N repeat row N-1; never stored)
    const int wrow0 = min(col0 + (lane & 15), N - 1);
    const int wrow1 = NMAT == 2 ? wrow0 : min(col0 + 16 + (lane & 15), N - 1);
    bs0 = B0 + boff + size_t(wrow0) * K + kg;
    bs1 = (NMAT == 2 ? B1 : B0) + boff + size_t(wrow1) * K + kg;
    kstride = 1;
  } else {
    // lane l loads k row l/2 of the step, columns c + 8 (l % 2) .. +7 of its stream's 16
    // (chunks past N re-read the last chunk of the row; never stored)
    const int c0 = min(col0 + 8 * (lane & 1), N - 8);
    const int c1 = NMAT == 2 ? c0 : min(col0 + 16 + 8 * (lane & 1), N - 8);
    bs0 = B0 + boff + size_t(lane >> 1) * N + c0;
    bs1 = (NMAT == 2 ? B1 : B0) + boff + size_t(lane >> 1) * N + c1;
    kstride = size_t(N);
  }
  // the wave's LDS blocks (k-major weights only): [stream][step] 1 KB each; row r of a
  // block at 32-byte slot r ^ 4 (r / 8 % 2), so a transposing read's two row quads per
  // half wave fall in different bank halves
  __shared__ __attribute__((aligned(1024))) char park[BKN ? 4 * 2 * kPipe * 1024 : 16];
  char* wpark = park + (BKN ? wave * 2 * kPipe * 1024 : 0);
  auto slot = [](int r) { return (r ^ (((r >> 3) & 1) << 2)) * 32; };
  const int woff = slot(lane >> 1) + 16 * (lane & 1);  // this lane's store
  // its transposing reads: k rows 8 (lane / 16) + (lane % 16) / 4 and four rows down
  const int roff0 = slot(8 * (lane >> 4) + ((lane & 15) >> 2)) + 8 * (lane & 3);
  const int roff1 = slot(8 * (lane >> 4) + ((lane & 15) >> 2) + 4) + 8 * (lane & 3);

  for (int m0 = 0; m0 < seg_n; m0 += 16 * kMaxRowBlocks) {
    const int nrb = min(kMaxRowBlocks, (seg_n - m0 + 15) / 16);
    // token row of each row block for this lane (rows past the segment repeat its last row)
    const T* arow[kMaxRowBlocks];
#pragma unroll
    for (int rb = 0; rb < kMaxRowBlocks; ++rb)
      arow[rb] = A + size_t(seg0 + min(m0 + rb * 16 + (lane & 15), seg_n - 1)) * K + kg;
    // the adapters of the rows that this wave finishes, asked for before the products
    int ids[KS > 1 ? 1 : kMaxRowBlocks] = {};
    if constexpr (std::is_same<AD, Adapters>::value) {
#pragma unroll
      for (int rb = 0; rb < (KS > 1 ? 1 : kMaxRowBlocks); ++rb) {
        const int r = m0 + (KS > 1 ? wave : rb) * 16 + (lane & 15);
        ids[rb] = r < seg_n ? ad.rid[seg0 + r] : -1;
      }
    }
    f32x4_t acc[2][kMaxRowBlocks];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int rb = 0; rb < kMaxRowBlocks; ++rb) acc[m][rb] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // two register sets of kPipe k steps: the loads of the next set are in flight
    // while the MFMAs of the current one run (four steps per set: fewer waves
    // fit, but each keeps more in flight; same-box A/B on the decode-sized
    // layer: 0 to -4% per layer against two steps, while capping registers for
    // more waves per SIMD made it 12% slower)
    u32x4_t w0[2][kPipe], w1[2][kPipe], a0[2][kPipe];
    const int nset = (ke - kb) / (KK * kPipe);
    auto load_set = [&](int b, int k0) {
#pragma unroll
      for (int u = 0; u < kPipe; ++u) {
        w0[b][u] = *reinterpret_cast<const u32x4_t*>(bs0 + size_t(k0 + KK * u) * kstride);
        w1[b][u] = *reinterpret_cast<const u32x4_t*>(bs1 + size_t(k0 + KK * u) * kstride);
        a0[b][u] = *reinterpret_cast<const u32x4_t*>(arow[0] + k0 + KK * u);
      }
    };
    // k-major weights: park the loaded blocks, then read the fragments back transposed
    auto transpose_set = [&](int b) {
      if constexpr (BKN) {
#pragma unroll
        for (int u = 0; u < kPipe; ++u) {
          *reinterpret_cast<u32x4_t*>(wpark + u * 1024 + woff) = w0[b][u];
          *reinterpret_cast<u32x4_t*>(wpark + (kPipe + u) * 1024 + woff) = w1[b][u];
        }
#pragma unroll
        for (int u = 0; u < kPipe; ++u) {
          w0[b][u] = __builtin_bit_cast(u32x4_t, read_kn_frag2(wpark + u * 1024 + roff0, wpark + u * 1024 + roff1));
          w1[b][u] = __builtin_bit_cast(u32x4_t, read_kn_frag2(wpark + (kPipe + u) * 1024 + roff0, wpark + (kPipe + u) * 1024 + roff1));
        }
      }
    };
    auto mma_set = [&](int b, int k0) {
      transpose_set(b);
#pragma unroll
      for (int u = 0; u < kPipe; ++u) {
#pragma unroll
        for (int rb = 0; rb < kMaxRowBlocks; ++rb) {
          if (rb < nrb) {
            const u32x4_t a = rb == 0 ? a0[b][u] : *reinterpret_cast<const u32x4_t*>(arow[rb] + k0 + KK * u);
            acc[0][rb] = Mma16<T>::mma(a, w0[b][u], acc[0][rb]);
            acc[1][rb] = Mma16<T>::mma(a, w1[b][u], acc[1][rb]);
          }
        }
      }
    };
    if (nset > 0) load_set(0, kb);
    int set = 0;
    for (; set + 2 <= nset; set += 2) {
      load_set(1, kb + (set + 1) * KK * kPipe);
      mma_set(0, kb + set * KK * kPipe);
      if (set + 2 < nset) load_set(0, kb + (set + 2) * KK * kPipe);
      mma_set(1, kb + (set + 1) * KK * kPipe);
    }
    if (set < nset) mma_set(0, kb + set * KK * kPipe);
    int k0 = kb + nset * KK * kPipe;
    for (; k0 < ke; k0 += KK) {
      u32x4_t v0 = *reinterpret_cast<const u32x4_t*>(bs0 + size_t(k0) * kstride);
      u32x4_t v1 = *reinterpret_cast<const u32x4_t*>(bs1 + size_t(k0) * kstride);
      if constexpr (BKN) {
        *reinterpret_cast<u32x4_t*>(wpark + woff) = v0;
        *reinterpret_cast<u32x4_t*>(wpark + kPipe * 1024 + woff) = v1;
        v0 = __builtin_bit_cast(u32x4_t, read_kn_frag2(wpark + roff0, wpark + roff1));
        v1 = __builtin_bit_cast(u32x4_t, read_kn_frag2(wpark + kPipe * 1024 + roff0, wpark + kPipe * 1024 + roff1));
      }
#pragma unroll
      for (int rb = 0; rb < kMaxRowBlocks; ++rb) {
        if (rb < nrb) {
          const u32x4_t a = *reinterpret_cast<const u32x4_t*>(arow[rb] + k0);
          acc[0][rb] = Mma16<T>::mma(a, v0, acc[0][rb]);
          acc[1][rb] = Mma16<T>::mma(a, v1, acc[1][rb]);
        }
      }
    }
    // with adapters K may end inside a step: its vectors past the end are zeros
    if constexpr (std::is_same<AD, Adapters>::value) {
      const int kt = KK * (K / KK);
      if (kt < K && (KS == 1 || wave == KS - 1)) {
        const u32x4_t zero = {0, 0, 0, 0};
        const bool a_in = kt + kg < K, b_in = BKN ? kt + (lane >> 1) < K : a_in;
        u32x4_t v0 = b_in ? *reinterpret_cast<const u32x4_t*>(bs0 + size_t(kt) * kstride) : zero;
        u32x4_t v1 = b_in ? *reinterpret_cast<const u32x4_t*>(bs1 + size_t(kt) * kstride) : zero;
        if constexpr (BKN) {
          *reinterpret_cast<u32x4_t*>(wpark + woff) = v0;
          *reinterpret_cast<u32x4_t*>(wpark + kPipe * 1024 + woff) = v1;
          v0 = __builtin_bit_cast(u32x4_t, read_kn_frag2(wpark + roff0, wpark + roff1));
          v1 = __builtin_bit_cast(u32x4_t, read_kn_frag2(wpark + kPipe * 1024 + roff0, wpark + kPipe * 1024 + roff1));
        }
#pragma unroll
        for (int rb = 0; rb < kMaxRowBlocks; ++rb) {
          if (rb < nrb) {
            const u32x4_t a = a_in ? *reinterpret_cast<const u32x4_t*>(arow[rb] + kt) : zero;
            acc[0][rb] = Mma16<T>::mma(a, v0, acc[0][rb]);
            acc[1][rb] = Mma16<T>::mma(a, v1, acc[1][rb]);
          }
        }
      }
    }
    // adapters' share, then the stores of one row block.  16x16 layout: lane -> weight row (column of
    // the output) lane & 15, register i -> token row 4*(lane/16) + i of the row block
    auto finish = [&](int rb, int id, f32x4_t& s0, f32x4_t& s1) {
      if constexpr (std::is_same<AD, Adapters>::value)
        add_adapters<T, NMAT>(ad, expert, seg0 + m0 + rb * 16, min(16, seg_n - m0 - rb * 16), id, col0, N, s0, s1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = m0 + rb * 16 + 4 * (lane >> 4) + i;
        if (r < seg_n) {
          T* crow = C + size_t(seg0 + r) * N;
          if (NMAT == 2) {
            const int col = col0 + (lane & 15);
            if (col < N) {
              crow[col] = Elem<T>::from_f32(silu(s0[i]) * s1[i]);
              if constexpr (SAVE) {
                Gs[size_t(seg0 + r) * N + col] = Elem<T>::from_f32(s0[i]);
                Us[size_t(seg0 + r) * N + col] = Elem<T>::from_f32(s1[i]);
              }
            }
          } else {
            const int c0 = col0 + (lane & 15), c1 = c0 + 16;
            if (c0 < N) crow[c0] = Elem<T>::from_f32(s0[i]);
            if (c1 < N) crow[c1] = Elem<T>::from_f32(s1[i]);
          }
        }
      }
    };
    if constexpr (KS == 1) {
#pragma unroll
      for (int rb = 0; rb < kMaxRowBlocks; ++rb)
        if (rb < nrb) finish(rb, ids[rb], acc[0][rb], acc[1][rb]);
    } else {
      static_assert(KS == kThreads / 64 && KS == kMaxRowBlocks, "a wave for every row block");
      __shared__ f32x4_t sums[KS][kMaxRowBlocks][2][64];
      if (m0 > 0) __syncthreads();  // the sums before these have been read
#pragma unroll
      for (int rb = 0; rb < kMaxRowBlocks; ++rb)
        if (rb < nrb) {
          sums[wave][rb][0][lane] = acc[0][rb];
          sums[wave][rb][1][lane] = acc[1][rb];
        }
      __syncthreads();
      if (wave < nrb) {
        f32x4_t s0 = sums[0][wave][0][lane], s1 = sums[0][wave][1][lane];
#pragma unroll
        for (int w = 1; w < KS; ++w) {
          s0 += sums[w][wave][0][lane];
          s1 += sums[w][wave][1][lane];
        }
        finish(wave, ids[0], s0, s1);
      }
    }
  }
}

// bkn: k-major weights (see gemm_kernel)
// ks: the waves split K (adapters alone).  experts: how many can have rows (with adapters: blocks of
// experts without any take their places for a while; one row on each of 8 of 128 experts, down product
// 11.8 -> 9.5 us)
template <typename T, int NMAT, class AD>
moe_status launch(const char* name, const T* A, const int32_t* offsets, const T* B0, const T* B1, T* C, int experts, int N,
                  int K, bool bkn, bool ks, hipStream_t s, T* Gs, T* Us, const AD& ad) {
  const int cols = ks ? cols_per_block<NMAT>() / 4 : cols_per_block<NMAT>();
  const dim3 grid(unsigned((N + cols - 1) / cols), unsigned(experts));
  constexpr bool kKn = sizeof(T) == 2;  // float32 layers come n-major alone
#define MOE_SKINNY(SAVE_, KS_)                                                                                     \
  do {                                                                                                             \
    if (kKn && bkn)                                                                                                \
      MOE_LAUNCH(name, (gemm_kernel<T, NMAT, SAVE_, kKn, AD, KS_>), grid, dim3(kThreads), 0, s, A, offsets, B0, B1, C, N, K, Gs, Us, ad); \
    else                                                                                                           \
      MOE_LAUNCH(name, (gemm_kernel<T, NMAT, SAVE_, false, AD, KS_>), grid, dim3(kThreads), 0, s, A, offsets, B0, B1, C, N, K, Gs, Us, ad); \
  } while (0)
  if constexpr (std::is_same<AD, Adapters>::value) {
    if (ks) MOE_SKINNY(false, 4);
    else MOE_SKINNY(false, 1);
  } else {
    if (NMAT == 2 && Gs != nullptr) MOE_SKINNY(NMAT == 2, 1);
    else MOE_SKINNY(false, 1);
  }
#undef MOE_SKINNY
  return MOE_OK;
}

constexpr int kFullBlocks = 1024;

// between(): enqueued between the two products
template <typename T, class AD, class Between>
moe_status launch_both(const FfnArgs& a, const AD& gu, const AD& dn, const Between& between) {
  const moe_layer_desc* d = a.d;
  const int L = d->local_count, H = d->hidden, I = d->intermediate;
  T* h = static_cast<T*>(a.h);
  const bool kn = d->weight_layout == MOE_WEIGHTS_IN_OUT;
  const int experts = std::is_same<AD, Adapters>::value ? int(std::min<int64_t>(a.max_pairs, L)) : L;
  // fewer than kFullBlocks blocks, if every row is another expert's, leave the waves waiting for
  // their own loads
  const auto ks = [&](int N, int cols) {
    return std::is_same<AD, Adapters>::value && int64_t(experts) * ((N + cols - 1) / cols) < kFullBlocks;
  };
  moe_status st = launch<T, 2>("ffn_gate_up", static_cast<const T*>(a.x_sorted), a.offsets,
                            static_cast<const T*>(a.w_gate), static_cast<const T*>(a.w_up), h, experts, I, H, kn, ks(I, cols_per_block<2>()), a.s,
                            static_cast<T*>(a.g_out), static_cast<T*>(a.u_out), gu);
  if (st != MOE_OK) return st;
  st = between();
  if (st != MOE_OK) return st;
  return launch<T, 1>("ffn_down", h, a.offsets, static_cast<const T*>(a.w_down), static_cast<const T*>(a.w_down),
                   static_cast<T*>(a.y_sorted), experts, H, I, kn, ks(H, cols_per_block<1>()), a.s, static_cast<T*>(nullptr),
                   static_cast<T*>(nullptr), dn);
}

}  // namespace skinny

}  // namespace

bool skinny_ffn_fits(const moe_layer_desc* d, int64_t max_pairs) {
  return d->dtype == MOE_BF16 && max_pairs <= int64_t(32) * d->local_count && skinny::supported(d->hidden) &&
         skinny::supported(d->intermediate);
}

moe_status launch_skinny_ffn(const FfnArgs& a) {
  return skinny::launch_both<bf16_t>(a, NoAdapters(), NoAdapters(), [] { return MOE_OK; });
}

// With adapters any width, and float32 rows where the weights lie along k.
bool skinny_adapted_fits(const moe_layer_desc* d, int64_t max_pairs) {
  return max_pairs <= int64_t(32) * d->local_count && (d->dtype == MOE_BF16 || d->weight_layout == MOE_WEIGHTS_OUT_IN);
}

moe_status launch_skinny_adapted(const AdaptedFfnArgs& a) {
  const Adapters gu = gate_up_adapters(a.f.d, a.ad, a.w), dn = down_adapters(a.f.d, a.ad, a.w);
  const auto between = [&] { return launch_adapter_shrink(a, true); };
  return a.f.d->dtype == MOE_BF16 ? skinny::launch_both<bf16_t>(a.f, gu, dn, between)
                                  : skinny::launch_both<float>(a.f, gu, dn, between);
}

}  // namespace moe
