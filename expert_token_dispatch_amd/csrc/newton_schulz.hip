// The weight update: momentum, orthogonalisation by Newton-Schulz steps, step on the weight.
//
// One step takes X to p(A) X with A = X X^T and p(t) = a + b t + c t^2 (m x m on the
// shorter side; for a tall matrix A = X^T X and the factor stands on the right), so a
// singular value s goes to s p(s^2) and the singular vectors stay.
//
// Steps on the m x m side.  p(A_0), p(A_1), ... are polynomials of A_0: they commute and
// are symmetric.  So a phase of several steps needs X only at its ends:
//   A_0 = X X^T;  P_j = p(A_j),  Q_{j+1} = P_j Q_j,  A_{j+1} = P_j (P_j A_j);  X <- Q X.
// P and Q are held without their multiples of I: P = a I + P', Q = q I + Q' with q = a^j,
// so every product is one of P' or Q' plus multiples of matrices at hand, added in float32
// (a I inside P would be rounded alike on the whole diagonal: 4% off for a matrix of rank
// one, whose large singular value lives on the difference of a and the rest).
// Every m x m product is symmetric: its upper triangle of tiles is computed and mirrored.
// In units of m^3 multiply-adds (r the ratio of the sides) five single steps cost
// 5 (3 r + 1), a phase of three and one of two 6 r + 14: the same at r = 1, two thirds
// at r = 8/3.
//
// Rounding.  Small singular values are multiplied by up to a^steps (485 for five usual
// steps) while the large ones stay near 1, and a rounding of X is relative to the large
// ones.  In bfloat16 that leaves 1 to 5% of error, in float16 0.1 to 0.6%, nearly all of
// it from the X of the first steps; A and P may be rounded to float16, for p changes
// little with them.  So a bf16 layer's products run on float16 operands (the same MFMA
// rate as bfloat16) scaled by powers of two that keep every value in its normal range,
// and the X of the first two steps are sums of two float16 (22 bits).  In a phase of three
// steps only X_0 is such an X.  Phases are at most three steps long, since rounding errors
// of A grow by up to a^2 a step in the directions where A is small; they average out over
// the shorter side (simulated error of the result, 0.16% of it the bfloat16 result's own:
// 0.9% at 64, 0.4% at 128, 0.25% at 512, against 0.2% in single steps), so matrices with a
// shorter side of up to kSingleSteps take single steps, where the launches count more
// than the products.  Float32 layers run on float32 operands in single steps (a phase
// would double the error).
#include <math.h>

#include <algorithm>

#include "ffn_common.h"
#include "kernels.h"

namespace moe {
namespace {

typedef _Float16 f16_t;
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

constexpr int kPad = 64;       // sides of the working matrices are multiples of this
constexpr int kThreads = 256;

// Scales of the working values.  Singular values are at most 3 (the coefficients are
// checked), so |X| <= 3, |A| <= 9, and |P'|, |Q'| <= a^3 <= 64 (up to a small factor): the
// largest stored values are 3 * 2^14, 9 * 2^12 and 64 * 2^9, below float16's 65504.
template <typename T> struct Scale;
template <> struct Scale<f16_t> { static constexpr int x = 14, a = 12, q = 9; };
template <> struct Scale<float> { static constexpr int x = 0, a = 0, q = 0; };

int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// ---- the plan of one call ------------------------------------------------------------
struct Plan {
  int count, rows, cols;  // the user's stack
  int rp, cp;             // sides rounded up
  int mp;                 // the shorter side, rounded up
  bool tall;
  size_t x_bytes, q_bytes;      // one stack of X, of m x m matrices
  int nblk;                     // partial sums of squares per matrix
  bool single;                  // phases of one step (see the top of the file)
  size_t o_part, o_x[4], o_q[5], bytes;
};

constexpr int kSingleSteps = 256;

// elements of a matrix that one block of the norm kernel adds up
constexpr int64_t kNormElems = 16384;
constexpr int kMaxPartials = 256;

Plan make_plan(const moe_muon_desc* m) {
  Plan p{};
  p.count = m->count;
  p.rows = m->rows;
  p.cols = m->cols;
  p.rp = int(round_up(m->rows, kPad));
  p.cp = int(round_up(m->cols, kPad));
  p.tall = m->rows > m->cols;
  p.mp = p.tall ? p.cp : p.rp;
  const size_t es = m->dtype == MOE_BF16 ? 2 : 4;
  p.x_bytes = align_up(size_t(p.count) * p.rp * p.cp * es, 256);
  p.q_bytes = align_up(size_t(p.count) * p.mp * p.mp * es, 256);
  const int64_t n = int64_t(m->rows) * m->cols;
  p.nblk = int(std::min<int64_t>(kMaxPartials, (n + kNormElems - 1) / kNormElems));
  size_t o = 0;
  auto take = [&](size_t b) {
    const size_t r = o;
    o += align_up(b, 256);
    return r;
  };
  p.o_part = take(size_t(p.count) * p.nblk * sizeof(double));
  p.single = m->dtype == MOE_F32 || std::min(m->rows, m->cols) <= kSingleSteps;
  // X and the X after it, then (float16) the low halves of X_0 and, in single steps, X_1
  const bool split = m->dtype == MOE_BF16;
  const int xs = split ? (p.single ? 4 : 3) : 2;
  for (int i = 0; i < xs; ++i) p.o_x[i] = take(p.x_bytes);
  for (int i = 0; i < (p.single ? 2 : 5); ++i) p.o_q[i] = take(p.q_bytes);
  p.bytes = o;
  return p;
}

// ---- momentum and norm ---------------------------------------------------------------
// Per matrix the sum of squares of U in double (a gradient's squares leave float32's range
// long before its values do), by blocks in a fixed order.  MOM: the momentum is updated
// on the way.  Bound by HBM.
template <typename T, bool MOM>
__global__ __launch_bounds__(kThreads) void norm_kernel(const T* __restrict__ g, float* __restrict__ mom, float mu,
                                                        int nesterov, int64_t n, double* __restrict__ part) {
  const size_t z = blockIdx.y;
  const T* gz = g + z * n;
  float* mz = MOM ? mom + z * n : nullptr;
  double s = 0.0;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < n; i += int64_t(gridDim.x) * kThreads) {
    float u = Elem<T>::to_f32(gz[i]);
    if constexpr (MOM) {
      const float v = mu * mz[i] + u;
      mz[i] = v;
      u = nesterov ? u + mu * v : v;
    }
    s += double(u) * double(u);
  }
  for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d, 64);
  __shared__ double w[kThreads / 64];
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) part[z * gridDim.x + blockIdx.x] = (w[0] + w[1]) + (w[2] + w[3]);
}

// X_0 = U / (|U| + eps), scaled, into the padded working matrices (hi, and lo with what
// hi's rounding left); the padding is zero.
template <typename T, typename W, bool MOM>
__global__ __launch_bounds__(kThreads) void start_kernel(const T* __restrict__ g, const float* __restrict__ mom, float mu,
                                                         int nesterov, int rows, int cols, int rp, int cp,
                                                         const double* __restrict__ part, int nblk, float eps,
                                                         W* __restrict__ hi, W* __restrict__ lo) {
  const size_t z = blockIdx.y;
  __shared__ double total;
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int i = 0; i < nblk; ++i) s += part[z * nblk + i];
    total = s;
  }
  __syncthreads();
  const double norm = sqrt(total) + double(eps);
  const double inv = norm > 0.0 ? double(1 << Scale<W>::x) / norm : (norm == 0.0 ? 0.0 : norm);
  const T* gz = g + z * rows * cols;
  const float* mz = MOM ? mom + z * rows * cols : nullptr;
  W* hz = hi + z * rp * cp;
  W* lz = lo == nullptr ? nullptr : lo + z * rp * cp;
  const int64_t n = int64_t(rp) * cp;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < n; i += int64_t(gridDim.x) * kThreads) {
    const int r = int(i / cp), c = int(i % cp);
    float x = 0.f;
    if (r < rows && c < cols) {
      const int64_t at = int64_t(r) * cols + c;
      float u = Elem<T>::to_f32(gz[at]);
      if constexpr (MOM) u = nesterov ? u + mu * mz[at] : mz[at];
      x = float(double(u) * inv);
    }
    const W h = W(x);
    hz[i] = h;
    if (lz != nullptr) lz[i] = W(x - float(h));
  }
}

// ---- products ------------------------------------------------------------------------
// C = alpha A B (+ beta D + beta2 D2) for every matrix of the stack.
struct Product {
  const void* a;      // AK: k-major, element (m, k) at a[k * lda + m]; else m-major
  const void* b;      // BK: k-major, element (n, k) at b[k * ldb + n]; else n-major
  const void* a2;     // second pair of operands, added (NULL: none)
  const void* b2;
  const void* d;      // added, elements where C's are (NULL: none)
  const void* d2;
  void* c;
  void* c2;           // what C's rounding leaves (NULL: not kept)
  size_t sa, sb, sc;  // elements from one matrix of the stack to the next 
  int m, n, k, lda, ldb, ldc;
  float alpha, beta, beta2;
  int sym;            // C is symmetric: upper tiles only, mirrored
  // the last product's epilogue: the result, or the step on the weight
  void* out;
  float* master;
  int rows, cols;
  float keep, step;   // W = keep W - step C
};

enum OutKind { kInner = 0, kResult = 1, kUpdate = 2 };

template <typename W> struct Mma;
template <> struct Mma<f16_t> {
  static constexpr int kVec = 1;  // 16-byte vectors of a lane's 8 k values
  __device__ static void mma(const uint4* a, const uint4* b, f32x16_t& c) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a[0]), __builtin_bit_cast(f16x8_t, b[0]), c,
                                               0, 0, 0);
  }
};
template <> struct Mma<float> {
  static constexpr int kVec = 2;
  __device__ static void mma(const uint4* a, const uint4* b, f32x16_t& c) {
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[v].x), __uint_as_float(b[v].x), c, 0, 0, 0);
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[v].y), __uint_as_float(b[v].y), c, 0, 0, 0);
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[v].z), __uint_as_float(b[v].z), c, 0, 0, 0);
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[v].w), __uint_as_float(b[v].w), c, 0, 0, 0);
    }
  }
};

// One operand's LDS tile: 64 rows (m or n) by kBK k values, m-major as [64][kBK + pad],
// k-major as [kBK][64 + pad].  128 bytes of k either way.
template <typename W, bool KM>
struct OpTile {
  static constexpr int kBK = 128 / int(sizeof(W));
  static constexpr int kEpv = 16 / int(sizeof(W));
  static constexpr int kRows = KM ? kBK : 64;
  static constexpr int kCols = KM ? 64 : kBK;
  static constexpr int kLd = kCols + kEpv;  // rows padded by 16 bytes
  static constexpr int kChunks = kRows * kCols / kEpv / kThreads;
  static constexpr int kElems = kRows * kLd;

  // the 16-byte pieces of this thread, from the tile's first row (m-major) or column
  __device__ static void load(const W* p, int ld, uint4 (&r)[kChunks]) {
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int c = threadIdx.x + j * kThreads;
      r[j] = *reinterpret_cast<const uint4*>(p + size_t(c / (kCols / kEpv)) * ld + (c % (kCols / kEpv)) * kEpv);
    }
  }
  __device__ static void store(W* t, const uint4 (&r)[kChunks]) {
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int c = threadIdx.x + j * kThreads;
      *reinterpret_cast<uint4*>(t + (c / (kCols / kEpv)) * kLd + (c % (kCols / kEpv)) * kEpv) = r[j];
    }
  }
  // row base + (lane & 31), k values kc + 8 (lane / 32) .. +7
  __device__ static void frag(const W* t, int base, int kc, uint4* f) {
    const int lane = threadIdx.x & 63;
    if constexpr (!KM) {
      const uint4* p = reinterpret_cast<const uint4*>(t + (base + (lane & 31)) * kLd + kc + 8 * (lane >> 5));
#pragma unroll
      for (int v = 0; v < Mma<W>::kVec; ++v) f[v] = p[v];
    } else if constexpr (sizeof(W) == 2) {
      const int G = lane >> 4, i = lane & 15;
      const W* p = t + (kc + 8 * (G >> 1) + (i >> 2)) * kLd + base + 16 * (G & 1) + 4 * (i & 3);
      f[0] = __builtin_bit_cast(uint4, read_kn_frag2(reinterpret_cast<const char*>(p),
                                                     reinterpret_cast<const char*>(p + 4 * kLd)));
    } else {
      const W* p = t + (kc + 8 * (lane >> 5)) * kLd + base + (lane & 31);
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(p[k * kLd]);
      f[0] = make_uint4(w[0], w[1], w[2], w[3]);
      f[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
};

// 64 x 64 tiles, four waves 2 x 2, one MFMA 32x32 block each; the next k slice is in
// registers while this one is multiplied.  Sides are multiples of 64, so no access needs
// a bound but the last product's into the user's matrix.
template <typename W, typename T, bool AK, bool BK, int OUT>
__global__ __launch_bounds__(kThreads) void product_kernel(Product p) {
  using TA = OpTile<W, AK>;
  using TB = OpTile<W, BK>;
  constexpr int kBK = TA::kBK;
  const int tm = blockIdx.y, tn = blockIdx.x;
  if (p.sym && tn < tm) return;
  const size_t z = blockIdx.z;
  __shared__ __attribute__((aligned(16))) W as[TA::kElems];
  __shared__ __attribute__((aligned(16))) W bs[TB::kElems];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  f32x16_t acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.f;
  const size_t ka = AK ? size_t(p.lda) : 1, kb = BK ? size_t(p.ldb) : 1;
  const size_t a0 = z * p.sa + (AK ? size_t(tm) * 64 : size_t(tm) * 64 * p.lda);
  const size_t b0 = z * p.sb + (BK ? size_t(tn) * 64 : size_t(tn) * 64 * p.ldb);
  const int slices = p.k / kBK, total = p.a2 != nullptr ? 2 * slices : slices;
  uint4 ra[TA::kChunks], rb[TB::kChunks];
  auto fetch = [&](int s) {
    const bool second = s >= slices;
    const size_t k0 = size_t(second ? s - slices : s) * kBK;
    TA::load(static_cast<const W*>(second ? p.a2 : p.a) + a0 + k0 * ka, p.lda, ra);
    TB::load(static_cast<const W*>(second ? p.b2 : p.b) + b0 + k0 * kb, p.ldb, rb);
  };
  fetch(0);
  for (int s = 0; s < total; ++s) {
    __syncthreads();
    TA::store(as, ra);
    TB::store(bs, rb);
    __syncthreads();
    if (s + 1 < total) fetch(s + 1);
#pragma unroll
    for (int kc = 0; kc < kBK; kc += 16) {
      uint4 fa[Mma<W>::kVec], fb[Mma<W>::kVec];
      TA::frag(as, wm, kc, fa);
      TB::frag(bs, wn, kc, fb);
      Mma<W>::mma(fa, fb, acc);
    }
  }
  // lane -> column (lane & 31), register r -> row 8 (r / 4) + 4 (lane / 32) + r % 4
  const int col = tn * 64 + wn + (lane & 31);
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int row = tm * 64 + wm + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
    const size_t ci = z * p.sc + size_t(row) * p.ldc + col;
    float v = p.alpha * acc[r];
    if (p.d2 != nullptr) v += p.beta2 * float(static_cast<const W*>(p.d2)[ci]);
    if (p.d != nullptr) v += p.beta * float(static_cast<const W*>(p.d)[ci]);
    if constexpr (OUT == kInner) {
      const W h = W(v);
      static_cast<W*>(p.c)[ci] = h;
      if (p.c2 != nullptr) static_cast<W*>(p.c2)[ci] = W(v - float(h));
      if (p.sym && tn != tm) static_cast<W*>(p.c)[z * p.sc + size_t(col) * p.ldc + row] = h;
    } else if (row < p.rows && col < p.cols) {
      const size_t at = z * p.rows * p.cols + size_t(row) * p.cols + col;
      T* o = static_cast<T*>(p.out) + at;
      if constexpr (OUT == kUpdate) {
        const float w = p.master != nullptr ? p.master[at] : Elem<T>::to_f32(*o);
        v = w * p.keep - v * p.step;
        if (p.master != nullptr) p.master[at] = v;
      }
      *o = Elem<T>::from_f32(v);
    }
  }
}

template <typename W, typename T, int OUT>
moe_status launch_product(const char* name, const Product& p, bool ak, bool bk, int count, hipStream_t s) {
  const dim3 grid(unsigned(p.n / 64), unsigned(p.m / 64), unsigned(count));
  if (ak && bk) {
    MOE_LAUNCH(name, (product_kernel<W, T, true, true, OUT>), grid, dim3(kThreads), 0, s, p);
  } else if (bk) {
    MOE_LAUNCH(name, (product_kernel<W, T, false, true, OUT>), grid, dim3(kThreads), 0, s, p);
  } else {
    MOE_LAUNCH(name, (product_kernel<W, T, false, false, OUT>), grid, dim3(kThreads), 0, s, p);
  }
  return MOE_OK;
}

#define TRY_NS(expr)                       \
  do {                                     \
    const moe_status _s = (expr);          \
    if (_s != MOE_OK) return _s;           \
  } while (0)

template <typename T, typename W>
struct Run {
  const MuonArgs& a;
  Plan p;
  char* base;
  static constexpr bool kSplit = sizeof(W) == 2;  // X_0 as the sum of two

  W* x(int i) const { return reinterpret_cast<W*>(base + p.o_x[i]); }
  W* q(int i) const { return reinterpret_cast<W*>(base + p.o_q[i]); }

  moe_status start() const {
    const int64_t n = int64_t(p.rows) * p.cols;
    const moe_muon_desc* m = a.m;
    const T* g = static_cast<const T*>(a.grad);
    double* part = reinterpret_cast<double*>(base + p.o_part);
    const dim3 gn(unsigned(p.nblk), unsigned(p.count));
    const int64_t np = int64_t(p.rp) * p.cp;
    const dim3 gs(unsigned(std::min<int64_t>(1024, (np + 2047) / 2048)), unsigned(p.count));
    W* lo = kSplit ? x(2) : nullptr;
    if (a.momentum != nullptr) {
      MOE_LAUNCH("muon_momentum", (norm_kernel<T, true>), gn, dim3(kThreads), 0, a.s, g, a.momentum, m->momentum,
                 m->nesterov, n, part);
      MOE_LAUNCH("muon_start", (start_kernel<T, W, true>), gs, dim3(kThreads), 0, a.s, g, a.momentum, m->momentum,
                 m->nesterov, p.rows, p.cols, p.rp, p.cp, part, p.nblk, m->eps, x(0), lo);
    } else {
      MOE_LAUNCH("orth_norm", (norm_kernel<T, false>), gn, dim3(kThreads), 0, a.s, g, static_cast<float*>(nullptr), 0.f,
                 0, n, part);
      MOE_LAUNCH("orth_start", (start_kernel<T, W, false>), gs, dim3(kThreads), 0, a.s, g,
                 static_cast<const float*>(nullptr), 0.f, 0, p.rows, p.cols, p.rp, p.cp, part, p.nblk, m->eps, x(0), lo);
    }
    return MOE_OK;
  }

  // A = X X^T (or X^T X)
  moe_status gram(const W* x, W* out) const {
    Product g{};
    g.a = g.b = x;
    g.c = out;
    g.sa = g.sb = size_t(p.rp) * p.cp;
    g.sc = size_t(p.mp) * p.mp;
    g.m = g.n = g.ldc = p.mp;
    g.k = p.tall ? p.rp : p.cp;
    g.lda = g.ldb = p.cp;
    g.alpha = ldexpf(1.f, Scale<W>::a - 2 * Scale<W>::x);
    g.sym = 1;
    return launch_product<W, T, kInner>("ns_gram", g, p.tall, p.tall, p.count, a.s);
  }

  // out = alpha u v + beta d (+ beta2 d2), all m x m, symmetric and commuting
  moe_status square(const char* name, const W* u, const W* v, W* out, float alpha, const W* d, float beta,
                    const W* d2 = nullptr, float beta2 = 0.f) const {
    Product g{};
    g.a = u;
    g.b = v;  // symmetric: its columns are its rows
    g.d = d;
    g.d2 = d2;
    g.c = out;
    g.sa = g.sb = g.sc = size_t(p.mp) * p.mp;
    g.m = g.n = g.k = g.lda = g.ldb = g.ldc = p.mp;
    g.alpha = alpha;
    g.beta = beta;
    g.beta2 = beta2;
    g.sym = 1;
    return launch_product<W, T, kInner>(name, g, false, false, p.count, a.s);
  }

  // (q0 I + q) X (or X (q0 I + q)), X = x + x2; to `out` (+ out2), or into the user's
  // result when out is NULL
  moe_status apply(float q0, const W* q, const W* x, const W* x2, W* out, W* out2) const {
    Product g{};
    const size_t sq = size_t(p.mp) * p.mp, sx = size_t(p.rp) * p.cp;
    // the low halves first, while the sums are small
    const W* first = x2 != nullptr ? x2 : x;
    const W* second = x2 != nullptr ? x : nullptr;
    if (p.tall) {
      g.a = first;
      g.a2 = second;
      g.b = q;
      g.b2 = q;
      g.sa = sx;
      g.sb = sq;
      g.lda = p.cp;
      g.ldb = p.mp;
    } else {
      g.a = q;
      g.a2 = second != nullptr ? q : nullptr;
      g.b = first;
      g.b2 = second;
      g.sa = sq;
      g.sb = sx;
      g.lda = p.mp;
      g.ldb = p.cp;
    }
    g.sc = sx;
    g.m = p.rp;
    g.n = g.ldc = p.cp;
    g.k = p.mp;
    g.d = x;
    g.d2 = x2;
    const bool bk = !p.tall;
    if (out != nullptr) {
      g.beta = g.beta2 = q0;
      g.c = out;
      g.c2 = out2;
      g.alpha = ldexpf(1.f, -Scale<W>::q);
      return launch_product<W, T, kInner>("ns_apply", g, false, bk, p.count, a.s);
    }
    g.alpha = ldexpf(1.f, -Scale<W>::q - Scale<W>::x);
    g.beta = g.beta2 = ldexpf(q0, -Scale<W>::x);
    g.out = a.out;
    g.rows = p.rows;
    g.cols = p.cols;
    if (a.momentum == nullptr) return launch_product<W, T, kResult>("ns_apply_result", g, false, bk, p.count, a.s);
    g.master = a.master;
    g.keep = 1.f - a.m->lr * a.m->weight_decay;
    g.step = a.m->lr * a.m->update_scale;
    return launch_product<W, T, kUpdate>("muon_apply", g, false, bk, p.count, a.s);
  }

  moe_status run() const {
    TRY_NS(start());
    const float iq = ldexpf(1.f, -Scale<W>::q);
    int cur = 0, done = 0;  // X in x(cur), its low half, if it has one, in x(cur + 2)
    bool split = kSplit;
    while (done < a.m->steps) {
      const int len = std::min(a.m->steps - done, p.single ? 1 : (done == 0 ? 3 : 2));
      // A in q(0); P, Q and two for what is being formed in the others
      W* A = q(0);
      W* Q = q(1);
      float q0 = a.ca;
      TRY_NS(gram(x(cur), A));
      for (int k = 0; k < len; ++k) {
        W* P = k == 0 ? Q : q(2);
        TRY_NS(square("ns_poly", A, A, P, ldexpf(a.cc, Scale<W>::q - 2 * Scale<W>::a), A,
                      ldexpf(a.cb, Scale<W>::q - Scale<W>::a)));
        if (k + 1 < len) {
          TRY_NS(square("ns_next", P, A, q(4), iq, A, a.ca));
          TRY_NS(square("ns_next", P, q(4), A, iq, q(4), a.ca));
        }
        if (k > 0) {
          W* N = Q == q(1) ? q(3) : q(1);
          TRY_NS(square("ns_join", P, Q, N, iq, Q, a.ca, P, q0));
          Q = N;
          q0 *= a.ca;
        }
      }
      done += len;
      const bool last = done == a.m->steps, keep = kSplit && p.single && done == 1;
      TRY_NS(apply(q0, Q, x(cur), split ? x(cur + 2) : nullptr, last ? nullptr : x(cur ^ 1), keep ? x((cur ^ 1) + 2) : nullptr));
      cur ^= 1;
      split = keep;
    }
    return MOE_OK;
  }
};

}  // namespace

int64_t muon_matrix_bytes(const moe_muon_desc* m) {
  return round_up(m->rows, kPad) * round_up(m->cols, kPad) * (m->dtype == MOE_BF16 ? 2 : 4);
}

size_t muon_workspace_bytes(const moe_muon_desc* m) { return make_plan(m).bytes; }

moe_status launch_muon(const MuonArgs& a) {
  const Plan p = make_plan(a.m);
  char* base = static_cast<char*>(a.ws);
  if (a.m->dtype == MOE_BF16) return Run<bf16_t, f16_t>{a, p, base}.run();
  return Run<float, float>{a, p, base}.run();
}

}  // namespace moe
