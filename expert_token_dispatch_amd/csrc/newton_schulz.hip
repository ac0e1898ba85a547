// The weight update: momentum, orthogonalisation by Newton-Schulz steps, step on the weight.
//
// One step takes X to p(A) X with A = X X^T and p(t) = a + b t + c t^2 (m x m on the
// shorter side; for a tall matrix A = X^T X and the factor stands on the right), so a
// singular value s goes to s p(s^2) and the singular vectors stay.
//
// Steps on the m x m side.  p(A_0), p(A_1), ... are polynomials of A_0: they commute and
// are symmetric.  So a phase of several steps needs X only at its ends:
//   A_0 = X X^T;  P_j = p(A_j),  Q_{j+1} = P_j Q_j,  A_{j+1} = P_j (P_j A_j);  X <- Q X.
// P and Q are held as a float32 diagonal and the rest, zero on its diagonal: the multiples
// of I that they carry (a, a^2, a^3 = 41) stand beside values of p of 0.7 for the large
// singular values, and rounding them with the rest would be rounding the difference.  With
// P = D_p + P' a product is P T = P' T + D_p T, and D_p T is added in the epilogue.
// Every m x m product is symmetric: its upper triangle of tiles is computed and mirrored.
// In units of m^3 multiply-adds (r the ratio of the sides) five single steps cost
// 5 (3 r + 1), a phase of three and one of two 6 r + 14: the same at r = 1, two thirds
// at r = 8/3.
//
// Rounding.  Small singular values are multiplied by up to a^steps (485 for five usual
// steps) while the large ones stay near 1, and a rounding of X is relative to the large
// ones.  In bfloat16 that leaves 1 to 5% of error; A and P may be rounded to float16, for
// their errors turn the singular vectors a little but put nothing into directions that X
// does not have.  So a bf16 layer's products run on float16 operands (the same MFMA rate as
// bfloat16) scaled by powers of two, and an X that more than two steps follow is the sum of
// two float16 (22 bits): one float16 would leave 2^-12 in every direction, a^3 = 41 times
// that after three steps, whole percents of a matrix with few directions (rank 4, one
// float16 from the third X on: 0.9% at 5 steps, 10% at 7, 330% at 10; so 0.3, 0.3 and 1.0%,
// where float32 leaves 1.2).  A is formed from the high half alone: what that leaves out
// averages out along K, as the roundings of P and Q do over the entries (1.5% in phases for
// one row of 700 x 520, up to 4% where all entries are alike, 0.3 to 0.6% for random vectors'
// products).  Phases are at most three steps long, since rounding errors
// of A grow by up to a^2 a step in the directions where A is small; they average out over
// the shorter side (simulated error of the result, 0.16% of it the bfloat16 result's own:
// 0.7% at 64, 0.28% at 128, 0.2% at 512, against 0.18% in single steps), so matrices with a
// shorter side of up to 128 take single steps, and up to 256 those that are less than twice
// as long, at some cost away from the square (128 matrices of 256 x 256: 327 us in phases, 319
// in single steps; of 256 x 500: 437 and 548), but not longer ones (32 of 256 x 1024: 224 and
// 282; 256 of 256 x 512: 740 and 1186).  Float32 layers run on float32 operands in single
// steps (a phase would double the error).
#include <math.h>

#include <algorithm>

#include "big_tile.h"
#include "kernels.h"

namespace moe {
namespace {

typedef _Float16 f16_t;
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

constexpr int kPad = 64;       // sides of the working matrices are multiples of this
constexpr int kThreads = 256;

// Scales of the working values.  Singular values are at most 3 (the coefficients are
// checked), so |X| <= 3, |A| <= 9, and |P|, |Q| <= a^3 <= 64 (up to a small factor): the
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
  size_t o_part, o_x[4], o_t[4], o_q[5], o_d[5], bytes;
};

bool single_steps(int rows, int cols) {
  const int shorter = std::min(rows, cols), longer = std::max(rows, cols);
  return shorter <= 128 || (shorter <= 256 && longer < 2 * shorter);
}

// Steps of the phase that starts after `done` of them.
int phase_steps(bool single, int done, int steps) { return std::min(steps - done, single ? 1 : (done == 0 ? 3 : 2)); }

// float16: whether X after `done` steps keeps a low half (X_0 always has one): where more than
// two follow.  In single steps X_1 always does; two steps still multiply its rounding by a^2 = 12.
bool keeps_low(bool single, int done, int steps) {
  return done < steps && (steps - done > 2 || (single && done == 1));
}

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
  p.single = m->dtype == MOE_F32 || single_steps(m->rows, m->cols);
  // X and the X after it, as they are and transposed, and their low halves; the X after X_0 is
  // the first that may keep one.  A low half is read as X is added (as it is) and as the operand
  // of an application: as it is for a tall matrix, else transposed.
  const int first = phase_steps(p.single, 0, m->steps);
  for (int i = 0; i < 4; ++i) {
    const bool used = i < 2 || (m->dtype == MOE_BF16 && (i == 2 || keeps_low(p.single, first, m->steps)));
    p.o_x[i] = take(used ? p.x_bytes : 0);
    p.o_t[i] = take(used && (i < 2 || !p.tall) ? p.x_bytes : 0);
  }
  for (int i = 0; i < (p.single ? 2 : 5); ++i) {
    p.o_q[i] = take(p.q_bytes);
    p.o_d[i] = take(size_t(p.count) * p.mp * sizeof(float));
  }
  p.bytes = o;
  return p;
}

// ---- momentum and norm ---------------------------------------------------------------
// Per matrix the sum of squares of U in double (a gradient's squares leave float32's range
// long before its values do), by blocks in a fixed order.  MOM: the momentum is updated
// on the way.  Bound by HBM.
template <typename T> struct alignas(16) Vec8 {
  T e[8];
};

// Eight elements of a row of `cols` from column c: in one piece where rows are whole pieces
// (vec), else one by one; zeros past the end.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int c, int cols, bool vec, float* f) {
  if (vec && c < cols) {
    const Vec8<T> v = *reinterpret_cast<const Vec8<T>*>(row + c);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = Elem<T>::to_f32(v.e[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = c + k < cols ? Elem<T>::to_f32(row[c + k]) : 0.f;
  }
}

// The stack is walked as runs of eight elements of the whole matrix (n is rows * cols: rows
// do not matter here).
template <typename T, bool MOM>
__global__ __launch_bounds__(kThreads) void norm_kernel(const T* __restrict__ g, float* __restrict__ mom, float mu,
                                                        int nesterov, int64_t n, double* __restrict__ part) {
  const size_t z = blockIdx.y;
  const T* gz = g + z * n;
  float* mz = MOM ? mom + z * n : nullptr;
  const bool vec = n % 8 == 0;  // every matrix starts on a whole piece
  double s = 0.0;
  for (int64_t i = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * 8; i < n; i += int64_t(gridDim.x) * kThreads * 8) {
    float u[8], m[8];
    const int left = int(n - i < 8 ? n - i : 8);
    load8(gz + i, 0, left, vec, u);
    if constexpr (MOM) {
      load8(mz + i, 0, left, vec, m);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m[k] = mu * m[k] + u[k];
        u[k] = nesterov ? u[k] + mu * m[k] : m[k];
      }
      if (vec) {
        reinterpret_cast<uint4*>(mz + i)[0] = pack16(m, float{});
        reinterpret_cast<uint4*>(mz + i)[1] = pack16(m + 4, float{});
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < left) mz[i + k] = m[k];
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) s += double(u[k]) * double(u[k]);
  }
  for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d, 64);
  __shared__ double w[kThreads / 64];
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) part[z * gridDim.x + blockIdx.x] = (w[0] + w[1]) + (w[2] + w[3]);
}

// X_0 = U / (|U| + eps), scaled, into the padded working matrices: X [rp, cp] and, since the
// products take every operand along K, X transposed [cp, rp].  lo and tlo (each may be NULL)
// receive what the rounding of hi left.  The padding is zero.  A block turns a tile of
// 64 x 64 in LDS, whose rows are an odd number of words, so reading down a column passes over
// the banks.  Bound by HBM (128 x 768 x 2048 in bfloat16, four working matrices written: 375
// us, 5.4 TB/s).
template <typename T, typename W, bool MOM>
__global__ __launch_bounds__(kThreads) void start_kernel(const T* __restrict__ g, const float* __restrict__ mom, float mu,
                                                         int nesterov, int rows, int cols, int rp, int cp,
                                                         const double* __restrict__ part, int nblk, float eps,
                                                         W* __restrict__ hi, W* __restrict__ lo, W* __restrict__ thi,
                                                         W* __restrict__ tlo) {
  constexpr bool kSplit = sizeof(W) == 2;
  constexpr int kLd = kSplit ? 66 : 65;
  __shared__ W th[64 * kLd], tl[kSplit ? 64 * kLd : 1];
  __shared__ double total;
  const size_t z = blockIdx.z;
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  const size_t n = size_t(rows) * cols, np = size_t(rp) * cp;
  const bool vec = cols % 8 == 0;
  float u[2][8] = {};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = r0 + 32 * h + threadIdx.x / 8, c = c0 + threadIdx.x % 8 * 8;
    if (r < rows && c < cols) {
      load8(g + z * n + size_t(r) * cols, c, cols, vec, u[h]);
      if constexpr (MOM) {
        float m[8];
        load8(mom + z * n + size_t(r) * cols, c, cols, vec, m);
#pragma unroll
        for (int k = 0; k < 8; ++k) u[h][k] = nesterov ? u[h][k] + mu * m[k] : m[k];
      }
    }
  }
  if (threadIdx.x < 64) {
    double s = 0.0;
    for (int i = threadIdx.x; i < nblk; i += 64) s += part[z * nblk + i];
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d, 64);
    if (threadIdx.x == 0) total = s;
  }
  __syncthreads();
  const double norm = sqrt(total) + double(eps);
  const double inv = norm > 0.0 ? double(1 << Scale<W>::x) / norm : (norm == 0.0 ? 0.0 : norm);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = 32 * h + threadIdx.x / 8, c = threadIdx.x % 8 * 8;
    Vec8<W> vh, vl;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = float(double(u[h][k]) * inv);
      vh.e[k] = W(x);
      vl.e[k] = W(x - float(vh.e[k]));
      th[r * kLd + c + k] = vh.e[k];
      if constexpr (kSplit) tl[r * kLd + c + k] = vl.e[k];
    }
    const size_t at = z * np + size_t(r0 + r) * cp + c0 + c;
    *reinterpret_cast<Vec8<W>*>(hi + at) = vh;
    if (kSplit && lo != nullptr) *reinterpret_cast<Vec8<W>*>(lo + at) = vl;
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = 32 * h + threadIdx.x / 8, r = threadIdx.x % 8 * 8;
    Vec8<W> vh, vl;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      vh.e[k] = th[(r + k) * kLd + c];
      if constexpr (kSplit) vl.e[k] = tl[(r + k) * kLd + c];
    }
    const size_t at = z * np + size_t(c0 + c) * rp + r0 + r;
    *reinterpret_cast<Vec8<W>*>(thi + at) = vh;
    if (kSplit && tlo != nullptr) *reinterpret_cast<Vec8<W>*>(tlo + at) = vl;
  }
}

// ---- products ------------------------------------------------------------------------
// An m x m matrix of the stack, scaled; P and Q with the diagonal in float32 and zero in o.
template <typename W> struct Sym {
  W* o;
  float* d;
};

// One product for every matrix of the stack, sum = A B (+ A2 B2), and what is made of it.
struct Product {
  const void* a;      // element (m, k) at a[m * lda + k]
  const void* b;      // element (n, k) at b[n * ldb + k]
  const void* a2;     // the second pair of operands (NULL: none)
  const void* b2;
  void* c;
  void* ct;           // C transposed (kApply)
  void* c2;           // what C's rounding leaves, and that transposed (kApply; or NULL)
  void* ct2;
  int ldct;
  size_t sa, sb, sc;  // elements from one matrix of the stack to the next
  int m, n, k, lda, ldb, ldc;
  float alpha;
  // kGram .. kJoin: C is symmetric, its upper tiles are formed and mirrored.
  //   kGram  C = alpha sum
  //   kPoly  C = alpha sum + g V, with k0 I
  //   kNext  C = alpha sum + g D_u V
  //   kJoin  C = alpha sum + g D_u V + h U D_v, with D_u D_v
  // kPoly and kJoin put the diagonal into dc (times unit) and leave C's zero.
  const void* u;
  const void* v;
  const float* du;
  const float* dv;
  float* dc;
  float g, h, k0, unit;
  // kApply and the last product: C = alpha sum + beta d (x + x2), d by row, or by column
  const void* x;
  const void* x2;
  const float* dq;
  float beta;
  int dq_col;
  int mp;             // elements from one matrix's diagonal to the next
  // the last product: the result, or the step on the weight
  void* out;
  float* master;
  int rows, cols;
  float keep, step;   // W = keep W - step C
};

enum Kind { kGram = 0, kPoly = 1, kNext = 2, kJoin = 3, kApply = 4, kResult = 5, kUpdate = 6 };

// Eight k values of 32 rows of each operand: one MFMA 32x32x16, or eight 32x32x2.
template <typename W> struct Mma;
template <> struct Mma<f16_t> {
  static constexpr int kVec = 1;  // 16-byte vectors of a lane's 8 k values
  __device__ static void mma(const u32x4_t* a, const u32x4_t* b, f32x16_t& c) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a[0]), __builtin_bit_cast(f16x8_t, b[0]), c,
                                               0, 0, 0);
  }
};
template <> struct Mma<float> {
  static constexpr int kVec = 2;
  __device__ static void mma(const u32x4_t* a, const u32x4_t* b, f32x16_t& c) {
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[v][k]), __uint_as_float(b[v][k]), c, 0, 0, 0);
  }
};

// ---- epilogues.  The products are formed as (B rows) x (A rows), so lane l holds row l % 32
// of a 32x32 block and register 4q + u its column 8q + 4 (l / 32) + u: four neighbouring
// columns at a time.  Sides of the working matrices are multiples of 64, so four columns, or
// eight, are inside a matrix or outside as a whole.
template <typename W> struct alignas(4 * sizeof(W)) Vec4 {
  W e[4];
};
template <typename W>
__device__ __forceinline__ void load4(const void* base, size_t at, float* f) {
  const Vec4<W> v = *reinterpret_cast<const Vec4<W>*>(static_cast<const W*>(base) + at);
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = float(v.e[k]);
}

// Four columns of the last product into the user's result or weight.
template <typename T, int KIND>
__device__ __forceinline__ void put_last(const Product& p, size_t z, int row, int col, const float* v) {
  if (row >= p.rows) return;
  const size_t at = z * p.rows * p.cols + size_t(row) * p.cols + col;
  T* o = static_cast<T*>(p.out) + at;
  if (p.cols % 4 == 0) {
    if (col >= p.cols) return;
    float w[4];
    if constexpr (KIND == kUpdate) {
      if (p.master != nullptr) {
        load4<float>(p.master, at, w);
      } else {
        const Vec4<T> b = *reinterpret_cast<const Vec4<T>*>(o);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = Elem<T>::to_f32(b.e[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = w[k] * p.keep - v[k] * p.step;
      if (p.master != nullptr) *reinterpret_cast<Vec4<float>*>(p.master + at) = Vec4<float>{w[0], w[1], w[2], w[3]};
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = v[k];
    }
    Vec4<T> r;
#pragma unroll
    for (int k = 0; k < 4; ++k) r.e[k] = Elem<T>::from_f32(w[k]);
    *reinterpret_cast<Vec4<T>*>(o) = r;
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (col + k >= p.cols) break;
    float w = v[k];
    if constexpr (KIND == kUpdate) {
      w = (p.master != nullptr ? p.master[at + k] : Elem<T>::to_f32(o[k])) * p.keep - w * p.step;
      if (p.master != nullptr) p.master[at + k] = w;
    }
    o[k] = Elem<T>::from_f32(w);
  }
}

// A tile of R x C in LDS, rows of RS bytes, into c at (row0, n0) of an m x n matrix, by
// 16-byte pieces; threads t of N.
template <typename W, int R, int C, int RS, int N>
__device__ __forceinline__ void store_tile(const char* lds, W* c, int ldc, int m, int n, int row0, int n0, int t) {
  constexpr int kEl = 16 / int(sizeof(W)), kPieces = C / kEl;
#pragma unroll
  for (int k = 0; k < (R * kPieces + N - 1) / N; ++k) {
    const int id = t + k * N, r = id / kPieces, e = (id % kPieces) * kEl;
    if (R * kPieces % N != 0 && id >= R * kPieces) break;
    if (row0 + r < m && n0 + e < n)
      *reinterpret_cast<u32x4_t*>(c + size_t(row0 + r) * ldc + n0 + e) =
          *reinterpret_cast<const u32x4_t*>(lds + r * RS + e * int(sizeof(W)));
  }
}

// The same tile transposed: its columns as rows n0 + .. of an n x m matrix.  float16: by the
// transposing LDS reads, 16 columns x 32 rows a wave and turn (lane group G rows 8 G .., lane i
// of a group column i).  float32: 16 columns x 16 rows, four rows a lane.  RS is chosen so that
// a read's rows lie in different banks.
template <typename W, int R, int C, int RS, int N>
__device__ __forceinline__ void store_tile_turned(const char* lds, W* c, int ldc, int m, int n, int row0, int n0, int t) {
  const int lane = t & 63, G = lane >> 4, il = lane & 15;
  constexpr int kRows = sizeof(W) == 2 ? 32 : 16, kTurns = (R / kRows) * (C / 16);
#pragma unroll
  for (int k = 0; k < (kTurns + N / 64 - 1) / (N / 64); ++k) {
    const int u = (t >> 6) + k * (N / 64);
    if (kTurns % (N / 64) != 0 && u >= kTurns) break;
    const int r0 = (u % (R / kRows)) * kRows + G * (kRows / 4), c0 = (u / (R / kRows)) * 16;
    u32x4_t v;
    if constexpr (sizeof(W) == 2) {
      const char* src = lds + (r0 + (il >> 2)) * RS + (c0 + 4 * (il & 3)) * 2;
      v = __builtin_bit_cast(u32x4_t, read_kn_frag2(src, src + 4 * RS));
    } else {
      const char* src = lds + r0 * RS + (c0 + il) * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const uint32_t*>(src + e * RS);
    }
    if (n0 + c0 + il < n && row0 + r0 < m) *reinterpret_cast<u32x4_t*>(c + size_t(n0 + c0 + il) * ldc + row0 + r0) = v;
  }
}

// ---- which tile a block forms.  Blocks that run at once on an XCD get consecutive tile
// numbers, so that its L2 holds the rows they share; the numbers run over (matrix, group of
// four n-tiles, m-tile, n-tile in the group), a symmetric product's over m <= n.
constexpr int kGroup = 4;

__host__ __device__ inline int sym_tiles(int t) { return t * (t + 1) / 2; }

// t / d by the high half of t * (2^64 / d + 1), exact below 2^31.  The compiler's division
// takes a block some hundred dependent instructions before its first load.
struct Divisor {
  uint64_t m;  // 0: d is 1
  Divisor() = default;
  explicit Divisor(int d) : m(d == 1 ? 0 : ~uint64_t(0) / uint64_t(d) + 1) {}
  __device__ __forceinline__ int operator()(int t) const { return m == 0 ? t : int(__umul64hi(uint64_t(t), m)); }
};

// t / w, w = 1, 2, 3 or 4
__device__ __forceinline__ int over_group(int t, int w) {
  return w == 3 ? int(__umulhi(unsigned(t), 0xAAAAAAABu) >> 1) : t >> (w >> 1);
}

struct TileMap {
  int MT, NT;  // m-tiles and n-tiles of a matrix
  int each;    // tiles of a matrix
  int per;     // tiles of an XCD
  int total;
  Divisor by_each, by_group;
  unsigned blocks() const { return unsigned(per) * big::kXcds; }
};

template <bool SYM>
TileMap tile_map(int m, int n, int bm, int bn, int count) {
  TileMap t;
  t.MT = (m + bm - 1) / bm;
  t.NT = (n + bn - 1) / bn;
  t.each = SYM ? sym_tiles(t.NT) : t.MT * t.NT;
  t.total = count * t.each;
  t.per = (t.total + big::kXcds - 1) / big::kXcds;
  t.by_each = Divisor(t.each);
  t.by_group = Divisor(t.MT * kGroup);
  return t;
}

// this block's matrix and tile; false: it has none
template <bool SYM>
__device__ __forceinline__ bool tile_of_block(const TileMap& map, size_t& z, int& tm, int& tn) {
  int t = int(blockIdx.x % big::kXcds) * map.per + int(blockIdx.x / big::kXcds);
  if (t >= map.total) return false;
  const int matrix = map.by_each(t);
  z = matrix;
  t -= matrix * map.each;
  if constexpr (SYM) {
    for (int g = 0;; ++g) {
      // the group's n-tiles 4g .. 4g + w - 1 have 4g + 1, .., 4g + w m-tiles
      const int w = min(kGroup, map.NT - g * kGroup), n = w * g * kGroup + sym_tiles(w);
      if (t >= n) {
        t -= n;
        continue;
      }
      if (t < w * g * kGroup) {
        tm = over_group(t, w);
        tn = g * kGroup + t - tm * w;
      } else {
        t -= w * g * kGroup;
        int r = 0;
        while (t >= w - r) t -= w - r++;  // rows of the triangle: w, w - 1, .. tiles
        tm = g * kGroup + r;
        tn = tm + t;
      }
      return true;
    }
  } else {
    const int g = map.by_group(t), w = min(kGroup, map.NT - g * kGroup);
    t -= g * map.MT * kGroup;
    tm = over_group(t, w);
    tn = g * kGroup + t - tm * w;
    return true;
  }
}

// Tiles of 64 x 64, four waves 2 x 2 of 32 x 32.  A stage is 128 bytes of k of the tile's A
// and B rows, filled by direct global->LDS loads (1 KB: eight rows) kSlots - 1 stages ahead,
// one barrier a stage.  16-byte piece c of row r sits at piece c ^ (r / 2 % 8), so the reads
// of 16 rows at one piece cover all banks.  KS > 1 (too few tiles for the card): KS groups of
// four waves take a range of K each, with a ring of its own; their sums are added in the order
// of the ranges, a share of the registers by each group.
//
// What bounds it: in float32 the MFMAs (32 matrices of 1024 x 1024, five steps: 5.6 ms, 126
// TFLOP/s).  Their stages are long, so two slots do, and five blocks a CU hide one another's
// barriers and epilogues: three and four slots took 9% longer, 128 x 128 tiles 10%.
template <typename W, int KS>
struct Ring {
  static constexpr int kStage = 2 * kPad * 128, kSlots = sizeof(W) == 4 || KS == 4 ? 2 : (KS == 2 ? 3 : 4);
  static constexpr int kRow = kPad * int(sizeof(W)) + (sizeof(W) == 2 ? 32 : 16);  // of the tile in LDS
  static constexpr int kPerWave = kStage / 1024 / 4, kLds = KS * kSlots * kStage;
  static_assert(kPad * kRow <= kLds, "the tile fits");
  static_assert(KS == 1 || KS * 16 * 256 * 4 <= kLds, "the groups' sums fit");
};

template <typename W, typename T, int KS, int KIND>
__device__ __forceinline__ void product_body(const Product& p, const TileMap& map, char* lds0) {
  using R = Ring<W, KS>;
  constexpr bool kSym = KIND <= kJoin;
  constexpr int kBytes = int(sizeof(W));
  size_t z;
  int tm, tn;
  if (!tile_of_block<kSym>(map, z, tm, tn)) return;
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) & 3), lane = threadIdx.x & 63;
  const int group = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  char* lds = lds0 + group * R::kSlots * R::kStage;
  // of a group, waves 0 and 1 load A rows, 2 and 3 B rows; rows past the matrix repeat its last one
  const bool is_a = wave < 2;
  const int ld = is_a ? p.lda : p.ldb, rows = is_a ? p.m : p.n;
  const size_t off = z * (is_a ? p.sa : p.sb);
  const uint32_t bytes = uint32_t(rows) * uint32_t(ld) * kBytes;
  const W* first = static_cast<const W*>(is_a ? p.a : p.b) + off;
  const W* second = p.a2 != nullptr ? static_cast<const W*>(is_a ? p.a2 : p.b2) + off : first;
  const __amdgpu_buffer_rsrc_t r0 = __builtin_amdgcn_make_buffer_rsrc(const_cast<W*>(first), 0, bytes, kRsrcFlags);
  const __amdgpu_buffer_rsrc_t r1 = __builtin_amdgcn_make_buffer_rsrc(const_cast<W*>(second), 0, bytes, kRsrcFlags);
  uint32_t vo[R::kPerWave];
#pragma unroll
  for (int j = 0; j < R::kPerWave; ++j) {
    const int r = (wave & 1) * 32 + 8 * j + (lane >> 3);  // row of the operand's part of the stage
    const int row = min((is_a ? tm : tn) * kPad + r, rows - 1);
    vo[j] = uint32_t(row) * uint32_t(ld) * kBytes + uint32_t(((lane & 7) ^ ((r >> 1) & 7)) * 16);
  }
  const int slices = p.k * kBytes / 128, total = p.a2 != nullptr ? 2 * slices : slices;
  const int turns = (total + KS - 1) / KS;            // this group's stages: mine from `from` on
  const int from = group * turns, mine = min(turns, total - from);
  auto issue = [&](int s) {  // the group's stage s, or the last one there is, into its slot
    const int st = min(from + s, total - 1);
    char* slot = lds + (s % R::kSlots) * R::kStage + R::kPerWave * wave * 1024;
    const uint32_t ko = uint32_t(st >= slices ? st - slices : st) * 128u;
#pragma unroll
    for (int j = 0; j < R::kPerWave; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(st >= slices ? r1 : r0, (lds_ptr_t)(slot + j * 1024), 16, vo[j], ko, 0, 0);
  };
  f32x16_t acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.f;
  const int sw = ((lane & 31) >> 1) & 7, ao = (wm + (lane & 31)) * 128, bo = (kPad + wn + (lane & 31)) * 128;
  constexpr int kVec = Mma<W>::kVec;
  for (int s = 0; s < R::kSlots - 1; ++s) issue(s);
  for (int s = 0; s < turns; ++s) {
    MOE_VMCNT(R::kPerWave * (R::kSlots - 2));  // this wave's loads of stage s have landed
    MOE_LGKMCNT0();                            // and its reads of stage s - 1
    block_barrier();                           // every wave's have
    issue(s + R::kSlots - 1);                  // into the slot stage s - 1 used
    if (KS > 1 && s >= mine) continue;         // the last range may be short
    const char* st = lds + (s % R::kSlots) * R::kStage;
#pragma unroll
    for (int kc = 0; kc < 8 / (2 * kVec); ++kc) {
      u32x4_t fa[kVec], fb[kVec];
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        const int c = (((2 * kc + (lane >> 5)) * kVec + v) ^ sw) * 16;
        fa[v] = *reinterpret_cast<const u32x4_t*>(st + ao + c);
        fb[v] = *reinterpret_cast<const u32x4_t*>(st + bo + c);
      }
      Mma<W>::mma(fb, fa, acc);
    }
  }
  MOE_VMCNT(0);  // the ring's last (repeated) loads land before the LDS is used again, or the block ends
  constexpr int kRegs = 16 / KS;  // of each accumulator, this thread's share of the epilogue
  if constexpr (KS > 1) {
    __syncthreads();
    float* sums = reinterpret_cast<float*>(lds0);
    const int t = threadIdx.x & 255;
#pragma unroll
    for (int r = 0; r < 16; ++r) sums[(group * 16 + r) * 256 + t] = acc[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRegs; ++r) {
      float v = 0.f;
#pragma unroll
      for (int g = 0; g < KS; ++g) v += sums[(g * 16 + group * kRegs + r) * 256 + t];
      acc[r] = v;
    }
  }
  __syncthreads();  // the LDS is read out
  const int row0 = tm * kPad, n0 = tn * kPad;
  constexpr int RS = R::kRow;
  const float* du = p.du + z * p.mp;
  const float* dv = p.dv + z * p.mp;
  const float* dq = p.dq + z * p.mp;
  f32x4_t low[kRegs / 4];
#pragma unroll
  for (int qq = 0; qq < kRegs / 4; ++qq) {
    const int rt = wm + (lane & 31), ct = wn + 8 * (group * (kRegs / 4) + qq) + 4 * (lane >> 5);
    const int row = row0 + rt, col = n0 + ct;
    const size_t ci = z * p.sc + size_t(row) * p.ldc + col;
    float v[4], f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = p.alpha * acc[4 * qq + e];
    if constexpr (kSym) {
      if constexpr (KIND != kGram) {
        load4<W>(p.v, ci, f);
        const float by = KIND == kPoly ? p.g : p.g * du[row];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += by * f[e];
      }
      if constexpr (KIND == kJoin) {
        load4<W>(p.u, ci, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += p.h * dv[col + e] * f[e];
      }
      if constexpr (KIND == kPoly || KIND == kJoin) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (row == col + e) {
            p.dc[z * p.mp + row] = v[e] * p.unit + (KIND == kPoly ? p.k0 : du[row] * dv[row]);
            v[e] = 0.f;
          }
      }
    } else {
      load4<W>(p.x, ci, f);
      if (p.x2 != nullptr) {
        float f2[4];
        load4<W>(p.x2, ci, f2);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] += f2[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += p.beta * dq[p.dq_col ? col + e : row] * f[e];
    }
    if constexpr (KIND == kResult || KIND == kUpdate) {
      put_last<T, KIND>(p, z, row, col, v);
    } else {
      Vec4<W> h;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h.e[e] = W(v[e]);
        if constexpr (KIND == kApply && kBytes == 2) low[qq][e] = v[e] - float(h.e[e]);
      }
      *reinterpret_cast<Vec4<W>*>(lds0 + rt * RS + ct * kBytes) = h;
    }
  }
  if constexpr (KIND != kResult && KIND != kUpdate) {
    constexpr int kAll = kThreads * KS;
    __syncthreads();
    W* c = static_cast<W*>(p.c) + z * p.sc;
    store_tile<W, kPad, kPad, RS, kAll>(lds0, c, p.ldc, p.m, p.n, row0, n0, threadIdx.x);
    if (kSym && tm != tn)
      store_tile_turned<W, kPad, kPad, RS, kAll>(lds0, c, p.ldc, p.m, p.n, row0, n0, threadIdx.x);
    if constexpr (KIND == kApply) {
      store_tile_turned<W, kPad, kPad, RS, kAll>(lds0, static_cast<W*>(p.ct) + z * p.sc, p.ldct, p.m, p.n, row0, n0,
                                             threadIdx.x);
      if (kBytes == 2 && p.c2 != nullptr) {  // the low halves, through the same tile
        __syncthreads();
#pragma unroll
        for (int qq = 0; qq < kRegs / 4; ++qq) {
          const int rt = wm + (lane & 31), ct = wn + 8 * (group * (kRegs / 4) + qq) + 4 * (lane >> 5);
          Vec4<W> l;
#pragma unroll
          for (int e = 0; e < 4; ++e) l.e[e] = W(low[qq][e]);
          *reinterpret_cast<Vec4<W>*>(lds0 + rt * RS + ct * kBytes) = l;
        }
        __syncthreads();
        store_tile<W, kPad, kPad, RS, kAll>(lds0, static_cast<W*>(p.c2) + z * p.sc, p.ldc, p.m, p.n, row0, n0, threadIdx.x);
        if (p.ct2 != nullptr)
          store_tile_turned<W, kPad, kPad, RS, kAll>(lds0, static_cast<W*>(p.ct2) + z * p.sc, p.ldct, p.m, p.n, row0, n0,
                                                 threadIdx.x);
      }
    }
  }
}

template <typename W, typename T, int KS, int KIND>
__global__ __launch_bounds__(kThreads * KS) void product_kernel(Product p, TileMap map) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  product_body<W, T, KS, KIND>(p, map, lds);
}

template <typename W, typename T, int KS, int KIND>
moe_status launch_ring(const char* name, const Product& p, int count, hipStream_t s) {
  auto kern = product_kernel<W, T, KS, KIND>;
  constexpr int lds = Ring<W, KS>::kLds;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return set_error(MOE_ERR_HIP, "%s: LDS attribute: %s", name, hipGetErrorString(e));
  const TileMap map = tile_map<KIND <= kJoin>(p.m, p.n, kPad, kPad, count);
  MOE_LAUNCH(name, kern, dim3(map.blocks()), dim3(kThreads * KS), lds, s, p, map);
  return MOE_OK;
}

// ---- the same on the large tile (float16) ----------------------------------------------
// 256 x 256 tiles of big_tile.h, both operands along K (with one of them the other way round,
// through the transposing LDS reads, a step of 64 k took 2.25 us against 1.69, with both 3.1).
// What bounds it: the MFMAs, and per tile some 20 us of prologue, epilogue and matrices read
// back, beside 1.69 us a step (16 matrices of 2880 x 2880, a product of two: 461 to 490 us, 830 to
// 780 TFLOP/s of the half that is computed; 128 of 768 x 768, 12 steps a tile: 120, 480).
// The accumulators hold four neighbouring columns of one row at a time, so the epilogue reads what it adds eight bytes a lane, turns the tile to
// float16 in LDS and writes whole row pieces; a symmetric product's tile off the diagonal
// is written a second time, its columns read back as rows by the transposing LDS reads.
// Rows of the LDS tile are 32 bytes longer than the tile: the four rows that such a read
// takes from lie in different banks.
namespace nsbig {

using big::BK;
using big::BM;
using big::BNE;
constexpr int kRS = BNE * 2 + 32;
constexpr size_t kLds = big::kLoopLdsMax > size_t(BM) * kRS ? big::kLoopLdsMax : size_t(BM) * kRS;

__device__ __forceinline__ void unpack4(uint2 w, float* f) {
  typedef _Float16 h4 __attribute__((ext_vector_type(4)));
  const h4 v = __builtin_bit_cast(h4, w);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = float(v[i]);
}
__device__ __forceinline__ uint2 pack4(const float* f) {
  typedef _Float16 h4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(uint2, h4{f16_t(f[0]), f16_t(f[1]), f16_t(f[2]), f16_t(f[3])});
}

// LOW (kApply): what the rounding of C leaves waits in registers and goes out through the same
// LDS tile.
template <int NW, int KIND, bool LOW>
__global__ __launch_bounds__(NW * 64) void tile_kernel(Product p, TileMap map) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  using S = big::Shape<false, NW>;
  constexpr int NB = S::NB, kThr = NW * 64;
  constexpr bool kSym = KIND <= kJoin;
  size_t z;
  int tm, tn;
  if (!tile_of_block<kSym>(map, z, tm, tn)) return;
  const int row0 = tm * BM, n0 = tn * BNE;

  big::Operands op;
  op.A = static_cast<const uint16_t*>(p.a) + z * p.sa;
  op.A2 = static_cast<const uint16_t*>(p.a2 != nullptr ? p.a2 : p.a) + z * p.sa;
  op.a_rows = p.m;
  op.lda = p.lda;
  op.Bg = static_cast<const uint16_t*>(p.b) + z * p.sb;
  op.Bu = static_cast<const uint16_t*>(p.b2 != nullptr ? p.b2 : p.b) + z * p.sb;
  op.b_rows = p.n;
  op.ldb = p.ldb;
  const int nk = p.k / BK;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int wm = S::wm(wave), wn = S::wn(wave), fr = lane & 31, g4 = lane >> 5;
  const float* du = p.du + z * p.mp;
  const float* dv = p.dv + z * p.mp;
  const float* dq = p.dq + z * p.mp;

  const auto epi = [&](f32x16_t (&acc)[4][NB]) {
    MOE_LGKMCNT0();
    block_barrier();  // every wave is done reading the last stage
    // what the epilogue adds, by buffer loads: rows past the matrix read as zero, so no load
    // hangs on a branch and many are in flight
    const auto rsrc = [&](const void* x) {
      return __builtin_amdgcn_make_buffer_rsrc(const_cast<f16_t*>(static_cast<const f16_t*>(x) + z * p.sc), 0,
                                               uint32_t(p.m) * uint32_t(p.ldc) * 2u, kRsrcFlags);
    };
    const __amdgpu_buffer_rsrc_t r0 = rsrc(kSym ? p.v : p.x);
    const __amdgpu_buffer_rsrc_t r1 = rsrc(kSym ? p.u : p.x2);
    const bool two = KIND == kJoin || (!kSym && p.x2 != nullptr);
    uint2 low[LOW ? 4 : 1][NB][4];
    f32x4_t dc4[NB][4];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = min(n0 + wn * NB * 32 + j * 32 + 8 * q + 4 * g4, p.n - 4);
        dc4[j][q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if constexpr (KIND == kJoin) dc4[j][q] = *reinterpret_cast<const f32x4_t*>(dv + col);
        if constexpr (!kSym)
          if (p.dq_col) dc4[j][q] = *reinterpret_cast<const f32x4_t*>(dq + col);
      }
    // a row block at a time: its loads take whole lines of 32 rows, piece after piece
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int rt = wm * 128 + i * 32 + fr, row = row0 + rt;
      const int rowc = min(row, p.m - 1);
      const float dri = KIND == kNext || KIND == kJoin ? du[rowc] : (!kSym && !p.dq_col ? dq[rowc] : 0.f);
      uint2 l0[NB][4], l1[NB][4];
      if constexpr (KIND != kGram) {
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int col = n0 + wn * NB * 32 + j * 32 + 8 * q + 4 * g4;
            const uint32_t off = (uint32_t(row) * uint32_t(p.ldc) + uint32_t(col)) * 2u;
            l0[j][q] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r0, off, 0, 0));
            l1[j][q] = make_uint2(0u, 0u);
            if (two) l1[j][q] = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r1, off, 0, 0));
          }
      }
#pragma unroll
      for (int j = 0; j < NB; ++j) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int cl = wn * NB * 32 + j * 32 + 8 * q + 4 * g4, col = n0 + cl;
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = p.alpha * acc[i][j][4 * q + e];
          if constexpr (KIND != kGram) {
            float f0[4], f1[4];
            unpack4(l0[j][q], f0);
            unpack4(l1[j][q], f1);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (KIND == kPoly) v[e] += p.g * f0[e];
              if constexpr (KIND == kNext) v[e] += p.g * dri * f0[e];
              if constexpr (KIND == kJoin) v[e] += p.g * dri * f0[e] + p.h * dc4[j][q][e] * f1[e];
              if constexpr (!kSym) v[e] += p.beta * (p.dq_col ? dc4[j][q][e] : dri) * (f0[e] + f1[e]);
            }
          }
          if constexpr (KIND == kPoly || KIND == kJoin) {
            if (tm == tn && unsigned(row - col) < 4u && row < p.m) {
              const int e = row - col;
              float d = 0.f;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (k == e) {
                  d = v[k];
                  v[k] = 0.f;
                }
              p.dc[z * p.mp + row] = d * p.unit + (KIND == kPoly ? p.k0 : dri * dv[row]);
            }
          }
          if constexpr (KIND == kUpdate) {
            put_last<bf16_t, KIND>(p, z, row, col, v);
          } else if constexpr (KIND == kResult) {
            *reinterpret_cast<uint2*>(lds + rt * kRS + cl * 2) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
          } else {
            *reinterpret_cast<uint2*>(lds + rt * kRS + cl * 2) = pack4(v);
            if constexpr (LOW) {
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] -= float(f16_t(v[e]));
              low[i][j][q] = pack4(v);
              asm volatile("" : "+v"(low[i][j][q].x), "+v"(low[i][j][q].y));  // here, not where it is stored: registers
            }
          }
        }
      }
    }
    if constexpr (KIND == kUpdate) return;
    MOE_LGKMCNT0();
    block_barrier();
    constexpr int kPieces = BNE / 8;
    if constexpr (KIND == kResult) {
      const int rows = p.rows - row0, cols = p.cols - n0;
      bf16_t* o = static_cast<bf16_t*>(p.out) + z * p.rows * p.cols + size_t(row0) * p.cols + n0;
#pragma unroll
      for (int k = 0; k < BM * kPieces / kThr; ++k) {
        const int id = tid + k * kThr, r = id / kPieces, c = (id % kPieces) * 8;
        if (r >= rows || c >= cols) continue;
        const char* src = lds + r * kRS + c * 2;
        if (p.cols % 8 == 0) {
          *reinterpret_cast<u32x4_t*>(o + size_t(r) * p.cols + c) = *reinterpret_cast<const u32x4_t*>(src);
        } else {
          for (int e = 0; e < 8 && c + e < cols; ++e)
            o[size_t(r) * p.cols + c + e] = reinterpret_cast<const bf16_t*>(src)[e];
        }
      }
    } else {
      f16_t* c = static_cast<f16_t*>(p.c) + z * p.sc;
      store_tile<f16_t, BM, BNE, kRS, kThr>(lds, c, p.ldc, p.m, p.n, row0, n0, tid);
      if (kSym ? tm != tn : p.ct != nullptr)
        store_tile_turned<f16_t, BM, BNE, kRS, kThr>(lds, kSym ? c : static_cast<f16_t*>(p.ct) + z * p.sc,
                                                     kSym ? p.ldc : p.ldct, p.m, p.n, row0, n0, tid);
      if constexpr (LOW) {
        MOE_LGKMCNT0();
        block_barrier();  // the high halves are read out
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int rt = wm * 128 + i * 32 + fr, cl = wn * NB * 32 + j * 32 + 8 * q + 4 * g4;
              *reinterpret_cast<uint2*>(lds + rt * kRS + cl * 2) = low[i][j][q];
            }
        MOE_LGKMCNT0();
        block_barrier();
        store_tile<f16_t, BM, BNE, kRS, kThr>(lds, static_cast<f16_t*>(p.c2) + z * p.sc, p.ldc, p.m, p.n, row0, n0, tid);
        if (p.ct2 != nullptr)
          store_tile_turned<f16_t, BM, BNE, kRS, kThr>(lds, static_cast<f16_t*>(p.ct2) + z * p.sc, p.ldct, p.m, p.n, row0,
                                                       n0, tid);
      }
    }
  };
  big::tile_loop<1, false, NW, false, false, big::F16, true>(op, p.n, nk, row0, n0, 0, p.a2 != nullptr ? 2 * nk : nk, lds, epi);
}

template <int NW, int KIND, bool LOW>
moe_status launch_nw(const char* name, const Product& p, int count, hipStream_t s) {
  auto kern = tile_kernel<NW, KIND, LOW>;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, int(kLds));
  if (e != hipSuccess) return set_error(MOE_ERR_HIP, "%s: LDS attribute: %s", name, hipGetErrorString(e));
  const TileMap map = tile_map<KIND <= kJoin>(p.m, p.n, BM, BNE, count);
  MOE_LAUNCH(name, kern, dim3(map.blocks()), dim3(NW * 64), kLds, s, p, map);
  return MOE_OK;
}

// Four waves from 64 steps of k on, eight below, as for the grouped products (K = 4096 and
// 14336: four are 2.7% faster; K = 768: 6% slower).
template <int KIND>
moe_status launch(const char* name, const Product& p, int count, hipStream_t s) {
  const bool four = p.k / BK >= 64;
  if constexpr (KIND == kApply) {
    if (p.c2 != nullptr)
      return four ? launch_nw<4, KIND, true>(name, p, count, s) : launch_nw<8, KIND, true>(name, p, count, s);
  }
  return four ? launch_nw<4, KIND, false>(name, p, count, s) : launch_nw<8, KIND, false>(name, p, count, s);
}

}  // namespace nsbig

// float16 phases: large tiles or small ones.  A round of large tiles on 256 CUs takes as long
// as some 1800 small ones (fitted to 18 stacks timed on both: 2 matrices of 2000 x 2000, 1056
// and 2048 small tiles a product, 943 us on large tiles and 844 on small ones; 4 of them 1073
// and 1555; 128 of 300 x 300, two rounds that are mostly padding, 782 and 528).
// Small tiles too few for the CUs split K over groups of waves: four while there is a CU for
// each tile, two while there are two tiles, and every group has two stages.
constexpr int kRound = 1800;
template <typename W, typename T, int KIND>
moe_status launch_product(const char* name, const Product& p, bool phases, int count, hipStream_t s) {
  const auto tiles = [&](int bt) {
    const int64_t m = (p.m + bt - 1) / bt, n = (p.n + bt - 1) / bt;
    return (KIND <= kJoin ? m * (m + 1) / 2 : m * n) * count;
  };
  if constexpr (sizeof(W) == 2) {
    if (phases && tiles(64) >= kRound * ((tiles(256) + 255) / 256)) return nsbig::launch<KIND>(name, p, count, s);
  }
  const int stages = p.k * int(sizeof(W)) / 128 * (p.a2 != nullptr ? 2 : 1);
  if (tiles(64) <= 256 && stages >= 8) return launch_ring<W, T, 4, KIND>(name, p, count, s);
  if (tiles(64) <= 512 && stages >= 4) return launch_ring<W, T, 2, KIND>(name, p, count, s);
  return launch_ring<W, T, 1, KIND>(name, p, count, s);
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
  W* xt(int i) const { return reinterpret_cast<W*>(base + p.o_t[i]); }
  Sym<W> q(int i) const {
    return {reinterpret_cast<W*>(base + p.o_q[i]), reinterpret_cast<float*>(base + p.o_d[i])};
  }

  moe_status start() const {
    const int64_t n = int64_t(p.rows) * p.cols;
    const moe_muon_desc* m = a.m;
    const T* g = static_cast<const T*>(a.grad);
    double* part = reinterpret_cast<double*>(base + p.o_part);
    const dim3 gn(unsigned(p.nblk), unsigned(p.count));
    const dim3 gs(unsigned(p.cp / 64), unsigned(p.rp / 64), unsigned(p.count));
    // the low half where the first application takes it as an operand, and in the X layout
    // for its epilogue
    W* lo = kSplit ? x(2) : nullptr;
    W* tlo = kSplit && !p.tall ? xt(2) : nullptr;
    const bool mom = a.momentum != nullptr;
    if (mom) {
      MOE_LAUNCH("muon_momentum", (norm_kernel<T, true>), gn, dim3(kThreads), 0, a.s, g, a.momentum, m->momentum,
                 m->nesterov, n, part);
    } else {
      MOE_LAUNCH("orth_norm", (norm_kernel<T, false>), gn, dim3(kThreads), 0, a.s, g, static_cast<float*>(nullptr), 0.f,
                 0, n, part);
    }
    if (mom) {
      MOE_LAUNCH("muon_start", (start_kernel<T, W, true>), gs, dim3(kThreads), 0, a.s, g, a.momentum, m->momentum,
                 m->nesterov, p.rows, p.cols, p.rp, p.cp, part, p.nblk, m->eps, x(0), lo, xt(0), tlo);
    } else {
      MOE_LAUNCH("orth_start", (start_kernel<T, W, false>), gs, dim3(kThreads), 0, a.s, g,
                 static_cast<const float*>(nullptr), 0.f, 0, p.rows, p.cols, p.rp, p.cp, part, p.nblk, m->eps, x(0), lo,
                 xt(0), tlo);
    }
    return MOE_OK;
  }

  // A = X X^T (or X^T X), X in x(i)
  moe_status gram(int i, Sym<W> out) const {
    Product g{};
    g.a = g.b = p.tall ? xt(i) : x(i);
    g.c = out.o;
    g.sa = g.sb = size_t(p.rp) * p.cp;
    g.sc = size_t(p.mp) * p.mp;
    g.m = g.n = g.ldc = g.mp = p.mp;
    g.k = p.tall ? p.rp : p.cp;
    g.lda = g.ldb = g.k;
    g.alpha = ldexpf(1.f, Scale<W>::a - 2 * Scale<W>::x);
    return launch_product<W, T, kGram>("ns_gram", g, !p.single, p.count, a.s);
  }

  // m x m products of commuting symmetric matrices, their scales 2^su, 2^sv, 2^so
  template <int KIND>
  moe_status square(const char* name, Sym<W> u, int su, Sym<W> v, int sv, Sym<W> out, int so, float factor = 1.f,
                    float linear = 1.f, float k0 = 0.f) const {
    Product g{};
    g.a = g.u = u.o;
    g.b = g.v = v.o;  // symmetric: its columns are its rows
    g.du = u.d;
    g.dv = v.d;
    g.c = out.o;
    g.dc = out.d;
    g.sa = g.sb = g.sc = size_t(p.mp) * p.mp;
    g.m = g.n = g.k = g.lda = g.ldb = g.ldc = g.mp = p.mp;
    g.alpha = ldexpf(factor, so - su - sv);
    g.g = ldexpf(linear, so - sv);
    g.h = ldexpf(1.f, so - su);
    g.k0 = k0;
    g.unit = ldexpf(1.f, -so);
    return launch_product<W, T, KIND>(name, g, !p.single, p.count, a.s);
  }

  // q X (or X q) for X in x(i), with its low half if `split`; into x(to), with its low half if
  // `keep`, or into the user's result (to < 0)
  moe_status apply(Sym<W> q, int i, bool split, int to, bool keep) const {
    Product g{};
    const size_t sq = size_t(p.mp) * p.mp, sx = size_t(p.rp) * p.cp;
    const W* hi = x(i);
    const W* lo = split ? x(i + 2) : nullptr;
    // the low halves first, while the sums are small
    const W* first = p.tall ? (split ? lo : hi) : (split ? xt(i + 2) : xt(i));
    const W* second = !split ? nullptr : (p.tall ? hi : xt(i));
    if (p.tall) {
      g.a = first;
      g.a2 = second;
      g.b = q.o;
      g.b2 = q.o;
      g.sa = sx;
      g.sb = sq;
      g.lda = p.cp;
      g.ldb = p.mp;
    } else {
      g.a = q.o;
      g.a2 = second != nullptr ? q.o : nullptr;
      g.b = first;
      g.b2 = second;
      g.sa = sq;
      g.sb = sx;
      g.lda = p.mp;
      g.ldb = p.rp;
    }
    g.sc = sx;
    g.m = p.rp;
    g.n = g.ldc = p.cp;
    g.k = g.mp = p.mp;
    g.x = hi;
    g.x2 = lo;
    g.dq = q.d;
    g.dq_col = p.tall;
    if (to >= 0) {
      g.c = x(to);
      g.ct = xt(to);
      g.ldct = p.rp;
      if (keep) {
        g.c2 = x(to + 2);
        g.ct2 = p.tall ? nullptr : xt(to + 2);
      }
      g.alpha = ldexpf(1.f, -Scale<W>::q);
      g.beta = 1.f;
      return launch_product<W, T, kApply>("ns_apply", g, !p.single, p.count, a.s);
    }
    g.alpha = ldexpf(1.f, -Scale<W>::q - Scale<W>::x);
    g.beta = ldexpf(1.f, -Scale<W>::x);
    g.out = a.out;
    g.rows = p.rows;
    g.cols = p.cols;
    if (a.momentum == nullptr) return launch_product<W, T, kResult>("ns_apply_result", g, !p.single, p.count, a.s);
    g.master = a.master;
    g.keep = 1.f - a.m->lr * a.m->weight_decay;
    g.step = a.m->lr * a.m->update_scale;
    return launch_product<W, T, kUpdate>("muon_apply", g, !p.single, p.count, a.s);
  }

  moe_status run() const {
    TRY_NS(start());
    constexpr int sa = Scale<W>::a, sq = Scale<W>::q;
    int cur = 0, done = 0;  // X in x(cur), its low half, if it has one, in x(cur + 2)
    bool split = kSplit;
    while (done < a.m->steps) {
      const int len = phase_steps(p.single, done, a.m->steps);
      // A in 0; Q in 1, P in 2 (Q and what it becomes in 1 and 3), and T = P A in 4
      int Q = 1;
      TRY_NS(gram(cur, q(0)));
      for (int k = 0; k < len; ++k) {
        const int P = k == 0 ? Q : 2;
        TRY_NS(square<kPoly>("ns_poly", q(0), sa, q(0), sa, q(P), sq, a.cc, a.cb, a.ca));
        if (k + 1 < len) {
          TRY_NS(square<kNext>("ns_next", q(P), sq, q(0), sa, q(4), sa));
          TRY_NS(square<kNext>("ns_next", q(P), sq, q(4), sa, q(0), sa));
        }
        if (k > 0) {
          const int N = Q == 1 ? 3 : 1;
          TRY_NS(square<kJoin>("ns_join", q(P), sq, q(Q), sq, q(N), sq));
          Q = N;
        }
      }
      done += len;
      const bool last = done == a.m->steps, keep = kSplit && keeps_low(p.single, done, a.m->steps);
      TRY_NS(apply(q(Q), cur, split, last ? -1 : cur ^ 1, keep));
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
