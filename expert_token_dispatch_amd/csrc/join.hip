// The join of a block with the residual stream, and its gradients.
//
// Around the layer stand two norms: one of the block's output before it is added to the
// residual stream, one of the stream before the next block.  With
// n(v; w) = v / sqrt(mean(v^2) + eps) * (offset + w),
//   z = x + scale * g * n(y; w_post)          h = n(z; w_pre)
// where g is a gate per channel, token or element (or its sigmoid), or 1.
//
// Both passes do a few operations per element they move, so they are bound by memory: each
// tensor is read once and written once.  A row's vectors stay in registers from the load to
// the store (one 16-byte vector of a row belongs to one thread throughout), so the two means
// of the forward are two reductions over the row's threads, not passes over memory; outputs
// may overwrite inputs for the same reason.  Every sum is float32, every output is rounded
// once, and h takes z before its rounding.
#include <math.h>

#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

struct JoinP {
  const void* x;
  const void* y;
  const void* gate;
  const void* w_post;
  const void* w_pre;
  void* z;
  void* h;
  int64_t rows;
  int H, nvec;  // row length, in elements and in 16-byte vectors
  int post_norm, gate_kind, gate_act;
  float eps, offset, scale;
};

struct JoinBwdP {
  const void* z;
  const void* y;
  const void* gate;
  const void* w_post;
  const void* w_pre;
  const void* dz;
  const void* dh;
  void* dx;
  void* dy;
  void* dgate;
  float* part;  // [sums][blocks][H]: column sums of each block's rows
  int p_pre, p_post, p_gate;  // which of the sums is whose, -1: not asked for
  int64_t rows;
  int H, nvec;
  int post_norm, gate_kind, gate_act;
  float eps, offset, scale;
};

// The gate's value; float32 layers take the full exponential.
template <typename T>
__device__ __forceinline__ float sigmoid(float v) {
  return 1.0f / (1.0f + (sizeof(T) == 4 ? expf(-v) : __expf(-v)));
}

// The same and its derivative s (1 - s), which is even in v and would cancel if it were formed from an s
// near 1: with e = exp(-|v|), s = 1 / (1 + e) or e / (1 + e), s (1 - s) = e / (1 + e)^2.
struct Sigmoid {
  float s, slope;
};
template <typename T>
__device__ __forceinline__ Sigmoid sigmoid_and_slope(float v) {
  const float e = sizeof(T) == 4 ? expf(-fabsf(v)) : __expf(-fabsf(v)), q = 1.0f / (1.0f + e);
  return {v < 0.0f ? e * q : q, e * q * q};
}

// Sums of N values over the NT threads of a row; every thread gets them.  `buf` alternates
// between two halves, so one barrier per reduction is enough.
template <int NT, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*buf)[NT / 64]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v[n] += __shfl_xor(v[n], d, 64);
  if constexpr (NT > 64) {
    constexpr int W = NT / 64;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if (lane == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) buf[n][wave] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += buf[n][w];
      v[n] = s;
    }
  }
}

template <typename T>
__device__ __forceinline__ uint4 load_vec(const void* p, size_t at) {
  return reinterpret_cast<const uint4*>(p)[at];
}

// 8192 x 4096 in bf16 takes 50 us, 5.3 TB/s, as fast as a large copy; 2047 x 2880 with a gate per
// element 15 us (4 TB/s: the ends of a short kernel).  128 threads of four vectors 53 and 18 us.
// NT threads and V vectors a thread hold a row.  Rows of one wave (NT = 64) go four to a
// block, longer ones take a block each.
template <typename T, int NT, int V>
__global__ __launch_bounds__(NT == 64 ? 256 : NT) void join_kernel(JoinP p) {
  constexpr int E = Elem<T>::kPerVec;
  __shared__ float buf[2][1][NT / 64];
  const int64_t block = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
  const int64_t row = NT == 64 ? block * 4 + (threadIdx.x >> 6) : block;
  if (row >= p.rows) return;  // whole blocks, or waves of one that no barrier follows
  const int tid = NT == 64 ? threadIdx.x & 63 : threadIdx.x;
  const size_t base = size_t(row) * p.nvec;
  const float inv_h = 1.0f / float(p.H);
  const uint4 none = make_uint4(0, 0, 0, 0);
  uint4 xr[V], yr[V], gr[V], wa[V], wb[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = tid + i * NT;
    const bool in = c < p.nvec;
    xr[i] = in ? load_vec<T>(p.x, base + c) : none;
    yr[i] = in && p.y != nullptr ? load_vec<T>(p.y, base + c) : none;
    gr[i] = none;
    if (in && p.gate_kind == MOE_GATE_ELEMENT) gr[i] = load_vec<T>(p.gate, base + c);
    if (in && p.gate_kind == MOE_GATE_CHANNEL) gr[i] = load_vec<T>(p.gate, c);
    wa[i] = in && p.w_post != nullptr ? load_vec<T>(p.w_post, c) : none;
    wb[i] = in && p.w_pre != nullptr ? load_vec<T>(p.w_pre, c) : none;
  }
  float zv[V][E];
#pragma unroll
  for (int i = 0; i < V; ++i) unpack16(xr[i], T(), zv[i]);
  if (p.y != nullptr) {
    float g_row = p.scale;
    if (p.gate_kind == MOE_GATE_TOKEN) {
      const float g = static_cast<const float*>(p.gate)[row];
      g_row *= p.gate_act == MOE_GATE_SIGMOID ? sigmoid<T>(g) : g;
    }
    float r = 1.0f;
    if (p.post_norm) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float f[E];
        unpack16(yr[i], T(), f);
#pragma unroll
        for (int e = 0; e < E; ++e) s[0] = fmaf(f[e], f[e], s[0]);
      }
      row_sum<NT, 1>(s, buf[0]);
      r = 1.0f / sqrtf(s[0] * inv_h + p.eps);
    }
    const bool whole = p.gate_kind == MOE_GATE_ELEMENT || p.gate_kind == MOE_GATE_CHANNEL;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float f[E], w[E], g[E];
      unpack16(yr[i], T(), f);
      unpack16(wa[i], T(), w);
      unpack16(gr[i], T(), g);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float b = f[e] * r;
        if (p.w_post != nullptr) b *= p.offset + w[e];
        float k = g_row;
        if (whole) k *= p.gate_act == MOE_GATE_SIGMOID ? sigmoid<T>(g[e]) : g[e];
        zv[i][e] = fmaf(k, b, zv[i][e]);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      if (c < p.nvec) reinterpret_cast<uint4*>(p.z)[base + c] = pack16(zv[i], T());
    }
  }
  if (p.h != nullptr) {
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) s[0] = fmaf(zv[i][e], zv[i][e], s[0]);
    row_sum<NT, 1>(s, buf[1]);
    const float r = 1.0f / sqrtf(s[0] * inv_h + p.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      float w[E], o[E];
      unpack16(wb[i], T(), w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        o[e] = zv[i][e] * r;
        if (p.w_pre != nullptr) o[e] *= p.offset + w[e];
      }
      if (c < p.nvec) reinterpret_cast<uint4*>(p.h)[base + c] = pack16(o, T());
    }
  }
}

// The gradients.  With zh = z r_z, yh = y r_y (y itself without its norm), b = yh (offset +
// w_post), a = dh (offset + w_pre):
//   D  = dz + r_z (a - zh mean(a zh))                       (= dx)
//   db = scale g D,  c = db (offset + w_post),  dy = r_y (c - yh mean(c yh))
//   dw_pre = sum dh zh,  dw_post = sum db yh,  dgate = scale D b (times a sigmoid's slope)
// At 8192 x 4096 in bf16 with a channel gate 88 us with the sums' kernel, 4.6 of the 5.2 TB/s that a
// large copy reaches: the sums of 512 blocks are another 50 MB, the rest the two waits of a row.
// (Loading the next row under this one, rows of 1024-thread blocks side by side and barriers
// that leave loads in flight were all slower, 96 to 150 us: registers, or rows in step.)
// r_z, r_y and the first mean are sums over the inputs alone, one reduction; mean(c yh) and a
// token gate's sum need D, a second one.  A block takes every gridDim.x-th row and keeps its
// threads' column sums in registers to the end, so the sums over tokens cost blocks * H
// floats of traffic instead of a pass; join_sum_kernel adds the blocks in order, which makes
// them the same every time.
template <typename T, int NT, int V>
__global__ __launch_bounds__(NT) void join_bwd_kernel(JoinBwdP p) {
  constexpr int E = Elem<T>::kPerVec;
  __shared__ float buf[2][3][NT / 64];
  const int tid = threadIdx.x;
  const float inv_h = 1.0f / float(p.H);
  const uint4 none = make_uint4(0, 0, 0, 0);
  uint4 wa[V], wb[V], gc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = tid + i * NT;
    const bool in = c < p.nvec;
    wa[i] = in && p.w_post != nullptr ? load_vec<T>(p.w_post, c) : none;
    wb[i] = in && p.w_pre != nullptr ? load_vec<T>(p.w_pre, c) : none;
    gc[i] = in && p.gate_kind == MOE_GATE_CHANNEL ? load_vec<T>(p.gate, c) : none;
  }
  float s_pre[V][E], s_post[V][E], s_gate[V][E];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) s_pre[i][e] = s_post[i][e] = s_gate[i][e] = 0.0f;
  const bool sig = p.gate_act == MOE_GATE_SIGMOID;

  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const size_t base = size_t(row) * p.nvec;
    uint4 zr[V], yr[V], dzr[V], dhr[V], ger[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      const bool in = c < p.nvec;
      zr[i] = in && p.dh != nullptr ? load_vec<T>(p.z, base + c) : none;
      dhr[i] = in && p.dh != nullptr ? load_vec<T>(p.dh, base + c) : none;
      yr[i] = in && p.y != nullptr ? load_vec<T>(p.y, base + c) : none;
      dzr[i] = in && p.dz != nullptr ? load_vec<T>(p.dz, base + c) : none;
      ger[i] = in && p.gate_kind == MOE_GATE_ELEMENT ? load_vec<T>(p.gate, base + c) : gc[i];
    }
    float g_raw = 0.0f;
    if (p.gate_kind == MOE_GATE_TOKEN) g_raw = static_cast<const float*>(p.gate)[row];

    float s[3] = {0.0f, 0.0f, 0.0f};  // sum z^2, sum a z, sum y^2
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float zf[E], hf[E], yf[E], w[E];
      unpack16(zr[i], T(), zf);
      unpack16(dhr[i], T(), hf);
      unpack16(yr[i], T(), yf);
      unpack16(wb[i], T(), w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float a = p.w_pre != nullptr ? hf[e] * (p.offset + w[e]) : hf[e];
        s[0] = fmaf(zf[e], zf[e], s[0]);
        s[1] = fmaf(a, zf[e], s[1]);
        s[2] = fmaf(yf[e], yf[e], s[2]);
      }
    }
    row_sum<NT, 3>(s, buf[0]);
    const float rz = p.dh != nullptr ? 1.0f / sqrtf(s[0] * inv_h + p.eps) : 0.0f;
    const float ry = p.post_norm ? 1.0f / sqrtf(s[2] * inv_h + p.eps) : 1.0f;
    const float mz = s[1] * rz * inv_h;  // mean(a zh)

    float dv[V][E];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      float zf[E], hf[E], w[E];
      unpack16(zr[i], T(), zf);
      unpack16(dhr[i], T(), hf);
      unpack16(wb[i], T(), w);
      unpack16(dzr[i], T(), dv[i]);
      if (p.dh != nullptr) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float zh = zf[e] * rz;
          const float a = p.w_pre != nullptr ? hf[e] * (p.offset + w[e]) : hf[e];
          s_pre[i][e] = fmaf(hf[e], zh, s_pre[i][e]);
          dv[i][e] = fmaf(rz, fmaf(-zh, mz, a), dv[i][e]);
        }
      }
      if (c < p.nvec) reinterpret_cast<uint4*>(p.dx)[base + c] = pack16(dv[i], T());
    }
    if (p.y == nullptr) {
      if (NT > 64) __syncthreads();  // buf[0] is written again
      continue;
    }

    Sigmoid g_row = {1.0f, 1.0f};  // a token gate's value and derivative
    if (p.gate_kind == MOE_GATE_TOKEN) g_row = sig ? sigmoid_and_slope<T>(g_raw) : Sigmoid{g_raw, 1.0f};
    const float k_row = p.scale * g_row.s;
    const bool whole = p.gate_kind == MOE_GATE_ELEMENT || p.gate_kind == MOE_GATE_CHANNEL;
    float t[2] = {0.0f, 0.0f};  // sum c yh, sum D b
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float yf[E], w[E], g[E], og[E];
      unpack16(yr[i], T(), yf);
      unpack16(wa[i], T(), w);
      unpack16(ger[i], T(), g);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float yh = yf[e] * ry;
        const float f = p.w_post != nullptr ? p.offset + w[e] : 1.0f;
        const Sigmoid gv = !whole ? Sigmoid{1.0f, 0.0f} : sig ? sigmoid_and_slope<T>(g[e]) : Sigmoid{g[e], 1.0f};
        const float db = k_row * gv.s * dv[i][e];
        const float dgb = dv[i][e] * (yh * f);
        t[0] = fmaf(db * f, yh, t[0]);
        t[1] += dgb;
        s_post[i][e] = fmaf(db, yh, s_post[i][e]);
        const float dg = whole ? p.scale * dgb : 0.0f;
        s_gate[i][e] += dg;  // a channel gate's slope is its rows' own factor: once, behind their sum
        og[e] = dg * gv.slope;
        dv[i][e] = db * f;  // c
      }
      const int c = tid + i * NT;
      if (p.gate_kind == MOE_GATE_ELEMENT && c < p.nvec) reinterpret_cast<uint4*>(p.dgate)[base + c] = pack16(og, T());
    }
    row_sum<NT, 2>(t, buf[1]);
    const float my = t[0] * inv_h;  // mean(c yh)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = tid + i * NT;
      float yf[E], o[E];
      unpack16(yr[i], T(), yf);
#pragma unroll
      for (int e = 0; e < E; ++e)  // without its norm dy is c, whatever y holds: 0 * inf would be NaN
        o[e] = p.post_norm ? ry * fmaf(-(yf[e] * ry), my, dv[i][e]) : dv[i][e];
      if (c < p.nvec) reinterpret_cast<uint4*>(p.dy)[base + c] = pack16(o, T());
    }
    if (p.gate_kind == MOE_GATE_TOKEN && tid == 0) static_cast<float*>(p.dgate)[row] = p.scale * t[1] * g_row.slope;
  }

#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = tid + i * NT;
    if (c >= p.nvec) continue;
    if (p.gate_kind == MOE_GATE_CHANNEL && sig) {
      float g[E];
      unpack16(gc[i], T(), g);
#pragma unroll
      for (int e = 0; e < E; ++e) s_gate[i][e] *= sigmoid_and_slope<T>(g[e]).slope;
    }
    auto put = [&](int which, const float (&v)[E]) {
      if (which < 0) return;
      float* dst = p.part + (size_t(which) * gridDim.x + blockIdx.x) * p.H + size_t(c) * E;
#pragma unroll
      for (int q = 0; q < E; q += 4) *reinterpret_cast<f32x4_t*>(dst + q) = f32x4_t{v[q], v[q + 1], v[q + 2], v[q + 3]};
    };
    put(p.p_pre, s_pre[i]);
    put(p.p_post, s_post[i]);
    put(p.p_gate, s_gate[i]);
  }
}

// Adds the blocks' column sums in a fixed order: 32 columns a block (a 128-byte line of each row
// of sums; half a line took 9.7 instead of 6 us for 25 MB), 128 threads down the rows with eight
// loads in flight.  Those eight, and the 128 after them, are added as trees: one after another they lost up to
// 30 units of 2^-24 of sums of 128 rows, 7 roundings lose 7 at most.
struct SumOut {
  void* out[3];
};
template <typename T>
__global__ __launch_bounds__(1024) void join_sum_kernel(const float* __restrict__ part, int blocks, int H, SumOut o) {
  constexpr int kCols = 32, kLanes = 128, kFlight = 8, kWaves = 16;
  __shared__ f32x4_t buf[kWaves][kCols / 4];
  const int sub = threadIdx.x & 7, lane = threadIdx.x >> 3, col = blockIdx.x * kCols + sub * 4;
  const float* src = part + size_t(blockIdx.y) * blocks * H + col;
  f32x4_t s = {0.f, 0.f, 0.f, 0.f};
  if (col < H) {
    for (int b0 = lane; b0 < blocks; b0 += kLanes * kFlight) {
      f32x4_t v[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int b = b0 + kLanes * u;
        v[u] = b < blocks ? *reinterpret_cast<const f32x4_t*>(src + size_t(b) * H) : f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int d = kFlight / 2; d >= 1; d >>= 1)
#pragma unroll
        for (int u = 0; u < d; ++u) v[u] += v[u + d];
      s += v[0];
    }
  }
#pragma unroll
  for (int d = 8; d < 64; d <<= 1)  // a wave has eight of the 128
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += __shfl_xor(s[e], d, 64);
  if ((threadIdx.x & 63) < 8) buf[threadIdx.x >> 6][sub] = s;
  __syncthreads();
  if (threadIdx.x < kCols && blockIdx.x * kCols + threadIdx.x < H) {
    const float* b = reinterpret_cast<const float*>(buf) + threadIdx.x;
    float a[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) a[w] = b[w * kCols];
#pragma unroll
    for (int d = kWaves / 2; d >= 1; d >>= 1)
#pragma unroll
      for (int w = 0; w < d; ++w) a[w] += a[w + d];
    static_cast<T*>(o.out[blockIdx.y])[blockIdx.x * kCols + threadIdx.x] = Elem<T>::from_f32(a[0]);
  }
}

int vectors(const moe_join_desc* j) { return int(size_t(j->hidden) * dtype_bytes(j->dtype) / 16); }

template <typename T, int NT, int V>
moe_status launch_fwd(const JoinP& p, hipStream_t s) {
  // at most 2^32 threads along x
  const int64_t blocks = NT == 64 ? (p.rows + 3) / 4 : p.rows, gx = std::min<int64_t>(blocks, 1 << 20);
  MOE_LAUNCH("block_join", (join_kernel<T, NT, V>), dim3(unsigned(gx), unsigned((blocks + gx - 1) / gx)),
             dim3(NT == 64 ? 256 : NT), 0, s, p);
  return MOE_OK;
}

template <typename T>
moe_status launch_fwd_t(const JoinP& p, hipStream_t s) {
  const int n = p.nvec;
  if (n <= 64) return launch_fwd<T, 64, 1>(p, s);
  if (n <= 128) return launch_fwd<T, 64, 2>(p, s);
  if (n <= 256) return launch_fwd<T, 256, 1>(p, s);
  if (n <= 512) return launch_fwd<T, 256, 2>(p, s);
  if (n <= 1024) return launch_fwd<T, 256, 4>(p, s);
  return launch_fwd<T, 1024, 2>(p, s);
}

// Threads of a row in the backward and vectors of a thread: one vector each up to 768 threads, and 512
// threads beyond, which leave each the registers for its sums (4096 x 8192 bf16: 106 us against
// 155 with 1024 threads, 3591 x 4672 float32 93 against 226; 5461 x 6144 bf16 106 with 768 threads,
// 114 with 384 of two vectors).  bf16 rows of more than 8192 spill all the same: 2730 x 12288 187 us
// (1024 threads of two vectors 517), 2048 x 16384 412 (418).
struct BwdShape {
  int nt, v;
};
BwdShape bwd_shape(const moe_join_desc* j) {
  const int n = vectors(j);
  for (int t : {64, 128, 192, 256, 384, 512, 768})
    if (n <= t) return {t, 1};
  return {512, (n + 511) / 512};
}
// Its blocks: as many on each of 256 CUs, up to 1024 vectors at once, and rows dealt evenly.  Half as many leave
// too few loads in flight (8192 x 4096 bf16 119 us instead of 88), twice as many write and read
// twice the sums (96 us); some CUs with a block more than others wait for those (262144 / 768 = 341
// blocks for 5692 x 4672: 138 instead of 105 us; 682 of 384 threads for 4096 x 2880: 56 instead of 44).
int bwd_blocks(const moe_join_desc* j) {
  const BwdShape w = bwd_shape(j);
  const int64_t most = 256 * std::max(1, 1024 / (w.nt * w.v));
  const int64_t each = std::max<int64_t>(1, (j->rows + most - 1) / most);
  return int((j->rows + each - 1) / each);
}

template <typename T, int NT, int V>
moe_status launch_bwd(const JoinBwdP& p, int blocks, hipStream_t s) {
  MOE_LAUNCH("block_join_bwd", (join_bwd_kernel<T, NT, V>), dim3(unsigned(blocks)), dim3(NT), 0, s, p);
  return MOE_OK;
}

template <typename T>
moe_status launch_bwd_t(const JoinBwdP& p, const BwdShape& w, int blocks, int sums, const SumOut& o, hipStream_t s) {
  const moe_status st = w.nt == 64    ? launch_bwd<T, 64, 1>(p, blocks, s)
                        : w.nt == 128 ? launch_bwd<T, 128, 1>(p, blocks, s)
                        : w.nt == 192 ? launch_bwd<T, 192, 1>(p, blocks, s)
                        : w.nt == 256 ? launch_bwd<T, 256, 1>(p, blocks, s)
                        : w.nt == 384 ? launch_bwd<T, 384, 1>(p, blocks, s)
                        : w.nt == 768 ? launch_bwd<T, 768, 1>(p, blocks, s)
                        : w.v == 1    ? launch_bwd<T, 512, 1>(p, blocks, s)
                        : w.v == 2    ? launch_bwd<T, 512, 2>(p, blocks, s)
                        : w.v == 3    ? launch_bwd<T, 512, 3>(p, blocks, s)
                                      : launch_bwd<T, 512, 4>(p, blocks, s);
  if (st != MOE_OK || sums == 0) return st;
  MOE_LAUNCH("block_join_bwd_sum", (join_sum_kernel<T>), dim3(unsigned((p.H + 31) / 32), unsigned(sums)), dim3(1024), 0, s,
             static_cast<const float*>(p.part), blocks, p.H, o);
  return MOE_OK;
}

}  // namespace

size_t join_workspace_bytes(const moe_join_desc* j) {
  const int sums = 1 + (j->post_norm ? 1 : 0) + (j->gate_kind == MOE_GATE_CHANNEL ? 1 : 0);
  return align_up(size_t(sums) * bwd_blocks(j) * j->hidden * sizeof(float), 256);
}

moe_status launch_join(const JoinArgs& a) {
  const moe_join_desc* j = a.j;
  const JoinP p{a.x,       a.y,          a.gate,       a.w_post,    a.w_pre, a.z, a.h, j->rows, j->hidden,
                vectors(j), j->post_norm, j->gate_kind, j->gate_act, j->eps,  j->weight_offset, j->residual_scale};
  return j->dtype == MOE_BF16 ? launch_fwd_t<bf16_t>(p, a.s) : launch_fwd_t<float>(p, a.s);
}

moe_status launch_join_backward(const JoinBwdArgs& a) {
  const moe_join_desc* j = a.j;
  SumOut o{};
  int sums = 0;
  auto ask = [&](void* out) {
    if (out == nullptr) return -1;
    o.out[sums] = out;
    return sums++;
  };
  const int p_pre = ask(a.dw_pre), p_post = ask(a.dw_post);
  const int p_gate = j->gate_kind == MOE_GATE_CHANNEL ? ask(a.dgate) : -1;
  const JoinBwdP p{a.z,  a.y,  a.gate, a.w_post, a.w_pre, a.dz, a.dh, a.dx, a.dy, a.dgate, static_cast<float*>(a.ws),
                   p_pre, p_post, p_gate, j->rows, j->hidden, vectors(j), j->post_norm, j->gate_kind, j->gate_act,
                   j->eps, j->weight_offset, j->residual_scale};
  return j->dtype == MOE_BF16 ? launch_bwd_t<bf16_t>(p, bwd_shape(j), bwd_blocks(j), sums, o, a.s)
                              : launch_bwd_t<float>(p, bwd_shape(j), bwd_blocks(j), sums, o, a.s);
}

}  // namespace moe
