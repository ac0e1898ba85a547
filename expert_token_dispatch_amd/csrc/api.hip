// libmoe C ABI: host-side validation, workspace layout and stage orchestration.
// The operations are defined in moe.h; every check below runs before any
// work is enqueued, following the Transformers "Expert parallelism" page's
// convention of rejecting a bad configuration before anything is sharded.
#include <cmath>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <mutex>

#include "kernels.h"

namespace moe {

namespace {
thread_local char g_err[1024] = "";
thread_local hipEvent_t g_prof_events[64];
thread_local int g_prof_count = 0;
thread_local int g_kernel_idx = 0;
thread_local int g_last_kernel_count = 0;
thread_local const char* g_kernel_names[64];

// Resets the per-call kernel counter; on exit records how many kernels ran.
struct CallScope {
  CallScope() { g_kernel_idx = 0; }
  ~CallScope() { g_last_kernel_count = g_kernel_idx; }
};
}  // namespace

moe_status set_error(moe_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return st;
}

void prof_before(const char* name, hipStream_t s) {
  if (g_kernel_idx < 64) g_kernel_names[g_kernel_idx] = name;
  if (2 * g_kernel_idx + 1 < g_prof_count && g_prof_events[2 * g_kernel_idx] != nullptr)
    (void)hipEventRecord(g_prof_events[2 * g_kernel_idx], s);
}

moe_status prof_after(const char* name, hipStream_t s) {
  const hipError_t e = hipGetLastError();
  if (2 * g_kernel_idx + 1 < g_prof_count && g_prof_events[2 * g_kernel_idx + 1] != nullptr)
    (void)hipEventRecord(g_prof_events[2 * g_kernel_idx + 1], s);
  ++g_kernel_idx;
  if (e != hipSuccess) return set_error(MOE_ERR_HIP, "%s: launch failed: %s", name, hipGetErrorString(e));
  return MOE_OK;
}

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

moe_status check_desc(const moe_layer_desc* d) {
  if (d == nullptr) return set_error(MOE_ERR_INVALID_ARG, "descriptor is NULL");
  if (d->num_tokens < 0) return set_error(MOE_ERR_INVALID_ARG, "num_tokens must be >= 0 (got %lld)", (long long)d->num_tokens);
  if (d->hidden <= 0 || d->hidden % 8 != 0)
    return set_error(MOE_ERR_INVALID_ARG, "hidden must be a positive multiple of 8 (got %d)", d->hidden);
  if (d->intermediate <= 0 || d->intermediate % 8 != 0)
    return set_error(MOE_ERR_INVALID_ARG, "intermediate must be a positive multiple of 8 (got %d)", d->intermediate);
  if (d->num_experts < 1) return set_error(MOE_ERR_INVALID_ARG, "num_experts must be >= 1 (got %d)", d->num_experts);
  if (d->top_k < 1 || d->top_k > d->num_experts)
    return set_error(MOE_ERR_INVALID_ARG, "top_k must be in [1, num_experts] (got %d, E=%d)", d->top_k, d->num_experts);
  if (d->local_begin < 0 || d->local_count < 1 || int64_t(d->local_begin) + d->local_count > d->num_experts)
    return set_error(MOE_ERR_INVALID_ARG, "local experts [%d, %d+%d) do not fit in [0, %d)", d->local_begin,
                     d->local_begin, d->local_count, d->num_experts);
  if (d->dtype != MOE_F32 && d->dtype != MOE_BF16) return set_error(MOE_ERR_INVALID_ARG, "unknown dtype %d", d->dtype);
  if (d->weight_layout != MOE_WEIGHTS_OUT_IN && d->weight_layout != MOE_WEIGHTS_IN_OUT)
    return set_error(MOE_ERR_INVALID_ARG, "unknown weight_layout %d", d->weight_layout);
  if (isnan(d->capacity_factor) || isinf(d->capacity_factor))
    return set_error(MOE_ERR_INVALID_ARG, "capacity_factor must be finite");
  if (d->num_tokens * int64_t(d->top_k) > INT32_MAX)
    return set_error(MOE_ERR_UNSUPPORTED, "num_tokens * top_k must be below 2^31");
  if (d->top_k > 32) return set_error(MOE_ERR_UNSUPPORTED, "top_k above 32 is not supported (got %d)", d->top_k);
  if (d->num_experts > 4096) return set_error(MOE_ERR_UNSUPPORTED, "num_experts above 4096 is not supported");
  return MOE_OK;
}

int64_t capacity_of(const moe_layer_desc* d) {
  if (d->capacity_factor <= 0.0f) return -1;
  const double c = floor(double(d->capacity_factor) * double(d->num_tokens) * double(d->top_k) / double(d->num_experts));
  return c > double(INT32_MAX) ? int64_t(INT32_MAX) : int64_t(c);
}

int64_t max_pairs_of(const moe_layer_desc* d) {
  const int64_t n = d->num_tokens * d->top_k;
  const int64_t c = capacity_of(d);
  return c < 0 ? n : std::min<int64_t>(n, int64_t(d->local_count) * c);
}

// moe_grouped_ffn's workspace: h [P_max, I], then the split-K pieces
size_t ffn_h_bytes(const moe_layer_desc* d) {
  return align_up(size_t(max_pairs_of(d)) * d->intermediate * dtype_bytes(d->dtype), 256);
}

// Layout of the moe_layer_forward workspace, or of another form's of the layer (which brings the
// scratch of its own feed-forward).
struct LayerWs {
  int32_t* topk_ids;
  float* topk_w;
  float* topk_logit;
  int32_t* counts;
  int32_t* offsets;
  int32_t* sorted_pairs;
  int32_t* pair_row;
  int64_t* num_dropped;
  void* route;
  void* dispatch;
  void* x_sorted;
  void* h;
  void* ffn_scratch;
  void* y_sorted;
  size_t bytes;
};

LayerWs layer_layout(const moe_layer_desc* d, void* base, size_t ffn_scratch) {
  const int64_t n = d->num_tokens * d->top_k;
  const int64_t pm = max_pairs_of(d);
  const size_t dt = dtype_bytes(d->dtype);
  char* p = static_cast<char*>(base);
  size_t o = 0;
  LayerWs w{};
  auto take = [&](size_t bytes) -> void* {
    void* r = p ? p + o : nullptr;
    o += align_up(bytes, 256);
    return r;
  };
  w.topk_ids = static_cast<int32_t*>(take(size_t(n) * 4));
  w.topk_w = static_cast<float*>(take(size_t(n) * 4));
  w.topk_logit = static_cast<float*>(take(size_t(n) * 4));
  w.counts = static_cast<int32_t*>(take(size_t(d->num_experts) * 4));
  w.offsets = static_cast<int32_t*>(take(size_t(d->local_count + 1) * 4));
  w.sorted_pairs = static_cast<int32_t*>(take(size_t(pm) * 4));
  w.pair_row = static_cast<int32_t*>(take(size_t(n) * 4));
  w.num_dropped = static_cast<int64_t*>(take(8));
  w.route = take(route_scratch_bytes(d));
  w.dispatch = take(dispatch_scratch_bytes(d));
  w.x_sorted = take(size_t(pm) * d->hidden * dt);
  w.h = take(size_t(pm) * d->intermediate * dt);
  w.ffn_scratch = ffn_scratch ? take(ffn_scratch) : nullptr;
  w.y_sorted = take(size_t(pm) * d->hidden * dt);
  w.bytes = o;
  return w;
}

LayerWs layer_layout(const moe_layer_desc* d, void* base) {
  return layer_layout(d, base, ffn_scratch_bytes(d, max_pairs_of(d)));
}
LayerWs packed_layer_layout(const moe_layer_desc* d, void* base) {
  return layer_layout(d, base, packed_ffn_scratch_bytes(d, max_pairs_of(d)));
}

// moe_grouped_ffn_backward's workspace: dg | du [P_max, 2I] and the large-tile path's scratch
size_t ffn_bwd_bytes(const moe_layer_desc* d) { return ffn_bwd_scratch_bytes(d, max_pairs_of(d)); }

// Layout of the moe_layer_backward workspace.
struct LayerBwdWs {
  void* dy_sorted;
  float* dl;
  void* dx_sorted;
  void* ffn;    // dg, du
  void* route;  // logit gradients
  size_t bytes;
};

LayerBwdWs layer_bwd_layout(const moe_layer_desc* d, void* base) {
  const int64_t pm = max_pairs_of(d);
  const size_t dt = dtype_bytes(d->dtype);
  char* p = static_cast<char*>(base);
  size_t o = 0;
  LayerBwdWs w{};
  auto take = [&](size_t bytes) -> void* {
    void* r = p ? p + o : nullptr;
    o += align_up(bytes, 256);
    return r;
  };
  w.dy_sorted = take(size_t(pm) * d->hidden * dt);
  w.dl = static_cast<float*>(take(size_t(d->num_tokens) * d->top_k * 4));
  w.dx_sorted = take(size_t(pm) * d->hidden * dt);
  w.ffn = take(ffn_bwd_bytes(d));
  w.route = take(route_bwd_scratch_bytes(d));
  w.bytes = o;
  return w;
}

size_t packed_stage_bytes(const moe_layer_desc* d, int32_t stage) {
  if (stage == MOE_STAGE_LAYER) return packed_layer_layout(d, nullptr).bytes;
  return ffn_h_bytes(d) + align_up(packed_ffn_scratch_bytes(d, max_pairs_of(d)), 256);
}

size_t stage_bytes(const moe_layer_desc* d, int32_t stage) {
  switch (stage) {
    case MOE_STAGE_ROUTE:
      return route_scratch_bytes(d);
    case MOE_STAGE_COMBINE:
      return 0;
    case MOE_STAGE_DISPATCH:
      return dispatch_scratch_bytes(d);
    case MOE_STAGE_FFN:
      return ffn_h_bytes(d) + align_up(ffn_scratch_bytes(d, max_pairs_of(d)), 256);
    case MOE_STAGE_LAYER:
      return layer_layout(d, nullptr).bytes;
    case MOE_STAGE_FFN_BACKWARD:
      return ffn_bwd_bytes(d);
    case MOE_STAGE_ROUTE_BACKWARD:
      return route_bwd_scratch_bytes(d);
    case MOE_STAGE_LAYER_BACKWARD:
      return layer_bwd_layout(d, nullptr).bytes;
    default:
      return 0;
  }
}

#define TRY_ZERO(expr)                 \
  do {                                 \
    const moe_status _z = (expr);      \
    if (_z != MOE_OK) return _z;       \
  } while (0)

#define REQUIRE_PTR(p, a)                                                                                  \
  do {                                                                                                     \
    if ((p) == nullptr) return set_error(MOE_ERR_INVALID_ARG, "%s is NULL", #p);                           \
    if (!aligned((p), (a))) return set_error(MOE_ERR_INVALID_ARG, "%s is not %d-byte aligned", #p, int(a)); \
  } while (0)
#define OPTIONAL_PTR(p, a)                                                                                  \
  do {                                                                                                     \
    if ((p) != nullptr && !aligned((p), (a)))                                                              \
      return set_error(MOE_ERR_INVALID_ARG, "%s is not %d-byte aligned", #p, int(a));                       \
  } while (0)

moe_status check_ws_bytes(size_t need, const void* ws, size_t ws_bytes) {
  if (need == 0) return MOE_OK;
  if (ws == nullptr || ws_bytes < need)
    return set_error(MOE_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given%s", need, ws_bytes,
                     ws == nullptr ? " (NULL)" : "");
  if (!aligned(ws, 256)) return set_error(MOE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return MOE_OK;
}

moe_status check_ws(const moe_layer_desc* d, int32_t stage, const void* ws, size_t ws_bytes) {
  return check_ws_bytes(stage_bytes(d, stage), ws, ws_bytes);
}

moe_status route_checks(const moe_layer_desc* d, const void* x, const void* w_router, const float* b_router,
                        const float* logits_in, const float* logits_out, const int32_t* topk_ids, const float* topk_w,
                        const float* topk_logit) {
  if (d->num_experts > 256) return set_error(MOE_ERR_UNSUPPORTED, "route: num_experts above 256 is not supported");
  if (logits_in == nullptr) {
    REQUIRE_PTR(x, 16);
    REQUIRE_PTR(w_router, 16);
    OPTIONAL_PTR(b_router, 4);
  } else {
    REQUIRE_PTR(logits_in, 4);
  }
  OPTIONAL_PTR(logits_out, 4);
  REQUIRE_PTR(topk_ids, 4);
  REQUIRE_PTR(topk_w, 4);
  OPTIONAL_PTR(topk_logit, 4);
  return MOE_OK;
}

moe_status dispatch_checks(const moe_layer_desc* d, const void* x, const int32_t* topk_ids, const float* topk_logit,
                           const int32_t* counts, const int32_t* offsets, const int32_t* sorted_pairs,
                           const int32_t* pair_row, const void* x_sorted, const int64_t* num_dropped) {
  if (d->local_count > 3000) return set_error(MOE_ERR_UNSUPPORTED, "dispatch: local_count above 3000 is not supported");
  REQUIRE_PTR(x, 16);
  REQUIRE_PTR(topk_ids, 4);
  if (d->capacity_factor > 0) {
    REQUIRE_PTR(topk_logit, 4);
  }
  REQUIRE_PTR(counts, 4);
  REQUIRE_PTR(offsets, 4);
  REQUIRE_PTR(sorted_pairs, 4);
  REQUIRE_PTR(pair_row, 4);
  REQUIRE_PTR(x_sorted, 16);
  OPTIONAL_PTR(num_dropped, 8);
  // the capacity cut holds an expert's pairs (at most one per token) in registers
  if (d->capacity_factor > 0 && d->num_tokens > 32768)
    return set_error(MOE_ERR_UNSUPPORTED, "capacity_factor > 0 supports at most 32768 tokens per call");
  return MOE_OK;
}

moe_status ffn_checks(const void* x_sorted, const int32_t* offsets, const void* w_gate, const void* w_up,
                      const void* w_down, const void* y_sorted) {
  REQUIRE_PTR(x_sorted, 16);
  REQUIRE_PTR(offsets, 4);
  REQUIRE_PTR(w_gate, 16);
  REQUIRE_PTR(w_up, 16);
  REQUIRE_PTR(w_down, 16);
  REQUIRE_PTR(y_sorted, 16);
  return MOE_OK;
}

moe_status combine_checks(const void* y_sorted, const int32_t* pair_row, const float* topk_w, const void* y) {
  REQUIRE_PTR(y_sorted, 16);
  REQUIRE_PTR(pair_row, 4);
  REQUIRE_PTR(topk_w, 4);
  REQUIRE_PTR(y, 16);
  return MOE_OK;
}

moe_status packed_desc_checks(const moe_layer_desc* d) {
  if (d->hidden % 32 != 0 || d->intermediate % 32 != 0)
    return set_error(MOE_ERR_UNSUPPORTED, "packed experts: hidden and intermediate must be multiples of 32 (got %d, %d)",
                     d->hidden, d->intermediate);
  return MOE_OK;
}

moe_status packed_checks(const moe_packed_experts* p) {
  if (p == nullptr) return set_error(MOE_ERR_INVALID_ARG, "packed is NULL");
  REQUIRE_PTR(p->gate_codes, 16);
  REQUIRE_PTR(p->gate_scales, 1);
  REQUIRE_PTR(p->up_codes, 16);
  REQUIRE_PTR(p->up_scales, 1);
  REQUIRE_PTR(p->down_codes, 16);
  REQUIRE_PTR(p->down_scales, 1);
  return MOE_OK;
}

moe_status packed_ffn_checks(const void* x_sorted, const int32_t* offsets, const moe_packed_experts* p,
                             const void* y_sorted) {
  REQUIRE_PTR(x_sorted, 16);
  REQUIRE_PTR(offsets, 4);
  REQUIRE_PTR(y_sorted, 16);
  return packed_checks(p);
}

moe_status pack_checks(int32_t count, int32_t out, int32_t in, int32_t dtype, int32_t layout, const void* w,
                       const void* codes, const void* scales) {
  if (count < 1) return set_error(MOE_ERR_INVALID_ARG, "count must be >= 1 (got %d)", count);
  if (count > 65535) return set_error(MOE_ERR_UNSUPPORTED, "count above 65535 is not supported (got %d)", count);
  if (out <= 0 || out % 8 != 0) return set_error(MOE_ERR_INVALID_ARG, "out must be a positive multiple of 8 (got %d)", out);
  if (in <= 0 || in % 32 != 0) return set_error(MOE_ERR_INVALID_ARG, "in must be a positive multiple of 32 (got %d)", in);
  if (dtype != MOE_F32 && dtype != MOE_BF16) return set_error(MOE_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (layout != MOE_WEIGHTS_OUT_IN && layout != MOE_WEIGHTS_IN_OUT)
    return set_error(MOE_ERR_INVALID_ARG, "unknown weight_layout %d", layout);
  if ((out + 63) / 64 > 65535) return set_error(MOE_ERR_UNSUPPORTED, "out above %d is not supported", 65535 * 64);
  REQUIRE_PTR(w, 16);
  REQUIRE_PTR(codes, 16);
  REQUIRE_PTR(scales, 1);
  return MOE_OK;
}

// Largest |s (a + b s^2 + c s^4)| over s in [0, top]: at an end or where the derivative
// a + 3 b s^2 + 5 c s^4 vanishes.
double largest_image(double a, double b, double c, double top) {
  auto f = [&](double s) { return fabs(s * (a + b * s * s + c * s * s * s * s)); };
  double best = f(top);
  const double disc = 9.0 * b * b - 20.0 * a * c;
  double roots[2] = {-1.0, -1.0};  // values of s^2
  if (c != 0.0) {
    if (disc >= 0.0) {
      roots[0] = (-3.0 * b + sqrt(disc)) / (10.0 * c);
      roots[1] = (-3.0 * b - sqrt(disc)) / (10.0 * c);
    }
  } else if (b != 0.0) {
    roots[0] = -a / (3.0 * b);
  }
  for (double r : roots)
    if (r > 0.0 && r < top * top) best = std::max(best, f(sqrt(r)));
  return best;
}

// What the update computes with: the descriptor's coefficients or the usual ones.
struct MuonCoefs {
  float a, b, c;
};
MuonCoefs muon_coefs(const moe_muon_desc* m) {
  if (m->coef_a == 0.f && m->coef_b == 0.f && m->coef_c == 0.f) return {3.4445f, -4.7750f, 2.0315f};
  return {m->coef_a, m->coef_b, m->coef_c};
}

moe_status muon_desc_checks(const moe_muon_desc* m) {
  if (m == nullptr) return set_error(MOE_ERR_INVALID_ARG, "descriptor is NULL");
  if (m->count < 1 || m->rows < 1 || m->cols < 1)
    return set_error(MOE_ERR_INVALID_ARG, "count, rows and cols must be >= 1 (got %d, %d, %d)", m->count, m->rows, m->cols);
  if (m->count > 65535) return set_error(MOE_ERR_UNSUPPORTED, "count above 65535 is not supported (got %d)", m->count);
  if (m->dtype != MOE_F32 && m->dtype != MOE_BF16) return set_error(MOE_ERR_INVALID_ARG, "unknown dtype %d", m->dtype);
  if (m->steps < 1 || m->steps > 10) return set_error(MOE_ERR_INVALID_ARG, "steps must be in [1, 10] (got %d)", m->steps);
  if (!std::isfinite(m->coef_a) || !std::isfinite(m->coef_b) || !std::isfinite(m->coef_c))
    return set_error(MOE_ERR_INVALID_ARG, "coefficients must be finite");
  const MuonCoefs k = muon_coefs(m);
  if (!(k.a > 0.f && k.a <= 4.f)) return set_error(MOE_ERR_INVALID_ARG, "coef_a must be in (0, 4] (got %g)", double(k.a));
  // singular values start in [0, 1]; the float16 working range is sized for values up to 3
  double top = 1.0;
  for (int i = 0; i < m->steps; ++i) {
    top = largest_image(k.a, k.b, k.c, top);
    if (!(top <= 3.0))
      return set_error(MOE_ERR_INVALID_ARG, "coefficients (%g, %g, %g) take a singular value past 3 in step %d",
                       double(k.a), double(k.b), double(k.c), i + 1);
    top = std::max(top, 1.0);
  }
  if (!(std::isfinite(m->eps) && m->eps >= 0.f)) return set_error(MOE_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!(m->momentum >= 0.f && m->momentum < 1.f))
    return set_error(MOE_ERR_INVALID_ARG, "momentum must be in [0, 1) (got %g)", double(m->momentum));
  if (m->nesterov != 0 && m->nesterov != 1)
    return set_error(MOE_ERR_INVALID_ARG, "nesterov must be 0 or 1 (got %d)", m->nesterov);
  if (!std::isfinite(m->lr) || !std::isfinite(m->update_scale) || !std::isfinite(m->weight_decay))
    return set_error(MOE_ERR_INVALID_ARG, "lr, update_scale and weight_decay must be finite");
  if (m->rows > 65535 * 64 || m->cols > 65535 * 64)
    return set_error(MOE_ERR_UNSUPPORTED, "rows and cols above %d are not supported (got %d, %d)", 65535 * 64, m->rows,
                     m->cols);
  if (muon_matrix_bytes(m) >= (int64_t(1) << 32))
    return set_error(MOE_ERR_UNSUPPORTED, "a matrix of %d x %d takes 4 GiB or more of workspace", m->rows, m->cols);
  return MOE_OK;
}

MuonArgs muon_args(const moe_muon_desc* m, void* ws, void* stream) {
  const MuonCoefs k = muon_coefs(m);
  MuonArgs a{};
  a.m = m;
  a.ca = k.a;
  a.cb = k.b;
  a.cc = k.c;
  a.ws = ws;
  a.s = static_cast<hipStream_t>(stream);
  return a;
}

// pointers false: only which of them are NULL counts
moe_status adapters_checks(const moe_adapters* a, bool pointers = true) {
  if (a == nullptr) return set_error(MOE_ERR_INVALID_ARG, "adapters are NULL");
  if (a->count < 1 || a->count > 65535)
    return set_error(MOE_ERR_INVALID_ARG, "adapters: count must be in [1, 65535] (got %d)", a->count);
  if (a->rank < 8 || a->rank > 128 || a->rank % 8 != 0)
    return set_error(MOE_ERR_INVALID_ARG, "adapters: rank must be a multiple of 8 in [8, 128] (got %d)", a->rank);
  const void* pairs[3][2] = {{a->gate_a, a->gate_b}, {a->up_a, a->up_b}, {a->down_a, a->down_b}};
  static const char* const names[3] = {"gate", "up", "down"};
  int given = 0;
  for (int i = 0; i < 3; ++i) {
    if ((pairs[i][0] == nullptr) != (pairs[i][1] == nullptr))
      return set_error(MOE_ERR_INVALID_ARG, "adapters: %s_a and %s_b: give both or neither", names[i], names[i]);
    if (pointers && (!aligned(pairs[i][0], 16) || !aligned(pairs[i][1], 16)))
      return set_error(MOE_ERR_INVALID_ARG, "adapters: %s_a or %s_b is not 16-byte aligned", names[i], names[i]);
    given += pairs[i][0] != nullptr;
  }
  if (given == 0) return set_error(MOE_ERR_INVALID_ARG, "adapters: no projection has a pair");
  if (pointers) OPTIONAL_PTR(a->scale, 4);
  return MOE_OK;
}

// the first products address a row block and an adapter's A with 32-bit offsets
moe_status adapted_desc_checks(const moe_layer_desc* d) {
  if (d->hidden > kAdapterMaxK || d->intermediate > kAdapterMaxK)
    return set_error(MOE_ERR_UNSUPPORTED, "adapters: hidden and intermediate above %d are not supported (got %d, %d)",
                     kAdapterMaxK, d->hidden, d->intermediate);
  if (max_pairs_of(d) > kAdapterMaxPairs)
    return set_error(MOE_ERR_UNSUPPORTED, "adapters: more than %d pairs a call are not supported", kAdapterMaxPairs);
  return MOE_OK;
}

// The layer's workspace with adapters: its intermediates, then the adapters' part (with the
// feed-forward's scratch); the feed-forward's alone: h, then that part.
size_t adapted_front_bytes(const moe_layer_desc* d, int32_t stage) {
  return stage == MOE_STAGE_LAYER ? layer_layout(d, nullptr, 0).bytes : ffn_h_bytes(d);
}
size_t adapted_stage_bytes(const moe_layer_desc* d, const moe_adapters* a, int32_t stage) {
  return adapted_front_bytes(d, stage) + carve_adapter_scratch(d, a, max_pairs_of(d), nullptr).bytes;
}
AdapterScratch adapted_scratch(const moe_layer_desc* d, const moe_adapters* a, int32_t stage, void* ws) {
  return carve_adapter_scratch(d, a, max_pairs_of(d), static_cast<char*>(ws) + adapted_front_bytes(d, stage));
}

moe_status join_desc_checks(const moe_join_desc* j) {
  if (j == nullptr) return set_error(MOE_ERR_INVALID_ARG, "descriptor is NULL");
  if (j->rows < 0) return set_error(MOE_ERR_INVALID_ARG, "rows must be >= 0 (got %lld)", (long long)j->rows);
  if (j->rows > INT32_MAX) return set_error(MOE_ERR_UNSUPPORTED, "rows must be below 2^31");
  if (j->hidden <= 0 || j->hidden % 8 != 0)
    return set_error(MOE_ERR_INVALID_ARG, "hidden must be a positive multiple of 8 (got %d)", j->hidden);
  if (j->dtype != MOE_F32 && j->dtype != MOE_BF16) return set_error(MOE_ERR_INVALID_ARG, "unknown dtype %d", j->dtype);
  if (size_t(j->hidden) * dtype_bytes(j->dtype) > size_t(kJoinMaxRowBytes))
    return set_error(MOE_ERR_UNSUPPORTED, "rows of more than %d bytes are not supported (hidden %d)", kJoinMaxRowBytes,
                     j->hidden);
  if (j->post_norm != 0 && j->post_norm != 1)
    return set_error(MOE_ERR_INVALID_ARG, "post_norm must be 0 or 1 (got %d)", j->post_norm);
  if (j->gate_kind < MOE_GATE_NONE || j->gate_kind > MOE_GATE_ELEMENT)
    return set_error(MOE_ERR_INVALID_ARG, "unknown gate_kind %d", j->gate_kind);
  if (j->gate_act != MOE_GATE_LINEAR && j->gate_act != MOE_GATE_SIGMOID)
    return set_error(MOE_ERR_INVALID_ARG, "unknown gate_act %d", j->gate_act);
  if (!(std::isfinite(j->eps) && j->eps > 0.f)) return set_error(MOE_ERR_INVALID_ARG, "eps must be finite and > 0");
  if (!std::isfinite(j->weight_offset) || !std::isfinite(j->residual_scale))
    return set_error(MOE_ERR_INVALID_ARG, "weight_offset and residual_scale must be finite");
  return MOE_OK;
}

// `out` is given exactly where `in` is
#define REQUIRE_BOTH(out, in, a)                                                                            \
  do {                                                                                                      \
    if (((out) == nullptr) != ((in) == nullptr))                                                            \
      return set_error(MOE_ERR_INVALID_ARG, "%s and %s: give both or neither", #out, #in);                  \
    OPTIONAL_PTR(out, a);                                                                                   \
  } while (0)

// What the forward and the backward take alike.
moe_status join_operand_checks(const moe_join_desc* j, const void* y, const void* gate, const void* w_post,
                               const void* w_pre) {
  if (y == nullptr && (j->post_norm || j->gate_kind != MOE_GATE_NONE))
    return set_error(MOE_ERR_INVALID_ARG, "without y post_norm has to be 0 and gate_kind MOE_GATE_NONE");
  OPTIONAL_PTR(y, 16);
  if ((gate == nullptr) != (j->gate_kind == MOE_GATE_NONE))
    return set_error(MOE_ERR_INVALID_ARG, "gate is %s and gate_kind %d", gate == nullptr ? "NULL" : "given", j->gate_kind);
  OPTIONAL_PTR(gate, j->gate_kind == MOE_GATE_TOKEN ? 4 : 16);
  if (!j->post_norm && w_post != nullptr)
    return set_error(MOE_ERR_INVALID_ARG, "w_post is given and post_norm is 0");
  OPTIONAL_PTR(w_post, 16);
  OPTIONAL_PTR(w_pre, 16);
  return MOE_OK;
}

moe_status saved_checks(const moe_saved* v) {
  if (v == nullptr) return set_error(MOE_ERR_INVALID_ARG, "saved is NULL");
  REQUIRE_PTR(v->topk_ids, 4);
  REQUIRE_PTR(v->topk_w, 4);
  REQUIRE_PTR(v->offsets, 4);
  REQUIRE_PTR(v->pair_row, 4);
  REQUIRE_PTR(v->x_sorted, 16);
  REQUIRE_PTR(v->gate, 16);
  REQUIRE_PTR(v->up, 16);
  REQUIRE_PTR(v->h, 16);
  REQUIRE_PTR(v->y_sorted, 16);
  return MOE_OK;
}

moe_status combine_bwd_checks(const void* dy, const void* y_sorted, const int32_t* pair_row, const float* topk_w,
                              const void* dy_sorted, const float* dl) {
  REQUIRE_PTR(dy, 16);
  REQUIRE_PTR(y_sorted, 16);
  REQUIRE_PTR(pair_row, 4);
  REQUIRE_PTR(topk_w, 4);
  REQUIRE_PTR(dy_sorted, 16);
  REQUIRE_PTR(dl, 4);
  return MOE_OK;
}

moe_status ffn_bwd_checks(const void* x_sorted, const int32_t* offsets, const void* w_gate, const void* w_up,
                          const void* w_down, const void* gate, const void* up, const void* h, const void* dy_sorted,
                          const void* dx_sorted, const void* dw_gate, const void* dw_up, const void* dw_down) {
  REQUIRE_PTR(x_sorted, 16);
  REQUIRE_PTR(offsets, 4);
  REQUIRE_PTR(w_gate, 16);
  REQUIRE_PTR(w_up, 16);
  REQUIRE_PTR(w_down, 16);
  REQUIRE_PTR(gate, 16);
  REQUIRE_PTR(up, 16);
  REQUIRE_PTR(h, 16);
  REQUIRE_PTR(dy_sorted, 16);
  REQUIRE_PTR(dx_sorted, 16);
  REQUIRE_PTR(dw_gate, 16);
  REQUIRE_PTR(dw_up, 16);
  REQUIRE_PTR(dw_down, 16);
  return MOE_OK;
}

moe_status route_bwd_checks(const void* x, const int32_t* topk_ids, const float* dl, const void* dw_router,
                            const float* db_router) {
  REQUIRE_PTR(x, 16);
  REQUIRE_PTR(topk_ids, 4);
  REQUIRE_PTR(dl, 4);
  REQUIRE_PTR(dw_router, 16);
  OPTIONAL_PTR(db_router, 16);
  return MOE_OK;
}

moe_status dispatch_bwd_checks(const void* dx_sorted, const int32_t* pair_row, const int32_t* topk_ids,
                               const float* dl, const void* w_router, const void* dx) {
  REQUIRE_PTR(dx_sorted, 16);
  REQUIRE_PTR(pair_row, 4);
  REQUIRE_PTR(topk_ids, 4);
  REQUIRE_PTR(dl, 4);
  REQUIRE_PTR(w_router, 16);
  REQUIRE_PTR(dx, 16);
  return MOE_OK;
}

// Zero weight gradients of a layer that saw no tokens (no expert received any).
moe_status zero_ffn_grads(const moe_layer_desc* d, void* dw_gate, void* dw_up, void* dw_down, hipStream_t s) {
  const size_t n = size_t(d->local_count) * d->intermediate * d->hidden * dtype_bytes(d->dtype);
  TRY_ZERO(launch_zero("ffn_bwd_zero", dw_gate, n, s));
  TRY_ZERO(launch_zero("ffn_bwd_zero", dw_up, n, s));
  return launch_zero("ffn_bwd_zero", dw_down, n, s);
}

moe_status zero_route_grads(const moe_layer_desc* d, void* dw_router, float* db_router, hipStream_t s) {
  TRY_ZERO(launch_zero("route_bwd_zero", dw_router, size_t(d->num_experts) * d->hidden * dtype_bytes(d->dtype), s));
  return launch_zero("route_bwd_zero", db_router, size_t(d->num_experts) * 4, s);
}

#define TRY(expr)                          \
  do {                                     \
    const moe_status _s = (expr);          \
    if (_s != MOE_OK) return _s;           \
  } while (0)

}  // namespace
}  // namespace moe

using namespace moe;

namespace moe {
namespace {
// Routing options: glossary "Load balancing and capacity" (selection bias, groups per token).
moe_status opts_checks(const moe_layer_desc* d, const moe_route_opts* o) {
  if (o == nullptr || o->num_groups <= 1) return MOE_OK;
  const int E = d->num_experts, G = o->num_groups;
  if (G > 16) return set_error(MOE_ERR_UNSUPPORTED, "route options: num_groups above 16 is not supported (got %d)", G);
  if (E % G != 0) return set_error(MOE_ERR_INVALID_ARG, "route options: num_groups %d does not divide E=%d", G, E);
  if (o->max_groups < 1 || o->max_groups > G)
    return set_error(MOE_ERR_INVALID_ARG, "route options: max_groups must be in [1, %d] (got %d)", G, o->max_groups);
  if (int64_t(o->max_groups) * (E / G) < d->top_k)
    return set_error(MOE_ERR_INVALID_ARG, "route options: %d groups of %d experts hold fewer than k=%d", o->max_groups,
                     E / G, d->top_k);
  return MOE_OK;
}

void apply_opts(RouteArgs& a, const moe_layer_desc* d, const moe_route_opts* o) {
  if (o == nullptr) return;
  a.sel_bias = o->selection_bias;
  if (o->num_groups > 1 && o->max_groups < o->num_groups) {
    a.group_size = d->num_experts / o->num_groups;
    a.max_groups = o->max_groups;
  }
}
}  // namespace
}  // namespace moe

// ---- the dispatch scratch of moe_dispatch_noalloc -----------------------------
// For callers that cannot allocate device memory (code under graph capture,
// tight serving loops, harnesses that forbid hipMalloc): the dispatch kernels'
// scratch (per-chunk histograms, per-chunk segment bases, pre-capacity
// offsets and permutation) lives in this file-scope device array instead of a
// caller workspace.  Each GPU holds its own copy for the life of the process.
// Host code never passes the array's name to a kernel (on the host it only
// names a stand-in): it resolves the device address once per device with
// hipGetSymbolAddress and passes that.
namespace moe {
namespace {
constexpr size_t kNoAllocScratchBytes = size_t(16) << 20;
constexpr int kMaxDevices = 64;
static __device__ __align__(256) char scratch[kNoAllocScratchBytes];

std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices];

// The current device's address of `scratch` (resolved on the first call per device).
moe_status noalloc_scratch(void** out) {
  int dev = -1;
  const hipError_t ge = hipGetDevice(&dev);
  if (ge != hipSuccess) return set_error(MOE_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(ge));
  if (dev < 0 || dev >= kMaxDevices) return set_error(MOE_ERR_UNSUPPORTED, "device %d: at most %d devices", dev, kMaxDevices);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_ptr[dev] == nullptr) {
    void* ptr = nullptr;
    const hipError_t e = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
    if (e != hipSuccess || ptr == nullptr)
      return set_error(MOE_ERR_HIP, "hipGetSymbolAddress(scratch) on device %d: %s", dev, hipGetErrorString(e));
    g_scratch_ptr[dev] = ptr;
  }
  *out = g_scratch_ptr[dev];
  return MOE_OK;
}
}  // namespace
}  // namespace moe

extern "C" {

const char* moe_last_error(void) { return g_err; }

const char* moe_version(void) { return "libmoe 0.1 (gfx950)"; }

moe_status moe_ep_local_range(int32_t num_experts, int32_t ep_size, int32_t rank, int32_t* begin, int32_t* count) {
  if (begin == nullptr || count == nullptr) return set_error(MOE_ERR_INVALID_ARG, "begin/count are NULL");
  if (num_experts < 1) return set_error(MOE_ERR_INVALID_ARG, "num_experts must be >= 1");
  if (ep_size < 1) return set_error(MOE_ERR_INVALID_ARG, "ep_size must be >= 1");
  if (rank < 0) return set_error(MOE_ERR_INVALID_ARG, "rank must be >= 0");
  if (num_experts % ep_size != 0)
    return set_error(MOE_ERR_INVALID_ARG, "ep_size %d does not divide num_experts %d", ep_size, num_experts);
  const int32_t per = num_experts / ep_size;
  *begin = (rank % ep_size) * per;
  *count = per;
  return MOE_OK;
}

int64_t moe_capacity(const moe_layer_desc* d) {
  if (check_desc(d) != MOE_OK) return -1;
  return capacity_of(d);
}

int64_t moe_max_pairs(const moe_layer_desc* d) {
  if (check_desc(d) != MOE_OK) return -1;
  return max_pairs_of(d);
}

moe_status moe_workspace_size(const moe_layer_desc* d, int32_t stage, size_t* bytes) {
  TRY(check_desc(d));
  if (bytes == nullptr) return set_error(MOE_ERR_INVALID_ARG, "bytes is NULL");
  if (stage < MOE_STAGE_ROUTE || stage > MOE_STAGE_LAYER_BACKWARD)
    return set_error(MOE_ERR_INVALID_ARG, "unknown stage %d", stage);
  *bytes = stage_bytes(d, stage);
  return MOE_OK;
}

moe_status moe_profile_events(void* const* events, int32_t count) {
  if (events == nullptr || count <= 0) {
    g_prof_count = 0;
    return MOE_OK;
  }
  if (count > 64 || count % 2 != 0)
    return set_error(MOE_ERR_INVALID_ARG, "profiling events: an even count of at most 64 (got %d)", count);
  for (int i = 0; i < count; ++i) {
    if ((events[i] == nullptr) != (events[i ^ 1] == nullptr))
      return set_error(MOE_ERR_INVALID_ARG, "profiling events %d and %d: give both or neither", i & ~1, i | 1);
    g_prof_events[i] = static_cast<hipEvent_t>(events[i]);
  }
  g_prof_count = count;
  return MOE_OK;
}

const char* moe_profile_kernel_name(int32_t i) {
  if (i < 0 || i >= g_last_kernel_count || i >= 64) return nullptr;
  return g_kernel_names[i];
}

int32_t moe_profile_kernel_count(void) { return g_last_kernel_count; }

moe_status moe_route_ex(const moe_layer_desc* d, const moe_route_opts* opts, const void* x, const void* w_router,
                        const float* b_router, const float* logits_in, float* logits_out, int32_t* topk_ids,
                        float* topk_w, float* topk_logit, void* ws, size_t ws_bytes, void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  if (d->num_tokens == 0) return MOE_OK;
  TRY(route_checks(d, x, w_router, b_router, logits_in, logits_out, topk_ids, topk_w, topk_logit));
  TRY(opts_checks(d, opts));
  if (logits_in == nullptr) TRY(check_ws(d, MOE_STAGE_ROUTE, ws, ws_bytes));
  RouteArgs a{d, x, w_router, b_router, logits_in, logits_out, topk_ids, topk_w, topk_logit,
              static_cast<float*>(ws), nullptr, static_cast<hipStream_t>(stream)};
  apply_opts(a, d, opts);
  return launch_route(a);
}

moe_status moe_route(const moe_layer_desc* d, const void* x, const void* w_router, const float* b_router,
                     const float* logits_in, float* logits_out, int32_t* topk_ids, float* topk_w, float* topk_logit,
                     void* ws, size_t ws_bytes, void* stream) {
  return moe_route_ex(d, nullptr, x, w_router, b_router, logits_in, logits_out, topk_ids, topk_w, topk_logit, ws,
                      ws_bytes, stream);
}

moe_status moe_selection_bias_update(const moe_layer_desc* d, const int32_t* counts, float* bias, float gamma,
                                     void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  if (counts == nullptr || bias == nullptr)
    return set_error(MOE_ERR_INVALID_ARG, "selection bias update: counts and bias are required");
  if (!std::isfinite(gamma)) return set_error(MOE_ERR_INVALID_ARG, "selection bias update: gamma must be finite");
  return launch_selection_bias_update(d, counts, bias, gamma, static_cast<hipStream_t>(stream));
}

moe_status moe_dispatch(const moe_layer_desc* d, const void* x, const int32_t* topk_ids, const float* topk_logit,
                        int32_t* counts, int32_t* offsets, int32_t* sorted_pairs, int32_t* pair_row, void* x_sorted,
                        int64_t* num_dropped, void* ws, size_t ws_bytes, void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  if (d->num_tokens == 0) return MOE_OK;
  TRY(dispatch_checks(d, x, topk_ids, topk_logit, counts, offsets, sorted_pairs, pair_row, x_sorted, num_dropped));
  TRY(check_ws(d, MOE_STAGE_DISPATCH, ws, ws_bytes));
  DispatchArgs a{d, x, topk_ids, topk_logit, counts, offsets, sorted_pairs, pair_row, x_sorted, num_dropped,
                 carve_dispatch_scratch(d, ws), capacity_of(d), false, static_cast<hipStream_t>(stream)};
  return launch_dispatch(a);
}

moe_status moe_dispatch_noalloc(const moe_layer_desc* d, const void* x, const int32_t* topk_ids,
                                const float* topk_logit, int32_t* counts, int32_t* offsets, int32_t* sorted_pairs,
                                int32_t* pair_row, void* x_sorted, int64_t* num_dropped, void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  if (d->num_tokens == 0) return MOE_OK;
  TRY(dispatch_checks(d, x, topk_ids, topk_logit, counts, offsets, sorted_pairs, pair_row, x_sorted, num_dropped));
  const size_t need = dispatch_scratch_bytes(d);
  if (need > kNoAllocScratchBytes)
    return set_error(MOE_ERR_UNSUPPORTED, "dispatch_noalloc: %zu bytes of scratch needed, the static buffer holds %zu",
                     need, kNoAllocScratchBytes);
  void* scr = nullptr;
  TRY(noalloc_scratch(&scr));
  // every scratch entry the kernels read is written earlier in the same call, so
  // nothing needs clearing between calls
  DispatchArgs a{d, x, topk_ids, topk_logit, counts, offsets, sorted_pairs, pair_row, x_sorted, num_dropped,
                 carve_dispatch_scratch(d, scr), capacity_of(d), false, static_cast<hipStream_t>(stream)};
  return launch_dispatch(a);
}

moe_status moe_grouped_ffn(const moe_layer_desc* d, const void* x_sorted, const int32_t* offsets, const void* w_gate,
                           const void* w_up, const void* w_down, void* y_sorted, void* ws, size_t ws_bytes,
                           void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  if (d->num_tokens == 0) return MOE_OK;
  TRY(ffn_checks(x_sorted, offsets, w_gate, w_up, w_down, y_sorted));
  TRY(check_ws(d, MOE_STAGE_FFN, ws, ws_bytes));
  void* scratch = ffn_scratch_bytes(d, max_pairs_of(d)) ? static_cast<char*>(ws) + ffn_h_bytes(d) : nullptr;
  FfnArgs a{d, x_sorted, offsets, w_gate, w_up, w_down, y_sorted, ws, scratch, max_pairs_of(d),
            static_cast<hipStream_t>(stream)};
  return launch_grouped_ffn(a);
}

moe_status moe_combine(const moe_layer_desc* d, const void* y_sorted, const int32_t* pair_row, const float* topk_w,
                       void* y, void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  if (d->num_tokens == 0) return MOE_OK;
  TRY(combine_checks(y_sorted, pair_row, topk_w, y));
  CombineArgs a{d, y_sorted, pair_row, topk_w, y, static_cast<hipStream_t>(stream)};
  return launch_combine(a);
}

moe_status moe_layer_forward(const moe_layer_desc* d, const void* x, const void* w_router, const float* b_router,
                             const void* w_gate, const void* w_up, const void* w_down, void* y, int32_t* topk_ids_out,
                             float* topk_w_out, int32_t* counts_out, int64_t* num_dropped_out, void* ws,
                             size_t ws_bytes, void* stream) {
  return moe_layer_forward_ex(d, nullptr, x, w_router, b_router, w_gate, w_up, w_down, y, topk_ids_out, topk_w_out,
                              counts_out, num_dropped_out, ws, ws_bytes, stream);
}

moe_status moe_layer_forward_ex(const moe_layer_desc* d, const moe_route_opts* opts, const void* x,
                                const void* w_router, const float* b_router, const void* w_gate, const void* w_up,
                                const void* w_down, void* y, int32_t* topk_ids_out, float* topk_w_out,
                                int32_t* counts_out, int64_t* num_dropped_out, void* ws, size_t ws_bytes,
                                void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  if (d->num_tokens == 0) return MOE_OK;
  TRY(check_ws(d, MOE_STAGE_LAYER, ws, ws_bytes));
  LayerWs w = layer_layout(d, ws);
  int32_t* ids = topk_ids_out ? topk_ids_out : w.topk_ids;
  float* tw = topk_w_out ? topk_w_out : w.topk_w;
  int32_t* counts = counts_out ? counts_out : w.counts;
  int64_t* dropped = num_dropped_out ? num_dropped_out : w.num_dropped;
  const bool cap = capacity_of(d) >= 0;
  TRY(route_checks(d, x, w_router, b_router, nullptr, nullptr, ids, tw, w.topk_logit));
  TRY(dispatch_checks(d, x, ids, w.topk_logit, counts, w.offsets, w.sorted_pairs, w.pair_row, w.x_sorted, dropped));
  TRY(ffn_checks(w.x_sorted, w.offsets, w_gate, w_up, w_down, w.y_sorted));
  TRY(combine_checks(w.y_sorted, w.pair_row, tw, y));
  TRY(opts_checks(d, opts));
  const hipStream_t s = static_cast<hipStream_t>(stream);

  const DispatchScratch scr = carve_dispatch_scratch(d, w.dispatch);
  // the router's top-k kernel also writes the per-chunk expert histograms
  RouteArgs ra{d, x, w_router, b_router, nullptr, nullptr, ids, tw, cap ? w.topk_logit : nullptr,
               static_cast<float*>(w.route), scr.blk_all, s};
  apply_opts(ra, d, opts);
  TRY(launch_route(ra));
  DispatchArgs da{d, x, ids, w.topk_logit, counts, w.offsets, w.sorted_pairs, w.pair_row, w.x_sorted, dropped,
                  scr, capacity_of(d), true, s};
  TRY(launch_dispatch(da));
  FfnArgs fa{d, w.x_sorted, w.offsets, w_gate, w_up, w_down, w.y_sorted, w.h, w.ffn_scratch, max_pairs_of(d), s};
  TRY(launch_grouped_ffn(fa));
  CombineArgs ca{d, w.y_sorted, w.pair_row, tw, y, s};
  return launch_combine(ca);
}

moe_status moe_grouped_ffn_train(const moe_layer_desc* d, const void* x_sorted, const int32_t* offsets,
                                 const void* w_gate, const void* w_up, const void* w_down, void* y_sorted, void* h,
                                 void* gate, void* up, void* ws, size_t ws_bytes, void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  if (d->num_tokens == 0) return MOE_OK;
  TRY(ffn_checks(x_sorted, offsets, w_gate, w_up, w_down, y_sorted));
  REQUIRE_PTR(h, 16);
  REQUIRE_PTR(gate, 16);
  REQUIRE_PTR(up, 16);
  TRY(check_ws(d, MOE_STAGE_FFN, ws, ws_bytes));
  void* scratch = ffn_scratch_bytes(d, max_pairs_of(d)) ? static_cast<char*>(ws) + ffn_h_bytes(d) : nullptr;
  FfnArgs a{d, x_sorted, offsets, w_gate, w_up, w_down, y_sorted, h, scratch, max_pairs_of(d),
            static_cast<hipStream_t>(stream), gate, up};
  return launch_grouped_ffn(a);
}

moe_status moe_layer_forward_train(const moe_layer_desc* d, const moe_route_opts* opts, const void* x,
                                   const void* w_router, const float* b_router, const void* w_gate, const void* w_up,
                                   const void* w_down, void* y, const moe_saved* saved, int32_t* counts_out,
                                   int64_t* num_dropped_out, void* ws, size_t ws_bytes, void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  if (d->num_tokens == 0) return MOE_OK;
  TRY(saved_checks(saved));
  TRY(check_ws(d, MOE_STAGE_LAYER, ws, ws_bytes));
  LayerWs w = layer_layout(d, ws);
  const moe_saved& v = *saved;
  int32_t* counts = counts_out ? counts_out : w.counts;
  int64_t* dropped = num_dropped_out ? num_dropped_out : w.num_dropped;
  const bool cap = capacity_of(d) >= 0;
  TRY(route_checks(d, x, w_router, b_router, nullptr, nullptr, v.topk_ids, v.topk_w, w.topk_logit));
  TRY(dispatch_checks(d, x, v.topk_ids, w.topk_logit, counts, v.offsets, w.sorted_pairs, v.pair_row, v.x_sorted,
                      dropped));
  TRY(ffn_checks(v.x_sorted, v.offsets, w_gate, w_up, w_down, v.y_sorted));
  TRY(combine_checks(v.y_sorted, v.pair_row, v.topk_w, y));
  TRY(opts_checks(d, opts));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const DispatchScratch scr = carve_dispatch_scratch(d, w.dispatch);
  RouteArgs ra{d, x, w_router, b_router, nullptr, nullptr, v.topk_ids, v.topk_w, cap ? w.topk_logit : nullptr,
               static_cast<float*>(w.route), scr.blk_all, s};
  apply_opts(ra, d, opts);
  TRY(launch_route(ra));
  DispatchArgs da{d, x, v.topk_ids, w.topk_logit, counts, v.offsets, w.sorted_pairs, v.pair_row, v.x_sorted,
                  dropped, scr, capacity_of(d), true, s};
  TRY(launch_dispatch(da));
  FfnArgs fa{d, v.x_sorted, v.offsets, w_gate, w_up, w_down, v.y_sorted, v.h, w.ffn_scratch, max_pairs_of(d), s,
             v.gate, v.up};
  TRY(launch_grouped_ffn(fa));
  CombineArgs ca{d, v.y_sorted, v.pair_row, v.topk_w, y, s};
  return launch_combine(ca);
}

moe_status moe_combine_backward(const moe_layer_desc* d, const void* dy, const void* y_sorted,
                                const int32_t* pair_row, const float* topk_w, void* dy_sorted, float* dl,
                                void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  if (d->num_tokens == 0) return MOE_OK;
  TRY(combine_bwd_checks(dy, y_sorted, pair_row, topk_w, dy_sorted, dl));
  CombineBwdArgs a{d, dy, y_sorted, pair_row, topk_w, dy_sorted, dl, static_cast<hipStream_t>(stream)};
  return launch_combine_backward(a);
}

moe_status moe_grouped_ffn_backward(const moe_layer_desc* d, const void* x_sorted, const int32_t* offsets,
                                    const void* w_gate, const void* w_up, const void* w_down, const void* gate,
                                    const void* up, const void* h, const void* dy_sorted, void* dx_sorted,
                                    void* dw_gate, void* dw_up, void* dw_down, void* ws, size_t ws_bytes,
                                    void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (d->num_tokens == 0) {
    REQUIRE_PTR(dw_gate, 16);
    REQUIRE_PTR(dw_up, 16);
    REQUIRE_PTR(dw_down, 16);
    return zero_ffn_grads(d, dw_gate, dw_up, dw_down, s);
  }
  TRY(ffn_bwd_checks(x_sorted, offsets, w_gate, w_up, w_down, gate, up, h, dy_sorted, dx_sorted, dw_gate, dw_up,
                     dw_down));
  TRY(check_ws(d, MOE_STAGE_FFN_BACKWARD, ws, ws_bytes));
  FfnBwdArgs a{d, x_sorted, offsets, w_gate, w_up, w_down, gate, up, h, dy_sorted, dx_sorted, dw_gate, dw_up,
               dw_down, ws, max_pairs_of(d), s};
  return launch_grouped_ffn_backward(a);
}

moe_status moe_route_backward(const moe_layer_desc* d, const void* x, const int32_t* topk_ids, const float* dl,
                              void* dw_router, float* db_router, void* ws, size_t ws_bytes, void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (d->num_tokens == 0) {
    REQUIRE_PTR(dw_router, 16);
    OPTIONAL_PTR(db_router, 16);
    return zero_route_grads(d, dw_router, db_router, s);
  }
  TRY(route_bwd_checks(x, topk_ids, dl, dw_router, db_router));
  TRY(check_ws(d, MOE_STAGE_ROUTE_BACKWARD, ws, ws_bytes));
  RouteBwdArgs a{d, x, topk_ids, dl, dw_router, db_router, ws, s};
  return launch_route_backward(a);
}

moe_status moe_dispatch_backward(const moe_layer_desc* d, const void* dx_sorted, const int32_t* pair_row,
                                 const int32_t* topk_ids, const float* dl, const void* w_router, void* dx,
                                 void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  if (d->num_tokens == 0) return MOE_OK;
  TRY(dispatch_bwd_checks(dx_sorted, pair_row, topk_ids, dl, w_router, dx));
  DispatchBwdArgs a{d, dx_sorted, pair_row, topk_ids, dl, w_router, dx, static_cast<hipStream_t>(stream)};
  return launch_dispatch_backward(a);
}

moe_status moe_layer_backward(const moe_layer_desc* d, const void* x, const void* w_router, const void* w_gate,
                              const void* w_up, const void* w_down, const moe_saved* saved, const void* dy,
                              void* dx, void* dw_router, float* db_router, void* dw_gate, void* dw_up,
                              void* dw_down, void* ws, size_t ws_bytes, void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (d->num_tokens == 0) {
    REQUIRE_PTR(dw_router, 16);
    OPTIONAL_PTR(db_router, 16);
    REQUIRE_PTR(dw_gate, 16);
    REQUIRE_PTR(dw_up, 16);
    REQUIRE_PTR(dw_down, 16);
    TRY(zero_route_grads(d, dw_router, db_router, s));
    return zero_ffn_grads(d, dw_gate, dw_up, dw_down, s);
  }
  TRY(saved_checks(saved));
  TRY(check_ws(d, MOE_STAGE_LAYER_BACKWARD, ws, ws_bytes));
  const moe_saved& v = *saved;
  LayerBwdWs w = layer_bwd_layout(d, ws);
  TRY(combine_bwd_checks(dy, v.y_sorted, v.pair_row, v.topk_w, w.dy_sorted, w.dl));
  TRY(ffn_bwd_checks(v.x_sorted, v.offsets, w_gate, w_up, w_down, v.gate, v.up, v.h, w.dy_sorted, w.dx_sorted,
                     dw_gate, dw_up, dw_down));
  TRY(route_bwd_checks(x, v.topk_ids, w.dl, dw_router, db_router));
  TRY(dispatch_bwd_checks(w.dx_sorted, v.pair_row, v.topk_ids, w.dl, w_router, dx));
  CombineBwdArgs ca{d, dy, v.y_sorted, v.pair_row, v.topk_w, w.dy_sorted, w.dl, s};
  TRY(launch_combine_backward(ca));
  FfnBwdArgs fa{d, v.x_sorted, v.offsets, w_gate, w_up, w_down, v.gate, v.up, v.h, w.dy_sorted, w.dx_sorted,
                dw_gate, dw_up, dw_down, w.ffn, max_pairs_of(d), s};
  TRY(launch_grouped_ffn_backward(fa));
  RouteBwdArgs ra{d, x, v.topk_ids, w.dl, dw_router, db_router, w.route, s};
  TRY(launch_route_backward(ra));
  DispatchBwdArgs da{d, w.dx_sorted, v.pair_row, v.topk_ids, w.dl, w_router, dx, s};
  return launch_dispatch_backward(da);
}

moe_status moe_pack_weights(int32_t count, int32_t out, int32_t in, int32_t dtype, int32_t weight_layout,
                            const void* w, void* codes, void* scales, void* stream) {
  CallScope scope;
  TRY(pack_checks(count, out, in, dtype, weight_layout, w, codes, scales));
  PackArgs a{count, out, in, dtype, weight_layout, const_cast<void*>(w), codes, scales, static_cast<hipStream_t>(stream)};
  return launch_pack("pack_weights", a);
}

moe_status moe_unpack_weights(int32_t count, int32_t out, int32_t in, int32_t dtype, int32_t weight_layout,
                              const void* codes, const void* scales, void* w, void* stream) {
  CallScope scope;
  TRY(pack_checks(count, out, in, dtype, weight_layout, w, codes, scales));
  PackArgs a{count, out, in, dtype, weight_layout, w, const_cast<void*>(codes), const_cast<void*>(scales),
             static_cast<hipStream_t>(stream)};
  return launch_unpack("unpack_weights", a);
}

moe_status moe_packed_workspace_size(const moe_layer_desc* d, int32_t stage, size_t* bytes) {
  TRY(check_desc(d));
  TRY(packed_desc_checks(d));
  if (bytes == nullptr) return set_error(MOE_ERR_INVALID_ARG, "bytes is NULL");
  if (stage != MOE_STAGE_FFN && stage != MOE_STAGE_LAYER)
    return set_error(MOE_ERR_INVALID_ARG, "stage %d has no packed form", stage);
  *bytes = packed_stage_bytes(d, stage);
  return MOE_OK;
}

moe_status moe_grouped_ffn_packed(const moe_layer_desc* d, const void* x_sorted, const int32_t* offsets,
                                  const moe_packed_experts* packed, void* y_sorted, void* ws, size_t ws_bytes,
                                  void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  TRY(packed_desc_checks(d));
  if (d->num_tokens == 0) return MOE_OK;
  TRY(packed_ffn_checks(x_sorted, offsets, packed, y_sorted));
  TRY(check_ws_bytes(packed_stage_bytes(d, MOE_STAGE_FFN), ws, ws_bytes));
  PackedFfnArgs a{d, x_sorted, offsets, packed, y_sorted, ws, static_cast<char*>(ws) + ffn_h_bytes(d), max_pairs_of(d),
                  static_cast<hipStream_t>(stream)};
  return launch_packed_ffn(a);
}

moe_status moe_layer_forward_packed(const moe_layer_desc* d, const moe_route_opts* opts, const void* x,
                                    const void* w_router, const float* b_router, const moe_packed_experts* packed,
                                    void* y, int32_t* topk_ids_out, float* topk_w_out, int32_t* counts_out,
                                    int64_t* num_dropped_out, void* ws, size_t ws_bytes, void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  TRY(packed_desc_checks(d));
  if (d->num_tokens == 0) return MOE_OK;
  TRY(check_ws_bytes(packed_stage_bytes(d, MOE_STAGE_LAYER), ws, ws_bytes));
  const LayerWs w = packed_layer_layout(d, ws);
  int32_t* ids = topk_ids_out ? topk_ids_out : w.topk_ids;
  float* tw = topk_w_out ? topk_w_out : w.topk_w;
  int32_t* counts = counts_out ? counts_out : w.counts;
  int64_t* dropped = num_dropped_out ? num_dropped_out : w.num_dropped;
  const bool cap = capacity_of(d) >= 0;
  TRY(route_checks(d, x, w_router, b_router, nullptr, nullptr, ids, tw, w.topk_logit));
  TRY(dispatch_checks(d, x, ids, w.topk_logit, counts, w.offsets, w.sorted_pairs, w.pair_row, w.x_sorted, dropped));
  TRY(packed_ffn_checks(w.x_sorted, w.offsets, packed, w.y_sorted));
  TRY(combine_checks(w.y_sorted, w.pair_row, tw, y));
  TRY(opts_checks(d, opts));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const DispatchScratch scr = carve_dispatch_scratch(d, w.dispatch);
  RouteArgs ra{d, x, w_router, b_router, nullptr, nullptr, ids, tw, cap ? w.topk_logit : nullptr,
               static_cast<float*>(w.route), scr.blk_all, s};
  apply_opts(ra, d, opts);
  TRY(launch_route(ra));
  DispatchArgs da{d, x, ids, w.topk_logit, counts, w.offsets, w.sorted_pairs, w.pair_row, w.x_sorted, dropped,
                  scr, capacity_of(d), true, s};
  TRY(launch_dispatch(da));
  PackedFfnArgs fa{d, w.x_sorted, w.offsets, packed, w.y_sorted, w.h, w.ffn_scratch, max_pairs_of(d), s};
  TRY(launch_packed_ffn(fa));
  CombineArgs ca{d, w.y_sorted, w.pair_row, tw, y, s};
  return launch_combine(ca);
}

moe_status moe_muon_workspace_size(const moe_muon_desc* m, size_t* bytes) {
  TRY(muon_desc_checks(m));
  if (bytes == nullptr) return set_error(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = muon_workspace_bytes(m);
  return MOE_OK;
}

moe_status moe_orthogonalize(const moe_muon_desc* m, const void* g, void* o, void* ws, size_t ws_bytes, void* stream) {
  CallScope scope;
  TRY(muon_desc_checks(m));
  REQUIRE_PTR(g, 16);
  REQUIRE_PTR(o, 16);
  TRY(check_ws_bytes(muon_workspace_bytes(m), ws, ws_bytes));
  MuonArgs a = muon_args(m, ws, stream);
  a.grad = g;
  a.out = o;
  return launch_muon(a);
}

moe_status moe_muon_update(const moe_muon_desc* m, const void* grad, float* momentum, float* master, void* weight,
                           void* ws, size_t ws_bytes, void* stream) {
  CallScope scope;
  TRY(muon_desc_checks(m));
  REQUIRE_PTR(grad, 16);
  REQUIRE_PTR(momentum, 16);
  OPTIONAL_PTR(master, 16);
  REQUIRE_PTR(weight, 16);
  TRY(check_ws_bytes(muon_workspace_bytes(m), ws, ws_bytes));
  MuonArgs a = muon_args(m, ws, stream);
  a.grad = grad;
  a.momentum = momentum;
  a.master = master;
  a.out = weight;
  return launch_muon(a);
}

moe_status moe_adapted_workspace_size(const moe_layer_desc* d, const moe_adapters* a, int32_t stage, size_t* bytes) {
  TRY(check_desc(d));
  TRY(adapted_desc_checks(d));
  TRY(adapters_checks(a, false));
  if (bytes == nullptr) return set_error(MOE_ERR_INVALID_ARG, "bytes is NULL");
  if (stage != MOE_STAGE_FFN && stage != MOE_STAGE_LAYER)
    return set_error(MOE_ERR_INVALID_ARG, "stage %d has no form with adapters", stage);
  *bytes = adapted_stage_bytes(d, a, stage);
  return MOE_OK;
}

moe_status moe_grouped_ffn_adapted(const moe_layer_desc* d, const void* x_sorted, const int32_t* offsets,
                                   const int32_t* sorted_pairs, const int32_t* adapter_ids, const void* w_gate,
                                   const void* w_up, const void* w_down, const moe_adapters* a, void* y_sorted, void* ws,
                                   size_t ws_bytes, void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  TRY(adapted_desc_checks(d));
  TRY(adapters_checks(a));
  if (d->num_tokens == 0) return MOE_OK;
  TRY(ffn_checks(x_sorted, offsets, w_gate, w_up, w_down, y_sorted));
  REQUIRE_PTR(sorted_pairs, 4);
  REQUIRE_PTR(adapter_ids, 4);
  TRY(check_ws_bytes(adapted_stage_bytes(d, a, MOE_STAGE_FFN), ws, ws_bytes));
  const AdapterScratch as = adapted_scratch(d, a, MOE_STAGE_FFN, ws);
  FfnArgs fa{d, x_sorted, offsets, w_gate, w_up, w_down, y_sorted, ws, as.ffn, max_pairs_of(d),
             static_cast<hipStream_t>(stream)};
  AdaptedFfnArgs aa{fa, sorted_pairs, adapter_ids, a, as};
  return launch_adapted_ffn(aa);
}

moe_status moe_layer_forward_adapted(const moe_layer_desc* d, const moe_route_opts* opts, const void* x,
                                     const int32_t* adapter_ids, const void* w_router, const float* b_router,
                                     const void* w_gate, const void* w_up, const void* w_down, const moe_adapters* a,
                                     void* y, int32_t* topk_ids_out, float* topk_w_out, int32_t* counts_out,
                                     int64_t* num_dropped_out, void* ws, size_t ws_bytes, void* stream) {
  CallScope scope;
  TRY(check_desc(d));
  TRY(adapted_desc_checks(d));
  TRY(adapters_checks(a));
  if (d->num_tokens == 0) return MOE_OK;
  TRY(check_ws_bytes(adapted_stage_bytes(d, a, MOE_STAGE_LAYER), ws, ws_bytes));
  REQUIRE_PTR(adapter_ids, 4);
  const LayerWs w = layer_layout(d, ws, 0);
  const AdapterScratch as = adapted_scratch(d, a, MOE_STAGE_LAYER, ws);
  int32_t* ids = topk_ids_out ? topk_ids_out : w.topk_ids;
  float* tw = topk_w_out ? topk_w_out : w.topk_w;
  int32_t* counts = counts_out ? counts_out : w.counts;
  int64_t* dropped = num_dropped_out ? num_dropped_out : w.num_dropped;
  const bool cap = capacity_of(d) >= 0;
  TRY(route_checks(d, x, w_router, b_router, nullptr, nullptr, ids, tw, w.topk_logit));
  TRY(dispatch_checks(d, x, ids, w.topk_logit, counts, w.offsets, w.sorted_pairs, w.pair_row, w.x_sorted, dropped));
  TRY(ffn_checks(w.x_sorted, w.offsets, w_gate, w_up, w_down, w.y_sorted));
  TRY(combine_checks(w.y_sorted, w.pair_row, tw, y));
  TRY(opts_checks(d, opts));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const DispatchScratch scr = carve_dispatch_scratch(d, w.dispatch);
  RouteArgs ra{d, x, w_router, b_router, nullptr, nullptr, ids, tw, cap ? w.topk_logit : nullptr,
               static_cast<float*>(w.route), scr.blk_all, s};
  apply_opts(ra, d, opts);
  TRY(launch_route(ra));
  DispatchArgs da{d, x, ids, w.topk_logit, counts, w.offsets, w.sorted_pairs, w.pair_row, w.x_sorted, dropped,
                  scr, capacity_of(d), true, s};
  TRY(launch_dispatch(da));
  FfnArgs fa{d, w.x_sorted, w.offsets, w_gate, w_up, w_down, w.y_sorted, w.h, as.ffn, max_pairs_of(d), s};
  AdaptedFfnArgs aa{fa, w.sorted_pairs, adapter_ids, a, as};
  TRY(launch_adapted_ffn(aa));
  CombineArgs ca{d, w.y_sorted, w.pair_row, tw, y, s};
  return launch_combine(ca);
}

moe_status moe_block_join(const moe_join_desc* j, const void* x, const void* y, const void* gate, const void* w_post,
                          const void* w_pre, void* z, void* h, void* stream) {
  CallScope scope;
  TRY(join_desc_checks(j));
  if (j->rows == 0) return MOE_OK;
  REQUIRE_PTR(x, 16);
  TRY(join_operand_checks(j, y, gate, w_post, w_pre));
  REQUIRE_BOTH(z, y, 16);
  OPTIONAL_PTR(h, 16);
  if (h == nullptr && (y == nullptr || w_pre != nullptr))
    return set_error(MOE_ERR_INVALID_ARG, "h is NULL and %s", y == nullptr ? "y too" : "w_pre is given");
  JoinArgs a{j, x, y, gate, w_post, w_pre, z, h, static_cast<hipStream_t>(stream)};
  return launch_join(a);
}

moe_status moe_join_workspace_size(const moe_join_desc* j, size_t* bytes) {
  TRY(join_desc_checks(j));
  if (bytes == nullptr) return set_error(MOE_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = join_workspace_bytes(j);
  return MOE_OK;
}

moe_status moe_block_join_backward(const moe_join_desc* j, const void* z, const void* y, const void* gate,
                                   const void* w_post, const void* w_pre, const void* dz, const void* dh, void* dx,
                                   void* dy, void* dgate, void* dw_post, void* dw_pre, void* ws, size_t ws_bytes,
                                   void* stream) {
  CallScope scope;
  TRY(join_desc_checks(j));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  REQUIRE_BOTH(dw_post, w_post, 16);
  REQUIRE_BOTH(dw_pre, w_pre, 16);
  if (j->rows == 0) {
    const size_t n = size_t(j->hidden) * dtype_bytes(j->dtype);
    if (j->gate_kind == MOE_GATE_CHANNEL) REQUIRE_PTR(dgate, 16);
    if (dw_post != nullptr) TRY(launch_zero("block_join_bwd_zero", dw_post, n, s));
    if (dw_pre != nullptr) TRY(launch_zero("block_join_bwd_zero", dw_pre, n, s));
    return j->gate_kind == MOE_GATE_CHANNEL ? launch_zero("block_join_bwd_zero", dgate, n, s) : MOE_OK;
  }
  TRY(join_operand_checks(j, y, gate, w_post, w_pre));
  OPTIONAL_PTR(dz, 16);
  OPTIONAL_PTR(dh, 16);
  if (dh != nullptr) {
    REQUIRE_PTR(z, 16);
  } else if (dz == nullptr || w_pre != nullptr) {
    return set_error(MOE_ERR_INVALID_ARG, "dh is NULL and %s", dz == nullptr ? "dz too" : "w_pre is given");
  }
  REQUIRE_PTR(dx, 16);
  REQUIRE_BOTH(dy, y, 16);
  REQUIRE_BOTH(dgate, gate, j->gate_kind == MOE_GATE_TOKEN ? 4 : 16);
  TRY(check_ws_bytes(join_workspace_bytes(j), ws, ws_bytes));
  JoinBwdArgs a{j, z, y, gate, w_post, w_pre, dz, dh, dx, dy, dgate, dw_post, dw_pre, ws, s};
  return launch_join_backward(a);
}

}  // extern "C"
