"""ctypes binding of libmoe (include/moe.h).  Argument marshalling only."""

from __future__ import annotations

import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(PKG, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = 0, -1, -2, -3, -4
MOE_F32, MOE_BF16 = 0, 1
MOE_WEIGHTS_OUT_IN, MOE_WEIGHTS_IN_OUT = 0, 1
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_TOKEN, MOE_GATE_ELEMENT = 0, 1, 2, 3
MOE_GATE_LINEAR, MOE_GATE_SIGMOID = 0, 1
MOE_STAGE_ROUTE, MOE_STAGE_DISPATCH, MOE_STAGE_FFN, MOE_STAGE_COMBINE, MOE_STAGE_LAYER = 0, 1, 2, 3, 4
MOE_STAGE_FFN_BACKWARD, MOE_STAGE_ROUTE_BACKWARD, MOE_STAGE_LAYER_BACKWARD = 5, 6, 7

_STATUS = {0: "MOE_OK", -1: "MOE_ERR_INVALID_ARG", -2: "MOE_ERR_UNSUPPORTED", -3: "MOE_ERR_WORKSPACE",
           -4: "MOE_ERR_HIP"}


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


class LayerDesc(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("hidden", ctypes.c_int32),
        ("intermediate", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("local_begin", ctypes.c_int32),
        ("local_count", ctypes.c_int32),
        ("capacity_factor", ctypes.c_float),
        ("dtype", ctypes.c_int32),
        ("weight_layout", ctypes.c_int32),
    ]


class RouteOpts(ctypes.Structure):
    """moe_route_opts: selection-only expert bias and groups per token (include/moe.h)."""
    _fields_ = [
        ("selection_bias", ctypes.c_void_p),
        ("num_groups", ctypes.c_int32),
        ("max_groups", ctypes.c_int32),
    ]


class Saved(ctypes.Structure):
    """moe_saved: what the training forward keeps for the backward (include/moe.h)."""
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("topk_ids", "topk_w", "offsets", "pair_row", "x_sorted", "gate", "up", "h", "y_sorted")]


class PackedExperts(ctypes.Structure):
    """moe_packed_experts: the local experts' weights in 4 bits (include/moe.h)."""
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("gate_codes", "gate_scales", "up_codes", "up_scales", "down_codes", "down_scales")]


class MuonDesc(ctypes.Structure):
    """moe_muon_desc: a stack of matrices and how it is updated (include/moe.h)."""
    _fields_ = [
        ("count", ctypes.c_int32),
        ("rows", ctypes.c_int32),
        ("cols", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("steps", ctypes.c_int32),
        ("coef_a", ctypes.c_float),
        ("coef_b", ctypes.c_float),
        ("coef_c", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("momentum", ctypes.c_float),
        ("nesterov", ctypes.c_int32),
        ("lr", ctypes.c_float),
        ("update_scale", ctypes.c_float),
        ("weight_decay", ctypes.c_float),
    ]


class Adapters(ctypes.Structure):
    """moe_adapters: low-rank pairs of many requests beside the expert weights (include/moe.h)."""
    _fields_ = [("count", ctypes.c_int32), ("rank", ctypes.c_int32)] + [(n, ctypes.c_void_p) for n in (
        "scale", "gate_a", "gate_b", "up_a", "up_b", "down_a", "down_b")]


class JoinDesc(ctypes.Structure):
    """moe_join_desc: the join of a block with the residual stream (include/moe.h)."""
    _fields_ = [
        ("rows", ctypes.c_int64),
        ("hidden", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("post_norm", ctypes.c_int32),
        ("gate_kind", ctypes.c_int32),
        ("gate_act", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("weight_offset", ctypes.c_float),
        ("residual_scale", ctypes.c_float),
    ]


def make_saved(t: dict) -> Saved:
    """t: a dict of device tensors under the moe_saved field names.  The struct
    keeps a reference to the dict, so the pointers stay valid while it lives."""
    v = Saved(*[_p(t[n]) for n, _ in Saved._fields_])
    v._tensors = t
    return v


def make_route_opts(selection_bias=None, num_groups: int = 0, max_groups: int = 0) -> RouteOpts:
    """selection_bias: float32 [E] device tensor or None.  The options keep a
    reference to it, so the pointer stays valid while they are alive."""
    o = RouteOpts(_p(selection_bias), int(num_groups), int(max_groups))
    o._bias = selection_bias
    return o


def make_desc(num_tokens: int, hidden: int, intermediate: int, num_experts: int, top_k: int,
              local_begin: int = 0, local_count: Optional[int] = None, capacity_factor: float = 0.0,
              dtype="bf16", weight_layout="out_in") -> LayerDesc:
    """weight_layout: "out_in" (w_gate, w_up [L, I, H], w_down [L, H, I]) or "in_out"
    (w_gate, w_up [L, H, I], w_down [L, I, H]), or the MOE_WEIGHTS_* value."""
    if isinstance(dtype, str):
        dtype = {"bf16": MOE_BF16, "f32": MOE_F32}[dtype]
    if isinstance(weight_layout, str):
        weight_layout = {"out_in": MOE_WEIGHTS_OUT_IN, "in_out": MOE_WEIGHTS_IN_OUT}[weight_layout]
    return LayerDesc(num_tokens, hidden, intermediate, num_experts, top_k, local_begin,
                     num_experts if local_count is None else local_count, capacity_factor, dtype, weight_layout)


def make_packed_experts(t: dict) -> PackedExperts:
    """t: a dict of uint8 device tensors under the moe_packed_experts field names.  The
    struct keeps a reference to the dict, so the pointers stay valid while it lives."""
    v = PackedExperts(*[_p(t[n]) for n, _ in PackedExperts._fields_])
    v._tensors = t
    return v


def make_muon_desc(count: int, rows: int, cols: int, dtype="bf16", steps: int = 5, momentum: float = 0.95,
                   nesterov: bool = True, lr: float = 0.0, update_scale: float = 1.0, weight_decay: float = 0.0,
                   eps: float = 1e-7, coefs=(0.0, 0.0, 0.0)) -> MuonDesc:
    """coefs: (a, b, c) of a Newton-Schulz step; all zero for the usual ones."""
    if isinstance(dtype, str):
        dtype = {"bf16": MOE_BF16, "f32": MOE_F32}[dtype]
    a, b, c = coefs
    return MuonDesc(count, rows, cols, dtype, steps, a, b, c, eps, momentum, int(nesterov), lr, update_scale,
                    weight_decay)


ADAPTED = ("gate", "up", "down")


def make_adapters(t: dict) -> Adapters:
    """t: a dict of device tensors under the moe_adapters field names: "gate_a" [count, L, rank, H],
    "gate_b" [count, L, I, rank], "up_a", "up_b" alike, "down_a" [count, L, rank, I], "down_b"
    [count, L, H, rank], and "scale" [count] float32; a projection's pair and the scale may be left
    out.  The struct keeps a reference to the dict, so the pointers stay valid while it lives."""
    t = {k: v for k, v in t.items() if v is not None}
    first = next((t[n + "_a"] for n in ADAPTED if n + "_a" in t), None)
    if first is None or first.dim() != 4:
        raise ValueError("adapters have an \"_a\" of at least one projection, of four dimensions")
    v = Adapters(first.shape[0], first.shape[2], *[_p(t.get(n)) for n, _ in Adapters._fields_[2:]])
    v._tensors, v._fits = t, None
    return v


def make_join_desc(rows: int, hidden: int, dtype="bf16", post_norm: bool = False, gate="none", gate_act="linear",
                   eps: float = 1e-6, weight_offset: float = 0.0, residual_scale: float = 1.0) -> JoinDesc:
    """gate: "none", "channel" [H], "token" [rows] float32 or "element" [rows, H]; gate_act: "linear" or
    "sigmoid" (or the MOE_GATE_* values)."""
    if isinstance(dtype, str):
        dtype = {"bf16": MOE_BF16, "f32": MOE_F32}[dtype]
    if isinstance(gate, str):
        gate = {"none": MOE_GATE_NONE, "channel": MOE_GATE_CHANNEL, "token": MOE_GATE_TOKEN,
                "element": MOE_GATE_ELEMENT}[gate]
    if isinstance(gate_act, str):
        gate_act = {"linear": MOE_GATE_LINEAR, "sigmoid": MOE_GATE_SIGMOID}[gate_act]
    return JoinDesc(rows, hidden, dtype, int(post_norm), gate, gate_act, eps, weight_offset, residual_scale)


_LIB = None
_VP = ctypes.c_void_p
_DP = ctypes.POINTER(LayerDesc)
_OP = ctypes.c_void_p  # moe_route_opts*, NULL allowed
_PP = ctypes.c_void_p  # moe_packed_experts*
_MP = ctypes.POINTER(MuonDesc)
_JP = ctypes.POINTER(JoinDesc)
_AP = ctypes.c_void_p  # moe_adapters*


def lib() -> ctypes.CDLL:
    """The loaded libmoe.so; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(lib_path):
            raise RuntimeError(f"{lib_path} is not built: run `python -m expert_token_dispatch_amd.build`")
        # torch first: its HIP runtime then serves libmoe too (one runtime per process)
        import torch  # noqa: F401
        L = ctypes.CDLL(lib_path)
        st = ctypes.c_int
        sig = {
            "moe_last_error": (ctypes.c_char_p, []),
            "moe_version": (ctypes.c_char_p, []),
            "moe_ep_local_range": (st, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]),
            "moe_capacity": (ctypes.c_int64, [_DP]),
            "moe_max_pairs": (ctypes.c_int64, [_DP]),
            "moe_workspace_size": (st, [_DP, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
            "moe_profile_events": (st, [ctypes.POINTER(_VP), ctypes.c_int32]),
            "moe_profile_kernel_name": (ctypes.c_char_p, [ctypes.c_int32]),
            "moe_profile_kernel_count": (ctypes.c_int32, []),
            "moe_route": (st, [_DP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
            "moe_dispatch": (st, [_DP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
            "moe_dispatch_noalloc": (st, [_DP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
            "moe_grouped_ffn": (st, [_DP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
            "moe_combine": (st, [_DP, _VP, _VP, _VP, _VP, _VP]),
            "moe_layer_forward": (st, [_DP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                       ctypes.c_size_t, _VP]),
            "moe_route_ex": (st, [_DP, _OP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
            "moe_layer_forward_ex": (st, [_DP, _OP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                          ctypes.c_size_t, _VP]),
            "moe_selection_bias_update": (st, [_DP, _VP, _VP, ctypes.c_float, _VP]),
            "moe_grouped_ffn_train": (st, [_DP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t,
                                           _VP]),
            "moe_layer_forward_train": (st, [_DP, _OP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                             ctypes.c_size_t, _VP]),
            "moe_combine_backward": (st, [_DP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
            "moe_grouped_ffn_backward": (st, [_DP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                              _VP, ctypes.c_size_t, _VP]),
            "moe_route_backward": (st, [_DP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
            "moe_dispatch_backward": (st, [_DP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
            "moe_layer_backward": (st, [_DP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                        ctypes.c_size_t, _VP]),
            "moe_pack_weights": (st, [ctypes.c_int32] * 5 + [_VP] * 4),
            "moe_unpack_weights": (st, [ctypes.c_int32] * 5 + [_VP] * 4),
            "moe_packed_workspace_size": (st, [_DP, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
            "moe_grouped_ffn_packed": (st, [_DP, _VP, _VP, _PP, _VP, _VP, ctypes.c_size_t, _VP]),
            "moe_layer_forward_packed": (st, [_DP, _OP, _VP, _VP, _VP, _PP, _VP, _VP, _VP, _VP, _VP, _VP,
                                              ctypes.c_size_t, _VP]),
            "moe_muon_workspace_size": (st, [_MP, ctypes.POINTER(ctypes.c_size_t)]),
            "moe_orthogonalize": (st, [_MP, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
            "moe_muon_update": (st, [_MP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
            "moe_adapted_workspace_size": (st, [_DP, _AP, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
            "moe_grouped_ffn_adapted": (st, [_DP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _AP, _VP, _VP, ctypes.c_size_t,
                                             _VP]),
            "moe_layer_forward_adapted": (st, [_DP, _OP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _AP, _VP, _VP, _VP, _VP,
                                               _VP, _VP, ctypes.c_size_t, _VP]),
            "moe_block_join": (st, [_JP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
            "moe_join_workspace_size": (st, [_JP, ctypes.POINTER(ctypes.c_size_t)]),
            "moe_block_join_backward": (st, [_JP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                                             ctypes.c_size_t, _VP]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _LIB = L
    return _LIB


def _check(status: int) -> None:
    if status != MOE_OK:
        raise MoeError(status, lib().moe_last_error().decode())


def _p(t) -> Optional[int]:
    """Device pointer of a torch tensor (None stays NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to libmoe must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    return t.data_ptr()


def _s(stream) -> Optional[int]:
    if stream is not None:
        return stream.cuda_stream
    import torch
    # the current stream's handle without a Stream object around it (0.3 instead of 2.7 us a call)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _ws(ws):
    return (None, 0) if ws is None else (_p(ws), ws.numel() * ws.element_size())


# ---- host helpers ------------------------------------------------------------
def moe_last_error() -> str:
    return lib().moe_last_error().decode()


def moe_version() -> str:
    return lib().moe_version().decode()


def moe_ep_local_range(num_experts: int, ep_size: int, rank: int) -> tuple[int, int]:
    b, c = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().moe_ep_local_range(num_experts, ep_size, rank, ctypes.byref(b), ctypes.byref(c)))
    return b.value, c.value


def moe_capacity(d: LayerDesc) -> int:
    return lib().moe_capacity(ctypes.byref(d))


def moe_max_pairs(d: LayerDesc) -> int:
    return lib().moe_max_pairs(ctypes.byref(d))


def moe_workspace_size(d: LayerDesc, stage: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().moe_workspace_size(ctypes.byref(d), stage, ctypes.byref(n)))
    return n.value


def moe_profile_events(handles) -> None:
    """handles: list of hipEvent_t values (ints; None for both of a kernel's pair skips it),
    or None/[] to switch timing off."""
    if not handles:
        _check(lib().moe_profile_events(None, 0))
        return
    arr = (_VP * len(handles))(*handles)
    _check(lib().moe_profile_events(arr, len(handles)))
    moe_profile_events._keep = arr  # the library keeps the handles, not the array


def moe_profile_kernel_count() -> int:
    return lib().moe_profile_kernel_count()


def moe_profile_kernel_name(i: int) -> Optional[str]:
    r = lib().moe_profile_kernel_name(i)
    return None if r is None else r.decode()


# ---- the five stage calls ------------------------------------------------------
def moe_route(d, x, w_router, b_router, topk_ids, topk_w, topk_logit=None, logits_in=None, logits_out=None,
              ws=None, stream=None) -> None:
    wp, wn = _ws(ws)
    _check(lib().moe_route(ctypes.byref(d), _p(x), _p(w_router), _p(b_router), _p(logits_in), _p(logits_out),
                           _p(topk_ids), _p(topk_w), _p(topk_logit), wp, wn, _s(stream)))


def moe_dispatch(d, x, topk_ids, topk_logit, counts, offsets, sorted_pairs, pair_row, x_sorted, num_dropped=None,
                 ws=None, stream=None) -> None:
    wp, wn = _ws(ws)
    _check(lib().moe_dispatch(ctypes.byref(d), _p(x), _p(topk_ids), _p(topk_logit), _p(counts), _p(offsets),
                              _p(sorted_pairs), _p(pair_row), _p(x_sorted), _p(num_dropped), wp, wn, _s(stream)))


def moe_dispatch_noalloc(d, x, topk_ids, topk_logit, counts, offsets, sorted_pairs, pair_row, x_sorted,
                         num_dropped=None, stream=None) -> None:
    _check(lib().moe_dispatch_noalloc(ctypes.byref(d), _p(x), _p(topk_ids), _p(topk_logit), _p(counts), _p(offsets),
                                      _p(sorted_pairs), _p(pair_row), _p(x_sorted), _p(num_dropped), _s(stream)))


def moe_grouped_ffn(d, x_sorted, offsets, w_gate, w_up, w_down, y_sorted, ws=None, stream=None) -> None:
    wp, wn = _ws(ws)
    _check(lib().moe_grouped_ffn(ctypes.byref(d), _p(x_sorted), _p(offsets), _p(w_gate), _p(w_up), _p(w_down),
                                 _p(y_sorted), wp, wn, _s(stream)))


def moe_combine(d, y_sorted, pair_row, topk_w, y, stream=None) -> None:
    _check(lib().moe_combine(ctypes.byref(d), _p(y_sorted), _p(pair_row), _p(topk_w), _p(y), _s(stream)))


def moe_layer_forward(d, x, w_router, b_router, w_gate, w_up, w_down, y, ws, topk_ids_out=None, topk_w_out=None,
                      counts_out=None, num_dropped_out=None, stream=None) -> None:
    wp, wn = _ws(ws)
    _check(lib().moe_layer_forward(ctypes.byref(d), _p(x), _p(w_router), _p(b_router), _p(w_gate), _p(w_up),
                                   _p(w_down), _p(y), _p(topk_ids_out), _p(topk_w_out), _p(counts_out),
                                   _p(num_dropped_out), wp, wn, _s(stream)))


# ---- routing options (glossary "Load balancing and capacity") --------------------
def _opts(opts) -> Optional[int]:
    return None if opts is None else ctypes.addressof(opts)


def moe_route_ex(d, opts, x, w_router, b_router, topk_ids, topk_w, topk_logit=None, logits_in=None, logits_out=None,
                 ws=None, stream=None) -> None:
    wp, wn = _ws(ws)
    _check(lib().moe_route_ex(ctypes.byref(d), _opts(opts), _p(x), _p(w_router), _p(b_router), _p(logits_in),
                              _p(logits_out), _p(topk_ids), _p(topk_w), _p(topk_logit), wp, wn, _s(stream)))


def moe_layer_forward_ex(d, opts, x, w_router, b_router, w_gate, w_up, w_down, y, ws, topk_ids_out=None,
                         topk_w_out=None, counts_out=None, num_dropped_out=None, stream=None) -> None:
    wp, wn = _ws(ws)
    _check(lib().moe_layer_forward_ex(ctypes.byref(d), _opts(opts), _p(x), _p(w_router), _p(b_router), _p(w_gate),
                                      _p(w_up), _p(w_down), _p(y), _p(topk_ids_out), _p(topk_w_out),
                                      _p(counts_out), _p(num_dropped_out), wp, wn, _s(stream)))


def moe_selection_bias_update(d, counts, bias, gamma: float, stream=None) -> None:
    _check(lib().moe_selection_bias_update(ctypes.byref(d), _p(counts), _p(bias), float(gamma), _s(stream)))


# ---- training: the backward pass (Transformers "Expert parallelism", "Token dispatch") ----
def _saved(v) -> Optional[int]:
    return None if v is None else ctypes.addressof(v)


def moe_grouped_ffn_train(d, x_sorted, offsets, w_gate, w_up, w_down, y_sorted, h, gate, up, ws=None,
                          stream=None) -> None:
    wp, wn = _ws(ws)
    _check(lib().moe_grouped_ffn_train(ctypes.byref(d), _p(x_sorted), _p(offsets), _p(w_gate), _p(w_up), _p(w_down),
                                       _p(y_sorted), _p(h), _p(gate), _p(up), wp, wn, _s(stream)))


def moe_layer_forward_train(d, opts, x, w_router, b_router, w_gate, w_up, w_down, y, saved, ws, counts_out=None,
                            num_dropped_out=None, stream=None) -> None:
    wp, wn = _ws(ws)
    _check(lib().moe_layer_forward_train(ctypes.byref(d), _opts(opts), _p(x), _p(w_router), _p(b_router), _p(w_gate),
                                         _p(w_up), _p(w_down), _p(y), _saved(saved), _p(counts_out),
                                         _p(num_dropped_out), wp, wn, _s(stream)))


def moe_combine_backward(d, dy, y_sorted, pair_row, topk_w, dy_sorted, dl, stream=None) -> None:
    _check(lib().moe_combine_backward(ctypes.byref(d), _p(dy), _p(y_sorted), _p(pair_row), _p(topk_w),
                                      _p(dy_sorted), _p(dl), _s(stream)))


def moe_grouped_ffn_backward(d, x_sorted, offsets, w_gate, w_up, w_down, gate, up, h, dy_sorted, dx_sorted, dw_gate,
                             dw_up, dw_down, ws=None, stream=None) -> None:
    wp, wn = _ws(ws)
    _check(lib().moe_grouped_ffn_backward(ctypes.byref(d), _p(x_sorted), _p(offsets), _p(w_gate), _p(w_up),
                                          _p(w_down), _p(gate), _p(up), _p(h), _p(dy_sorted), _p(dx_sorted),
                                          _p(dw_gate), _p(dw_up), _p(dw_down), wp, wn, _s(stream)))


def moe_route_backward(d, x, topk_ids, dl, dw_router, db_router=None, ws=None, stream=None) -> None:
    wp, wn = _ws(ws)
    _check(lib().moe_route_backward(ctypes.byref(d), _p(x), _p(topk_ids), _p(dl), _p(dw_router), _p(db_router),
                                    wp, wn, _s(stream)))


def moe_dispatch_backward(d, dx_sorted, pair_row, topk_ids, dl, w_router, dx, stream=None) -> None:
    _check(lib().moe_dispatch_backward(ctypes.byref(d), _p(dx_sorted), _p(pair_row), _p(topk_ids), _p(dl),
                                       _p(w_router), _p(dx), _s(stream)))


def moe_layer_backward(d, x, w_router, w_gate, w_up, w_down, saved, dy, dx, dw_router, db_router, dw_gate, dw_up,
                       dw_down, ws, stream=None) -> None:
    wp, wn = _ws(ws)
    _check(lib().moe_layer_backward(ctypes.byref(d), _p(x), _p(w_router), _p(w_gate), _p(w_up), _p(w_down),
                                    _saved(saved), _p(dy), _p(dx), _p(dw_router), _p(db_router), _p(dw_gate),
                                    _p(dw_up), _p(dw_down), wp, wn, _s(stream)))


# ---- expert weights in 4 bits ------------------------------------------------------------
def _layout(weight_layout) -> int:
    if isinstance(weight_layout, str):
        return {"out_in": MOE_WEIGHTS_OUT_IN, "in_out": MOE_WEIGHTS_IN_OUT}[weight_layout]
    return weight_layout


def _stack_args(w, codes, scales, weight_layout):
    """The call's sizes, from a weight stack [count, out, in] (or [count, in, out]) and its packed tensors."""
    import torch
    layout = _layout(weight_layout)
    if w.dim() != 3 or w.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("a weight stack is a bfloat16 or float32 tensor of three dimensions")
    count, out, in_ = w.shape if layout == MOE_WEIGHTS_OUT_IN else (w.shape[0], w.shape[2], w.shape[1])
    for name, t, last in (("codes", codes, in_ // 2), ("scales", scales, in_ // 32)):
        if t.dtype != torch.uint8 or tuple(t.shape) != (count, out, last):
            raise ValueError(f"{name} of this stack is a uint8 tensor {(count, out, last)}")
    return count, out, in_, MOE_BF16 if w.dtype == torch.bfloat16 else MOE_F32, layout


def moe_pack_weights(w, codes, scales, weight_layout="out_in", stream=None) -> None:
    """w [count, out, in] (or [count, in, out] for "in_out") into uint8 codes [count, out, in / 2] and
    scales [count, out, in / 32]."""
    _check(lib().moe_pack_weights(*_stack_args(w, codes, scales, weight_layout), _p(w), _p(codes), _p(scales),
                                  _s(stream)))


def moe_unpack_weights(codes, scales, w, weight_layout="out_in", stream=None) -> None:
    _check(lib().moe_unpack_weights(*_stack_args(w, codes, scales, weight_layout), _p(codes), _p(scales), _p(w),
                                    _s(stream)))


def moe_packed_workspace_size(d: LayerDesc, stage: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().moe_packed_workspace_size(ctypes.byref(d), stage, ctypes.byref(n)))
    return n.value


def _packed(d, v) -> Optional[int]:
    """The struct's address; its tensors have to be the stacks that d describes, since the kernels
    take every extent from d."""
    import torch
    if v is None:
        return None
    t = getattr(v, "_tensors", None)  # none: a struct of the caller's own pointers
    for name, out, in_ in (("gate", d.intermediate, d.hidden), ("up", d.intermediate, d.hidden),
                           ("down", d.hidden, d.intermediate)):
        for field, last in ((name + "_codes", in_ // 2), (name + "_scales", in_ // 32)):
            want = (d.local_count, out, last)
            if t is not None and (t[field].dtype != torch.uint8 or tuple(t[field].shape) != want):
                raise ValueError(f"{field} of this layer is a uint8 tensor {want}")
    return ctypes.addressof(v)


def moe_grouped_ffn_packed(d, x_sorted, offsets, packed, y_sorted, ws=None, stream=None) -> None:
    pk = _packed(d, packed)
    wp, wn = _ws(ws)
    _check(lib().moe_grouped_ffn_packed(ctypes.byref(d), _p(x_sorted), _p(offsets), pk, _p(y_sorted), wp, wn,
                                        _s(stream)))


def moe_layer_forward_packed(d, opts, x, w_router, b_router, packed, y, ws, topk_ids_out=None, topk_w_out=None,
                             counts_out=None, num_dropped_out=None, stream=None) -> None:
    pk = _packed(d, packed)
    wp, wn = _ws(ws)
    _check(lib().moe_layer_forward_packed(ctypes.byref(d), _opts(opts), _p(x), _p(w_router), _p(b_router), pk, _p(y),
                                          _p(topk_ids_out), _p(topk_w_out), _p(counts_out), _p(num_dropped_out), wp, wn,
                                          _s(stream)))


# ---- training: the weight update -----------------------------------------------------------
def moe_muon_workspace_size(m: MuonDesc) -> int:
    n = ctypes.c_size_t()
    _check(lib().moe_muon_workspace_size(ctypes.byref(m), ctypes.byref(n)))
    return n.value


def _muon_shapes(m, f32, **tensors):
    import torch
    for name, t in tensors.items():
        want = torch.float32 if name in f32 or m.dtype == MOE_F32 else torch.bfloat16
        if t is not None and (tuple(t.shape) != (m.count, m.rows, m.cols) or t.dtype != want):
            raise ValueError(f"{name} of this update is a {want} tensor {(m.count, m.rows, m.cols)}")


def moe_orthogonalize(m, g, o, ws, stream=None) -> None:
    _muon_shapes(m, (), g=g, o=o)
    wp, wn = _ws(ws)
    _check(lib().moe_orthogonalize(ctypes.byref(m), _p(g), _p(o), wp, wn, _s(stream)))


def moe_muon_update(m, grad, momentum, weight, ws, master=None, stream=None) -> None:
    _muon_shapes(m, ("momentum", "master"), grad=grad, momentum=momentum, weight=weight, master=master)
    wp, wn = _ws(ws)
    _check(lib().moe_muon_update(ctypes.byref(m), _p(grad), _p(momentum), _p(master), _p(weight), wp, wn, _s(stream)))


def _expect(what, items) -> None:
    """(name, tensor, shape, type) that a call describes by its descriptor: the kernels take every extent
    from there, and run on the current device."""
    dev = -1
    for name, t, shape, dtype in items:
        if t is None:
            continue
        if t.shape != shape or t.dtype is not dtype:
            raise ValueError(f"{name} of this {what} is a {dtype} tensor {tuple(shape)}")
        d = t.get_device()
        if d != dev:  # the first one, or one elsewhere than those before
            import torch
            if d >= 0 and (dev >= 0 or d != torch.cuda.current_device()):
                raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
            dev = d


# ---- low-rank adapters beside the experts' weights -------------------------------------------
def _adapters(d, v) -> Optional[int]:
    """The struct's address; its tensors have to be the stacks that d describes, since the kernels
    take every extent from d and the struct."""
    import torch
    if v is None:
        return None
    t = getattr(v, "_tensors", None)  # none: a struct of the caller's own pointers
    if t is not None:
        dt = torch.bfloat16 if d.dtype == MOE_BF16 else torch.float32
        n, L, R, H, I = v.count, d.local_count, v.rank, d.hidden, d.intermediate
        on_gpu = next(iter(t.values())).get_device() >= 0
        key = (dt, n, L, R, H, I, torch.cuda.current_device() if on_gpu else None)
        if v._fits != key:
            shapes = {"scale": ((n,), torch.float32)}
            for name, out, in_ in (("gate", I, H), ("up", I, H), ("down", H, I)):
                shapes[name + "_a"], shapes[name + "_b"] = ((n, L, R, in_), dt), ((n, L, out, R), dt)
            if set(t) - set(shapes):
                raise ValueError(f"adapters have no {sorted(set(t) - set(shapes))}")
            _expect("layer's adapters", [(k, x, *shapes[k]) for k, x in t.items()])
            v._fits = key  # the tensors are the struct's own: looked at once for each kind of layer and device
    return ctypes.addressof(v)


def moe_adapted_workspace_size(d: LayerDesc, adapters, stage: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().moe_adapted_workspace_size(ctypes.byref(d), _adapters(d, adapters), stage, ctypes.byref(n)))
    return n.value


def _ids(d, adapter_ids) -> None:
    import torch
    _expect("layer", (("adapter_ids", adapter_ids, (d.num_tokens,), torch.int32),))


def moe_grouped_ffn_adapted(d, x_sorted, offsets, sorted_pairs, adapter_ids, w_gate, w_up, w_down, adapters, y_sorted,
                            ws, stream=None) -> None:
    ad = _adapters(d, adapters)
    _ids(d, adapter_ids)
    wp, wn = _ws(ws)
    _check(lib().moe_grouped_ffn_adapted(ctypes.byref(d), _p(x_sorted), _p(offsets), _p(sorted_pairs), _p(adapter_ids),
                                         _p(w_gate), _p(w_up), _p(w_down), ad, _p(y_sorted), wp, wn, _s(stream)))


def moe_layer_forward_adapted(d, opts, x, adapter_ids, w_router, b_router, w_gate, w_up, w_down, adapters, y, ws,
                              topk_ids_out=None, topk_w_out=None, counts_out=None, num_dropped_out=None,
                              stream=None) -> None:
    ad = _adapters(d, adapters)
    _ids(d, adapter_ids)
    wp, wn = _ws(ws)
    _check(lib().moe_layer_forward_adapted(ctypes.byref(d), _opts(opts), _p(x), _p(adapter_ids), _p(w_router),
                                           _p(b_router), _p(w_gate), _p(w_up), _p(w_down), ad, _p(y), _p(topk_ids_out),
                                           _p(topk_w_out), _p(counts_out), _p(num_dropped_out), wp, wn, _s(stream)))


# ---- the join with the residual stream ------------------------------------------------------
def _join_items(j, gate):
    """Shapes and types of a join's rows, weights and gate."""
    import torch
    dt = torch.bfloat16 if j.dtype == MOE_BF16 else torch.float32
    T, H, k = j.rows, j.hidden, j.gate_kind
    rows, gdt = (T, H), dt
    shape = (H,) if k == MOE_GATE_CHANNEL else rows
    if k == MOE_GATE_TOKEN:
        shape, gdt = (T,), torch.float32
    elif k == MOE_GATE_NONE and gate is not None:  # the library refuses it
        shape, gdt = gate.shape, gate.dtype
    return dt, rows, (H,), shape, gdt


def moe_block_join(j, x, y, gate, w_post, w_pre, z, h, stream=None) -> None:
    dt, rows, chan, shape, gdt = _join_items(j, gate)
    _expect("join", (("x", x, rows, dt), ("y", y, rows, dt), ("gate", gate, shape, gdt), ("w_post", w_post, chan, dt),
                     ("w_pre", w_pre, chan, dt), ("z", z, rows, dt), ("h", h, rows, dt)))
    _check(lib().moe_block_join(ctypes.byref(j), _p(x), _p(y), _p(gate), _p(w_post), _p(w_pre), _p(z), _p(h),
                                _s(stream)))


def moe_join_workspace_size(j: JoinDesc) -> int:
    n = ctypes.c_size_t()
    _check(lib().moe_join_workspace_size(ctypes.byref(j), ctypes.byref(n)))
    return n.value


def moe_block_join_backward(j, z, y, gate, w_post, w_pre, dz, dh, dx, dy, dgate, dw_post, dw_pre, ws,
                            stream=None) -> None:
    dt, rows, chan, shape, gdt = _join_items(j, gate)
    _expect("join", (("z", z, rows, dt), ("y", y, rows, dt), ("gate", gate, shape, gdt), ("w_post", w_post, chan, dt),
                     ("w_pre", w_pre, chan, dt), ("dz", dz, rows, dt), ("dh", dh, rows, dt), ("dx", dx, rows, dt),
                     ("dy", dy, rows, dt), ("dgate", dgate, shape, gdt), ("dw_post", dw_post, chan, dt),
                     ("dw_pre", dw_pre, chan, dt)))
    wp, wn = _ws(ws)
    _check(lib().moe_block_join_backward(ctypes.byref(j), _p(z), _p(y), _p(gate), _p(w_post), _p(w_pre), _p(dz),
                                         _p(dh), _p(dx), _p(dy), _p(dgate), _p(dw_post), _p(dw_pre), wp, wn,
                                         _s(stream)))
