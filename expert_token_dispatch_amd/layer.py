"""Buffer management around the C ABI: one MoE layer's device tensors, and the join around it.

MoELayer owns the weights (torch device tensors in the library's layout), the
workspaces, and the stage outputs, and calls the libmoe entry points on the
current torch stream.  It computes nothing itself.  A layer's calls share its
workspaces, captured ones too: on several streams each has to wait for the one
before, or take a MoELayer of its own around the same weights.
"""

from __future__ import annotations

from typing import Optional

import numpy as np
import torch

from . import _lib as L


def to_device(a: Optional[np.ndarray], dtype: str, device="cuda") -> Optional[torch.Tensor]:
    """Host array -> device tensor.  bf16 arrays arrive as uint16 bit patterns."""
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    if dtype == "bf16" and a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).to(device).view(torch.bfloat16)
    return torch.from_numpy(a).to(device)


def torch_dtype(dtype: str):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


class MoELayer:
    def __init__(self, desc: L.LayerDesc, w_router, b_router, w_gate, w_up, w_down, device="cuda"):
        self.desc = desc
        self.device = torch.device(device)
        self.dtype = "bf16" if desc.dtype == L.MOE_BF16 else "f32"
        self.w_router, self.b_router = w_router, b_router
        self.w_gate, self.w_up, self.w_down = w_gate, w_up, w_down
        self.max_pairs = L.moe_max_pairs(desc)
        self._ws = {}

    @classmethod
    def from_host(cls, desc: L.LayerDesc, inp: dict, device="cuda") -> "MoELayer":
        dt = "bf16" if desc.dtype == L.MOE_BF16 else "f32"
        return cls(desc, to_device(inp["w_router"], dt, device), to_device(inp.get("b_router"), "f32", device),
                   to_device(inp["w_gate"], dt, device), to_device(inp["w_up"], dt, device),
                   to_device(inp["w_down"], dt, device), device)

    def workspace(self, stage: int) -> Optional[torch.Tensor]:
        if stage not in self._ws:
            n = L.moe_workspace_size(self.desc, stage)
            # 256-byte aligned: torch's caching allocator hands out 512-byte aligned blocks
            self._ws[stage] = torch.empty(max(n, 1), dtype=torch.uint8, device=self.device) if n else None
        return self._ws[stage]

    def _empty(self, shape, dtype):
        return torch.empty(shape, dtype=dtype, device=self.device)

    # ---- stages ------------------------------------------------------------
    def route(self, x, logits_in=None, want_logits=False, want_topk_logit=None, opts=None):
        d = self.desc
        T, k, E = d.num_tokens, d.top_k, d.num_experts
        out = {"topk_ids": self._empty((T, k), torch.int32), "topk_w": self._empty((T, k), torch.float32)}
        if want_topk_logit is None:
            want_topk_logit = d.capacity_factor > 0
        out["topk_logit"] = self._empty((T, k), torch.float32) if want_topk_logit else None
        out["logits"] = self._empty((T, E), torch.float32) if want_logits else None
        L.moe_route_ex(d, opts, x, self.w_router, self.b_router, out["topk_ids"], out["topk_w"], out["topk_logit"],
                       logits_in=logits_in, logits_out=out["logits"], ws=self.workspace(L.MOE_STAGE_ROUTE))
        return out

    def dispatch(self, x, topk_ids, topk_logit=None):
        d = self.desc
        T, k, E, Lc, H = d.num_tokens, d.top_k, d.num_experts, d.local_count, d.hidden
        pm = max(self.max_pairs, 1)
        out = {
            "counts": self._empty((E,), torch.int32),
            "offsets": self._empty((Lc + 1,), torch.int32),
            "sorted_pairs": torch.full((pm,), -1, dtype=torch.int32, device=self.device),
            "pair_row": self._empty((T * k,), torch.int32),
            "x_sorted": self._empty((pm, H), x.dtype),
            "num_dropped": torch.zeros((1,), dtype=torch.int64, device=self.device),
        }
        L.moe_dispatch(d, x, topk_ids, topk_logit, out["counts"], out["offsets"], out["sorted_pairs"],
                       out["pair_row"], out["x_sorted"], out["num_dropped"], ws=self.workspace(L.MOE_STAGE_DISPATCH))
        return out

    def grouped_ffn(self, x_sorted, offsets):
        d = self.desc
        y_sorted = self._empty((max(self.max_pairs, 1), d.hidden), x_sorted.dtype)
        L.moe_grouped_ffn(d, x_sorted, offsets, self.w_gate, self.w_up, self.w_down, y_sorted,
                          ws=self.workspace(L.MOE_STAGE_FFN))
        return y_sorted

    def combine(self, y_sorted, pair_row, topk_w):
        d = self.desc
        y = self._empty((d.num_tokens, d.hidden), y_sorted.dtype)
        L.moe_combine(d, y_sorted, pair_row, topk_w, y)
        return y

    def forward(self, x, y=None, topk_ids_out=None, topk_w_out=None, counts_out=None, num_dropped_out=None,
                opts=None):
        """opts: an L.RouteOpts (selection bias, groups per token) or None."""
        d = self.desc
        if y is None:
            y = self._empty((d.num_tokens, d.hidden), x.dtype)
        L.moe_layer_forward_ex(d, opts, x, self.w_router, self.b_router, self.w_gate, self.w_up, self.w_down, y,
                               self.workspace(L.MOE_STAGE_LAYER), topk_ids_out, topk_w_out, counts_out,
                               num_dropped_out)
        return y

    def update_selection_bias(self, counts, bias, gamma):
        """One balancing step on the float32 [E] bias from a batch's [E] int32 expert loads."""
        L.moe_selection_bias_update(self.desc, counts, bias, gamma)
        return bias

    # ---- experts in 4 bits -----------------------------------------------------
    def pack_experts(self) -> L.PackedExperts:
        """The experts' weights as 4-bit codes with a scale per 32 inputs, in new tensors."""
        d = self.desc
        Lc, H, I = d.local_count, d.hidden, d.intermediate
        t = {}
        for name, w, out, in_ in (("gate", self.w_gate, I, H), ("up", self.w_up, I, H), ("down", self.w_down, H, I)):
            codes, scales = t[name + "_codes"], t[name + "_scales"] = (
                self._empty((Lc, out, in_ // 2), torch.uint8), self._empty((Lc, out, in_ // 32), torch.uint8))
            L.moe_pack_weights(w, codes, scales, weight_layout=d.weight_layout)
        return L.make_packed_experts(t)

    def packed_workspace(self, stage: int) -> torch.Tensor:
        key = ("packed", stage)
        if key not in self._ws:
            n = L.moe_packed_workspace_size(self.desc, stage)
            self._ws[key] = torch.empty(max(n, 1), dtype=torch.uint8, device=self.device)
        return self._ws[key]

    def grouped_ffn_packed(self, x_sorted, offsets, packed):
        """grouped_ffn on the weights that `packed` (pack_experts) stands for."""
        d = self.desc
        y_sorted = self._empty((max(self.max_pairs, 1), d.hidden), x_sorted.dtype)
        L.moe_grouped_ffn_packed(d, x_sorted, offsets, packed, y_sorted, ws=self.packed_workspace(L.MOE_STAGE_FFN))
        return y_sorted

    def forward_packed(self, x, packed, y=None, topk_ids_out=None, topk_w_out=None, counts_out=None,
                       num_dropped_out=None, opts=None):
        """forward on packed experts; the layer's own expert weights are not read."""
        d = self.desc
        if y is None:
            y = self._empty((d.num_tokens, d.hidden), x.dtype)
        L.moe_layer_forward_packed(d, opts, x, self.w_router, self.b_router, packed, y,
                                   self.packed_workspace(L.MOE_STAGE_LAYER), topk_ids_out, topk_w_out, counts_out,
                                   num_dropped_out)
        return y

    # ---- adapters of many requests beside the experts' weights --------------------
    def adapted_workspace(self, adapters, stage: int) -> torch.Tensor:
        has = tuple(getattr(adapters, n + "_a") is not None for n in L.ADAPTED)
        key = ("adapted", stage, adapters.rank, has)
        if key not in self._ws:
            n = L.moe_adapted_workspace_size(self.desc, adapters, stage)
            self._ws[key] = torch.empty(max(n, 1), dtype=torch.uint8, device=self.device)
        return self._ws[key]

    def grouped_ffn_adapted(self, x_sorted, offsets, sorted_pairs, adapters, adapter_ids):
        """grouped_ffn with each token's adapter (L.make_adapters; adapter_ids [T] int32, -1 for none)."""
        d = self.desc
        y_sorted = self._empty((max(self.max_pairs, 1), d.hidden), x_sorted.dtype)
        L.moe_grouped_ffn_adapted(d, x_sorted, offsets, sorted_pairs, adapter_ids, self.w_gate, self.w_up, self.w_down,
                                  adapters, y_sorted, self.adapted_workspace(adapters, L.MOE_STAGE_FFN))
        return y_sorted

    def forward_adapted(self, x, adapters, adapter_ids, y=None, topk_ids_out=None, topk_w_out=None, counts_out=None,
                        num_dropped_out=None, opts=None):
        """forward with each token's adapter beside the experts' weights."""
        d = self.desc
        if y is None:
            y = self._empty((d.num_tokens, d.hidden), x.dtype)
        L.moe_layer_forward_adapted(d, opts, x, adapter_ids, self.w_router, self.b_router, self.w_gate, self.w_up,
                                    self.w_down, adapters, y, self.adapted_workspace(adapters, L.MOE_STAGE_LAYER),
                                    topk_ids_out, topk_w_out, counts_out, num_dropped_out)
        return y

    def staged(self, x, logits_in=None, opts=None):
        """The four stage calls one after another; returns every intermediate."""
        r = self.route(x, logits_in=logits_in, want_logits=True, want_topk_logit=True, opts=opts)
        dd = self.dispatch(x, r["topk_ids"], r["topk_logit"])
        ys = self.grouped_ffn(dd["x_sorted"], dd["offsets"])
        y = self.combine(ys, dd["pair_row"], r["topk_w"])
        return {**r, **dd, "y_sorted": ys, "y": y}

    # ---- training (Transformers "Expert parallelism", "Token dispatch") ----------
    def saved_buffers(self, x_dtype) -> dict:
        """Device buffers for the intermediates the training forward keeps."""
        d = self.desc
        T, k, Lc, H, I = d.num_tokens, d.top_k, d.local_count, d.hidden, d.intermediate
        pm = max(self.max_pairs, 1)
        return {
            "topk_ids": self._empty((max(T, 1), k), torch.int32),
            "topk_w": self._empty((max(T, 1), k), torch.float32),
            "offsets": self._empty((Lc + 1,), torch.int32),
            "pair_row": self._empty((max(T * k, 1),), torch.int32),
            "x_sorted": self._empty((pm, H), x_dtype),
            "gate": self._empty((pm, I), x_dtype),
            "up": self._empty((pm, I), x_dtype),
            "h": self._empty((pm, I), x_dtype),
            "y_sorted": self._empty((pm, H), x_dtype),
        }

    def forward_train(self, x, opts=None, saved=None, y=None, counts_out=None, num_dropped_out=None):
        """The layer forward that keeps what the backward needs; returns (y, saved)."""
        d = self.desc
        if y is None:
            y = self._empty((d.num_tokens, d.hidden), x.dtype)
        if saved is None:
            saved = L.make_saved(self.saved_buffers(x.dtype))
        L.moe_layer_forward_train(d, opts, x, self.w_router, self.b_router, self.w_gate, self.w_up, self.w_down, y,
                                  saved, self.workspace(L.MOE_STAGE_LAYER), counts_out, num_dropped_out)
        return y, saved

    def grad_buffers(self, x_dtype) -> dict:
        d = self.desc
        T, E, Lc, H, I = d.num_tokens, d.num_experts, d.local_count, d.hidden, d.intermediate
        return {
            "dx": self._empty((max(T, 1), H), x_dtype),
            "dw_router": self._empty((E, H), x_dtype),
            "db_router": self._empty((E,), torch.float32) if self.b_router is not None else None,
            # the weight gradients take the weights' layout
            "dw_gate": self._empty(tuple(self.w_gate.shape), x_dtype),
            "dw_up": self._empty(tuple(self.w_up.shape), x_dtype),
            "dw_down": self._empty(tuple(self.w_down.shape), x_dtype),
        }

    def backward(self, x, saved, dy, grads=None) -> dict:
        """Gradients of the layer given dy, from forward_train's saved intermediates."""
        if grads is None:
            grads = self.grad_buffers(dy.dtype)
        L.moe_layer_backward(self.desc, x, self.w_router, self.w_gate, self.w_up, self.w_down, saved, dy,
                             grads["dx"], grads["dw_router"], grads["db_router"], grads["dw_gate"], grads["dw_up"],
                             grads["dw_down"], self.workspace(L.MOE_STAGE_LAYER_BACKWARD))
        return grads

    def staged_backward(self, x, saved, dy) -> dict:
        """The four backward stage calls one after another; returns every intermediate."""
        d = self.desc
        T, k, H = d.num_tokens, d.top_k, d.hidden
        pm = max(self.max_pairs, 1)
        t = saved._tensors
        g = self.grad_buffers(dy.dtype)
        dys = self._empty((pm, H), dy.dtype)
        dl = self._empty((max(T, 1), k), torch.float32)
        L.moe_combine_backward(d, dy, t["y_sorted"], t["pair_row"], t["topk_w"], dys, dl)
        dxs = self._empty((pm, H), dy.dtype)
        L.moe_grouped_ffn_backward(d, t["x_sorted"], t["offsets"], self.w_gate, self.w_up, self.w_down, t["gate"],
                                   t["up"], t["h"], dys, dxs, g["dw_gate"], g["dw_up"], g["dw_down"],
                                   ws=self.workspace(L.MOE_STAGE_FFN_BACKWARD))
        L.moe_route_backward(d, x, t["topk_ids"], dl, g["dw_router"], g["db_router"],
                             ws=self.workspace(L.MOE_STAGE_ROUTE_BACKWARD))
        L.moe_dispatch_backward(d, dxs, t["pair_row"], t["topk_ids"], dl, self.w_router, g["dx"])
        return {**g, "dy_sorted": dys, "dl": dl, "dx_sorted": dxs}

    # ---- the weight update -------------------------------------------------------
    MUON_WEIGHTS = ("w_gate", "w_up", "w_down")

    def muon_state(self, master: bool = True) -> dict:
        """Momentum (zeros) of the expert weights and, for bf16 layers with `master`, float32 copies of them."""
        names = self.MUON_WEIGHTS
        st = {n: torch.zeros(getattr(self, n).shape, dtype=torch.float32, device=self.device) for n in names}
        m = {n: getattr(self, n).float() for n in names} if master and self.dtype == "bf16" else {}
        return {"momentum": st, "master": m}

    def muon_update(self, grads: dict, state: dict, lr: float, momentum: float = 0.95, nesterov: bool = True,
                    weight_decay: float = 0.0, update_scale: Optional[float] = None, steps: int = 5):
        """One Muon step on the expert weights, in place, from backward()'s gradients and muon_state().
        update_scale: factor of the orthogonalised update, by default 0.2 sqrt(longer side), which
        gives its entries the size of an Adam step's."""
        descs = {}
        for n in self.MUON_WEIGHTS:
            shape = getattr(self, n).shape
            scale = 0.2 * max(shape[1:]) ** 0.5 if update_scale is None else update_scale
            descs[n] = L.make_muon_desc(*shape, dtype=self.dtype, steps=steps, momentum=momentum, nesterov=nesterov, lr=lr,
                                        update_scale=scale, weight_decay=weight_decay)
        key = ("muon", steps)  # one workspace for the three stacks, which follow each other; never replaced
        if key not in self._ws:
            size = max(L.moe_muon_workspace_size(m) for m in descs.values())
            self._ws[key] = torch.empty(size, dtype=torch.uint8, device=self.device)
        ws = self._ws[key]
        for n, m in descs.items():
            L.moe_muon_update(m, grads["d" + n], state["momentum"][n], getattr(self, n), ws, master=state["master"].get(n))


class BlockJoin:
    """What stands between a block and the next: the norm of the block's output, its gate and scale, the
    residual sum, and the next block's norm.  Owns the norm weights; its calls share no buffers, so that
    several may run at once.

    w_post: the norm after the block (post_norm without it: a norm of factor 1); w_pre: the next block's
    norm (next_norm without it: a norm of factor 1).  gate: "none", "channel", "token" or "element"; the
    gate itself is an argument of the calls, since all kinds but "channel" depend on the tokens."""

    def __init__(self, hidden: int, dtype: str = "bf16", w_post=None, w_pre=None, post_norm: Optional[bool] = None,
                 next_norm: Optional[bool] = None, gate="none", gate_act="linear", eps: float = 1e-6,
                 weight_offset: float = 0.0, residual_scale: float = 1.0, device="cuda"):
        self.hidden, self.dtype, self.device = hidden, dtype, torch.device(device)
        self.w_post, self.w_pre = w_post, w_pre
        self.post_norm = w_post is not None if post_norm is None else post_norm
        self.next_norm = w_pre is not None if next_norm is None else next_norm
        self.gate, self.gate_act = gate, gate_act
        self.eps, self.weight_offset, self.residual_scale = eps, weight_offset, residual_scale

    def desc(self, rows: int, with_block: bool = True) -> L.JoinDesc:
        return L.make_join_desc(rows, self.hidden, self.dtype, post_norm=with_block and self.post_norm,
                                gate=self.gate if with_block else "none", gate_act=self.gate_act, eps=self.eps,
                                weight_offset=self.weight_offset, residual_scale=self.residual_scale)

    def workspace(self, rows: int = (1 << 31) - 1) -> torch.Tensor:
        """A new one for the backward of so many rows, by default of any number.  Each call takes its own: torch's
        allocator keeps what a stream has used for that stream, and a graph's memory for that graph."""
        return torch.empty(L.moe_join_workspace_size(self.desc(rows)), dtype=torch.uint8, device=self.device)

    def forward(self, x, y=None, gate=None, z=None, h=None):
        """(z, h) of the stream x and the block's output y; without y, (x, h): the norm before a first block.
        h is None without a next norm."""
        j = self.desc(x.shape[0], y is not None)
        if z is None and y is not None:
            z = torch.empty_like(x)
        if h is None and self.next_norm:
            h = torch.empty_like(x)
        L.moe_block_join(j, x, y, gate, self.w_post if y is not None else None, self.w_pre, z, h)
        return (x if y is None else z), h

    def backward(self, z, y=None, gate=None, dz=None, dh=None, grads: Optional[dict] = None) -> dict:
        """Gradients dx, and with y also dy, dgate, dw_post, and dw_pre, from those of forward()'s results.
        grads: tensors for them under these names, for exactly those that there are."""
        j = self.desc(z.shape[0], y is not None)
        w_post = self.w_post if y is not None else None
        if grads is None:
            def like(t):
                return None if t is None else torch.empty_like(t)
            grads = {"dx": like(z), "dy": like(y), "dgate": like(gate), "dw_post": like(w_post), "dw_pre": like(self.w_pre)}
        out = [grads.get(n) for n in ("dx", "dy", "dgate", "dw_post", "dw_pre")]
        L.moe_block_join_backward(j, z, y, gate, w_post, self.w_pre, dz, dh, *out, self.workspace(z.shape[0]))
        return grads
