"""Adapters beside the experts without a GPU: the oracle against merged weights, workspaces, and
refused calls (none of them reaches a kernel)."""

import ctypes

import numpy as np
import pytest

import expert_token_dispatch_amd as etd
from expert_token_dispatch_amd import _lib as L
from oracle import adapters as oa

PAIRS = ("gate_a", "gate_b", "up_a", "up_b", "down_a", "down_b")


def test_oracle_is_the_experts_with_merged_weights():
    """One adapter for every row: the same as the experts whose weights are W + scale B A."""
    rng = np.random.default_rng(1)
    Lc, H, I, R, n = 3, 8, 16, 4, 2
    x, off, ids = rng.standard_normal((7, H)), [0, 4, 4, 7], [1] * 7
    w = {"gate": rng.standard_normal((Lc, I, H)), "up": rng.standard_normal((Lc, I, H)), "down": rng.standard_normal((Lc, H, I))}
    ad = {}
    for name, N, K in (("gate", I, H), ("up", I, H), ("down", H, I)):
        ad[name + "_a"], ad[name + "_b"] = rng.standard_normal((n, Lc, R, K)), rng.standard_normal((n, Lc, N, R))
    s = np.array([9.0, 0.5])
    merged = {k: v + 0.5 * np.einsum("lnr,lrk->lnk", ad[k + "_b"][1], ad[k + "_a"][1]) for k, v in w.items()}
    np.testing.assert_allclose(oa.grouped_ffn(x, off, ids, w, ad, s), oa.grouped_ffn(x, off, [-1] * 7, merged, {}, s), rtol=1e-10)
    none = oa.grouped_ffn(x, off, [2, -1, 7, -3, 2, 2, 2], w, ad, s)
    np.testing.assert_allclose(none, oa.grouped_ffn(x, off, ids, w, {}, s), rtol=1e-12)


def _struct(**over):
    a = dict(count=3, rank=16, scale=256, **{n: 256 for n in PAIRS})
    a.update(over)
    return L.Adapters(*[a[n] for n, _ in L.Adapters._fields_])


STRUCT_BAD = [
    dict(count=0), dict(count=65536), dict(rank=0), dict(rank=12), dict(rank=136), dict(rank=-8), dict(gate_a=None),
    dict(gate_b=None), dict(up_b=None), dict(down_a=None), {n: None for n in PAIRS},
]
# refused by the calls alone: the size asks only which pointers are NULL
CALL_BAD = STRUCT_BAD + [dict(gate_a=264), dict(up_b=260), dict(down_b=258), dict(scale=258)]


@pytest.mark.parametrize("over", CALL_BAD)
def test_adapters_refused(over):
    d, lib, a, n = etd.make_desc(4, 64, 128, 8, 2), L.lib(), _struct(**over), ctypes.c_size_t()
    at = ctypes.addressof(a)
    if over in STRUCT_BAD:
        assert lib.moe_adapted_workspace_size(ctypes.byref(d), at, L.MOE_STAGE_FFN, ctypes.byref(n)) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_grouped_ffn_adapted(ctypes.byref(d), *[256] * 7, at, 256, 256, 1 << 40, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_layer_forward_adapted(ctypes.byref(d), None, 256, 256, 256, None, 256, 256, 256, at, 256, None, None, None,
                                         None, 256, 1 << 40, None) == L.MOE_ERR_INVALID_ARG
    assert "adapters" in L.moe_last_error() or "scale" in L.moe_last_error()


def test_null_adapters_and_unknown_stages():
    d, lib, n = etd.make_desc(4, 64, 128, 8, 2), L.lib(), ctypes.c_size_t()
    a = _struct()
    at = ctypes.addressof(a)
    assert lib.moe_adapted_workspace_size(ctypes.byref(d), None, L.MOE_STAGE_FFN, ctypes.byref(n)) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_adapted_workspace_size(ctypes.byref(d), at, L.MOE_STAGE_ROUTE, ctypes.byref(n)) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_adapted_workspace_size(ctypes.byref(d), at, L.MOE_STAGE_FFN, None) == L.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("H,I", [((1 << 22) + 8, 64), (64, (1 << 22) + 8)])
def test_the_widest_rows_are_unsupported(H, I):
    d, a, n = etd.make_desc(4, H, I, 8, 2), _struct(), ctypes.c_size_t()
    at = ctypes.addressof(a)
    assert L.lib().moe_adapted_workspace_size(ctypes.byref(d), at, L.MOE_STAGE_FFN, ctypes.byref(n)) == L.MOE_ERR_UNSUPPORTED
    assert L.lib().moe_grouped_ffn_adapted(ctypes.byref(d), *[256] * 7, at, 256, 256, 1 << 60, None) == L.MOE_ERR_UNSUPPORTED


def test_more_pairs_than_a_launch_holds_are_unsupported():
    d, a, n = etd.make_desc((1 << 26) + 1, 64, 64, 8, 2), _struct(), ctypes.c_size_t()
    at = ctypes.addressof(a)
    assert L.lib().moe_adapted_workspace_size(ctypes.byref(d), at, L.MOE_STAGE_FFN, ctypes.byref(n)) == L.MOE_ERR_UNSUPPORTED
    assert L.lib().moe_grouped_ffn_adapted(ctypes.byref(d), *[256] * 7, at, 256, 256, 1 << 60, None) == L.MOE_ERR_UNSUPPORTED


# x_sorted, offsets, sorted_pairs, adapter_ids, w_gate, w_up, w_down, (adapters), y_sorted, ws
@pytest.mark.parametrize("arg", [0, 1, 2, 3, 4, 5, 6, 8])
@pytest.mark.parametrize("value", [None, 258])
def test_ffn_arguments_refused(arg, value):
    a = _struct()
    args = [256] * 7 + [ctypes.addressof(a), 256, 256]
    args[arg] = value
    d = etd.make_desc(4, 64, 128, 8, 2)
    assert L.lib().moe_grouped_ffn_adapted(ctypes.byref(d), *args, 1 << 40, None) == L.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_workspaces(dtype):
    d, lib = etd.make_desc(500, 64, 128, 8, 2, dtype=dtype), L.lib()
    width = 4   # float32, or two bfloat16
    for stage in (L.MOE_STAGE_FFN, L.MOE_STAGE_LAYER):
        plain = etd.moe_workspace_size(d, stage)
        full = etd.moe_adapted_workspace_size(d, _struct(), stage)
        down = etd.moe_adapted_workspace_size(d, _struct(gate_a=None, gate_b=None, up_a=None, up_b=None), stage)
        assert full - plain >= 1000 * (3 * 16 * width + 4)
        assert full - down == 1000 * 2 * 16 * width  # a multiple of 256
    need = etd.moe_adapted_workspace_size(d, _struct(), L.MOE_STAGE_FFN)
    a = _struct()
    args = [256] * 7 + [ctypes.addressof(a), 256]
    assert lib.moe_grouped_ffn_adapted(ctypes.byref(d), *args, 256, need - 1, None) == L.MOE_ERR_WORKSPACE
    assert lib.moe_grouped_ffn_adapted(ctypes.byref(d), *args, None, need, None) == L.MOE_ERR_WORKSPACE


def test_no_tokens_is_no_work():
    d, a = etd.make_desc(0, 64, 128, 8, 2), _struct()
    at = ctypes.addressof(a)
    assert L.lib().moe_grouped_ffn_adapted(ctypes.byref(d), *[None] * 7, at, None, None, 0, None) == L.MOE_OK
    assert L.lib().moe_layer_forward_adapted(ctypes.byref(d), None, *[None] * 7, at, *[None] * 6, 0, None) == L.MOE_OK


def test_the_binding_refuses_other_stacks():
    torch = pytest.importorskip("torch")
    d = etd.make_desc(4, 64, 128, 8, 2)

    def make(**over):
        bf = torch.bfloat16
        t = {"gate_a": torch.zeros(3, 8, 16, 64, dtype=bf), "gate_b": torch.zeros(3, 8, 128, 16, dtype=bf),
             "down_a": torch.zeros(3, 8, 16, 128, dtype=bf), "down_b": torch.zeros(3, 8, 64, 16, dtype=bf),
             "scale": torch.zeros(3)}
        t.update(over)
        t = {k: v for k, v in t.items() if v is not None}
        a = next(v for k, v in t.items() if k.endswith("_a"))
        v = L.Adapters(a.shape[0], a.shape[2], *[256 if n in t else None for n, _ in L.Adapters._fields_[2:]])
        v._tensors, v._fits = t, None
        return v
    assert L._adapters(d, make()) and etd.moe_adapted_workspace_size(d, make(), L.MOE_STAGE_FFN)
    for bad in (dict(gate_b=torch.zeros(3, 8, 64, 16, dtype=torch.bfloat16)), dict(down_a=torch.zeros(3, 8, 16, 128)),
                dict(scale=torch.zeros(2)), dict(scale=torch.zeros(3, dtype=torch.bfloat16)), dict(extra=torch.zeros(1)),
                dict(down_b=torch.zeros(2, 8, 64, 16, dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match="adapters"):
            L._adapters(d, make(**bad))
    with pytest.raises(ValueError, match="adapters"):
        L._adapters(etd.make_desc(4, 64, 136, 8, 2), make())
    with pytest.raises(ValueError, match="at least one projection"):
        etd.make_adapters({"scale": torch.zeros(3)})
    with pytest.raises(ValueError, match="adapter_ids"):
        L._ids(d, torch.zeros(5, dtype=torch.int32))
    with pytest.raises(ValueError, match="adapter_ids"):
        L._ids(d, torch.zeros(4, dtype=torch.int64))


class _OnGpu0:
    """What the binding asks of a tensor on the first GPU."""

    def __init__(self, t):
        self.shape, self.dtype, self.device = t.shape, t.dtype, "cuda:0"

    def get_device(self):
        return 0


def test_the_binding_looks_again_on_another_device_and_after_a_changed_count(monkeypatch):
    torch = pytest.importorskip("torch")
    d, bf = etd.make_desc(4, 64, 128, 8, 2), torch.bfloat16
    v = L.Adapters(3, 16, None, None, None, None, None, 256, 256)
    v._tensors = {"down_a": _OnGpu0(torch.empty(3, 8, 16, 128, dtype=bf)), "down_b": _OnGpu0(torch.empty(3, 8, 64, 16, dtype=bf))}
    v._fits = None
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert L._adapters(d, v) and L._adapters(d, v)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device is cuda:1"):
        L._adapters(d, v)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert L._adapters(d, v)
    v.count = 4
    with pytest.raises(ValueError, match="adapters"):
        L._adapters(d, v)
    v.count, v.rank = 3, 24
    with pytest.raises(ValueError, match="adapters"):
        L._adapters(d, v)
