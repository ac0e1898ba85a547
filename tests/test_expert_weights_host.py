"""4-bit expert weights and the weight update without a GPU: every call here is refused
before any work is enqueued, or is a T == 0 no-op."""

import ctypes

import pytest
import torch

import expert_token_dispatch_amd as etd
from expert_token_dispatch_amd import _lib as L


def _packed(**null):
    return L.PackedExperts(*[None if n in null else 256 for n, _ in L.PackedExperts._fields_])


PACK_BAD = [
    (dict(count=0), "INVALID_ARG"), (dict(count=65536), "UNSUPPORTED"), (dict(out=0), "INVALID_ARG"),
    (dict(out=12), "INVALID_ARG"), (dict(in_=0), "INVALID_ARG"), (dict(in_=48), "INVALID_ARG"),
    (dict(dtype=5), "INVALID_ARG"), (dict(layout=2), "INVALID_ARG"), (dict(w=None), "INVALID_ARG"),
    (dict(codes=None), "INVALID_ARG"), (dict(scales=None), "INVALID_ARG"), (dict(w=264), "INVALID_ARG"),
    (dict(codes=264), "INVALID_ARG"),
]


@pytest.mark.parametrize("over,code", PACK_BAD)
def test_pack_and_unpack_refusals(over, code):
    a = dict(count=2, out=16, in_=64, dtype=L.MOE_BF16, layout=0, w=256, codes=256, scales=256)
    a.update(over)
    lib, want = L.lib(), getattr(L, "MOE_ERR_" + code)
    head = (a["count"], a["out"], a["in_"], a["dtype"], a["layout"])
    assert lib.moe_pack_weights(*head, a["w"], a["codes"], a["scales"], None) == want
    assert L.moe_last_error()
    assert lib.moe_unpack_weights(*head, a["codes"], a["scales"], a["w"], None) == want


def test_packed_workspace_covers_the_intermediates():
    d = etd.make_desc(1000, 512, 896, 8, 2)
    ffn = etd.moe_packed_workspace_size(d, L.MOE_STAGE_FFN)
    assert ffn >= 2000 * 896 * 2
    assert etd.moe_packed_workspace_size(d, L.MOE_STAGE_LAYER) >= ffn + 2 * 2000 * 512 * 2
    n = ctypes.c_size_t()
    lib = L.lib()
    assert lib.moe_packed_workspace_size(ctypes.byref(d), L.MOE_STAGE_ROUTE, ctypes.byref(n)) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_packed_workspace_size(ctypes.byref(d), L.MOE_STAGE_FFN, None) == L.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("H,I", [(40, 64), (64, 72)])
def test_packed_sizes_off_the_group_are_unsupported(H, I):
    lib, d = L.lib(), etd.make_desc(16, H, I, 8, 2)
    p = _packed()
    n = ctypes.c_size_t()
    assert lib.moe_packed_workspace_size(ctypes.byref(d), L.MOE_STAGE_FFN, ctypes.byref(n)) == L.MOE_ERR_UNSUPPORTED
    assert lib.moe_grouped_ffn_packed(ctypes.byref(d), 256, 256, ctypes.addressof(p), 256, 256, 1 << 30, None) \
        == L.MOE_ERR_UNSUPPORTED
    assert "multiples of 32" in L.moe_last_error()
    assert lib.moe_layer_forward_packed(ctypes.byref(d), None, 256, 256, None, ctypes.addressof(p), 256, None, None,
                                        None, None, 256, 1 << 30, None) == L.MOE_ERR_UNSUPPORTED


def test_packed_calls_refuse_bad_arguments():
    lib, d = L.lib(), etd.make_desc(16, 64, 64, 8, 2)
    b = ctypes.byref(d)
    ok = _packed()

    def ffn(x=256, off=256, p=ok, y=256, ws=256, n=1 << 30):
        return lib.moe_grouped_ffn_packed(b, x, off, None if p is None else ctypes.addressof(p), y, ws, n, None)

    assert ffn(p=None) == L.MOE_ERR_INVALID_ARG and "packed is NULL" in L.moe_last_error()
    for name, _ in L.PackedExperts._fields_:
        assert ffn(p=_packed(**{name: 1})) == L.MOE_ERR_INVALID_ARG and name in L.moe_last_error()
    assert ffn(x=None) == L.MOE_ERR_INVALID_ARG
    assert ffn(off=258) == L.MOE_ERR_INVALID_ARG
    assert ffn(y=264) == L.MOE_ERR_INVALID_ARG
    assert ffn(ws=None) == L.MOE_ERR_WORKSPACE
    assert ffn(n=etd.moe_packed_workspace_size(d, L.MOE_STAGE_FFN) - 1) == L.MOE_ERR_WORKSPACE
    assert ffn(ws=272) == L.MOE_ERR_INVALID_ARG
    opts = L.make_route_opts(None, 3, 1)
    st = lib.moe_layer_forward_packed(b, ctypes.addressof(opts), 256, 256, None, ctypes.addressof(ok), 256, None, None,
                                      None, None, 256, 1 << 30, None)
    assert st == L.MOE_ERR_INVALID_ARG and "route options" in L.moe_last_error()
    st = lib.moe_layer_forward_packed(b, None, 256, 256, None, ctypes.addressof(ok), 256, None, None, None, None, None,
                                      0, None)
    assert st == L.MOE_ERR_WORKSPACE


def test_packed_calls_with_zero_tokens_do_nothing():
    lib, d = L.lib(), etd.make_desc(0, 64, 64, 8, 2)
    assert lib.moe_grouped_ffn_packed(ctypes.byref(d), None, None, None, None, None, 0, None) == L.MOE_OK
    assert lib.moe_layer_forward_packed(ctypes.byref(d), *([None] * 11), 0, None) == L.MOE_OK
    assert lib.moe_profile_kernel_count() == 0


MUON_BAD = [
    (dict(count=0), "INVALID_ARG"), (dict(rows=0), "INVALID_ARG"), (dict(cols=0), "INVALID_ARG"),
    (dict(count=65536), "UNSUPPORTED"), (dict(dtype=7), "INVALID_ARG"), (dict(steps=0), "INVALID_ARG"),
    (dict(steps=11), "INVALID_ARG"), (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=float("nan")), "INVALID_ARG"),
    (dict(momentum=1.0), "INVALID_ARG"), (dict(momentum=-0.1), "INVALID_ARG"),
    (dict(momentum=float("nan")), "INVALID_ARG"), (dict(nesterov=2), "INVALID_ARG"),
    (dict(lr=float("inf")), "INVALID_ARG"), (dict(update_scale=float("nan")), "INVALID_ARG"),
    (dict(weight_decay=float("inf")), "INVALID_ARG"),
    (dict(coefs=(4.5, -4.0, 1.0)), "INVALID_ARG"),       # a past 4
    (dict(coefs=(-1.0, 0.0, 0.0)), "INVALID_ARG"),
    (dict(coefs=(3.5, 0.0, 0.0)), "INVALID_ARG"),        # 1 -> 3.5
    (dict(coefs=(2.0, 0.0, 0.0)), "INVALID_ARG"),        # 1 -> 2 -> 4 in the second step
    (dict(coefs=(1.0, 9.0, -9.0)), "INVALID_ARG"),       # both ends fine, past 3 between them
    (dict(coefs=(float("nan"), 0.0, 0.0)), "INVALID_ARG"),
    (dict(rows=65536, cols=32768), "UNSUPPORTED"),       # 4 GiB in float16
    (dict(rows=4194241, cols=1), "UNSUPPORTED"),
]


@pytest.mark.parametrize("over,code", MUON_BAD)
def test_muon_descriptor_refusals(over, code):
    a = dict(count=2, rows=16, cols=24)
    a.update(over)
    m = etd.make_muon_desc(**a)
    if "nesterov" in over:
        m.nesterov = over["nesterov"]
    lib, want, n = L.lib(), getattr(L, "MOE_ERR_" + code), ctypes.c_size_t()
    b = ctypes.byref(m)
    assert lib.moe_muon_workspace_size(b, ctypes.byref(n)) == want, L.moe_last_error()
    assert lib.moe_orthogonalize(b, 256, 256, 256, 1 << 40, None) == want
    assert lib.moe_muon_update(b, 256, 256, None, 256, 256, 1 << 40, None) == want


def test_muon_refuses_bad_pointers_and_workspaces():
    lib, m = L.lib(), etd.make_muon_desc(2, 16, 24)
    b, n = ctypes.byref(m), etd.moe_muon_workspace_size(m)
    assert lib.moe_muon_workspace_size(None, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_muon_workspace_size(b, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_orthogonalize(b, None, 256, 256, n, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_orthogonalize(b, 256, 264, 256, n, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_orthogonalize(b, 256, 256, 256, n - 1, None) == L.MOE_ERR_WORKSPACE
    assert lib.moe_orthogonalize(b, 256, 256, None, n, None) == L.MOE_ERR_WORKSPACE
    assert lib.moe_orthogonalize(b, 256, 256, 264, n, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_muon_update(b, 256, None, None, 256, 256, n, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_muon_update(b, 256, 256, 264, 256, 256, n, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_muon_update(b, 256, 256, None, None, 256, n, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_muon_update(b, 256, 256, None, 256, 256, 0, None) == L.MOE_ERR_WORKSPACE


def test_muon_accepts_the_usual_coefficients_and_gentle_ones():
    for coefs in ((0.0, 0.0, 0.0), (3.4445, -4.7750, 2.0315), (1.875, -1.25, 0.375), (1.5, -0.5, 0.0)):
        assert etd.moe_muon_workspace_size(etd.make_muon_desc(1, 100, 60, steps=10, coefs=coefs)) > 0


def test_wrappers_check_shapes_and_types():
    w = torch.zeros((2, 16, 64), dtype=torch.bfloat16)
    codes, scales = torch.zeros((2, 16, 32), dtype=torch.uint8), torch.zeros((2, 16, 2), dtype=torch.uint8)
    for bad in ((w.half(), codes, scales), (w[0], codes, scales), (w, codes[:1], scales), (w, codes, scales.int()),
                (w, codes[..., :16], scales)):
        with pytest.raises(ValueError):
            etd.moe_pack_weights(*bad)
    with pytest.raises(ValueError):   # stored the other way round
        etd.moe_unpack_weights(codes, scales, w, weight_layout="in_out")
    m = etd.make_muon_desc(2, 16, 64)
    f = w.float()
    with pytest.raises(ValueError):
        etd.moe_orthogonalize(m, f, w, None)
    with pytest.raises(ValueError):
        etd.moe_muon_update(m, w, w, w, None)              # momentum is float32
    with pytest.raises(ValueError):
        etd.moe_muon_update(m, w, f, w, None, master=f[:, :8])
