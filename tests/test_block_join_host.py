"""The join with the residual stream without a GPU: the oracle's gradients against differences of
its forward, and refused calls (none of them reaches a kernel)."""

import ctypes

import numpy as np
import pytest

import expert_token_dispatch_amd as etd
from expert_token_dispatch_amd import _lib as L
from oracle import block_join as oj

GATES = ("none", "channel", "token", "element")


def _inputs(rng, gate, post, T=5, H=8):
    shape = {"none": None, "channel": (H,), "token": (T,), "element": (T, H)}[gate]
    return {"x": rng.standard_normal((T, H)), "y": rng.standard_normal((T, H)),
            "gate": None if shape is None else rng.standard_normal(shape),
            "w_post": 1 + 0.2 * rng.standard_normal(H) if post else None, "w_pre": 1 + 0.2 * rng.standard_normal(H)}


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("post,sigmoid", [(False, False), (True, False), (True, True)])
def test_oracle_gradients_are_the_forwards_differences(gate, post, sigmoid):
    rng = np.random.default_rng(GATES.index(gate) * 3 + post + sigmoid)
    v = _inputs(rng, gate, post)
    j = oj.Join(post, gate, sigmoid, 1e-3, 0.25, 0.7)
    dz, dh = rng.standard_normal((2, 5, 8))

    def loss(u):
        f = oj.forward(j, **u)
        return (f["z"] * dz).sum() + (f["h"] * dh).sum()

    z = oj.forward(j, **v)["z"]
    got = oj.backward(j, z, v["y"], v["gate"], v["w_post"], v["w_pre"], dz, dh)
    step = 1e-6
    for name, grad in (("x", "dx"), ("y", "dy"), ("gate", "dgate"), ("w_post", "dw_post"), ("w_pre", "dw_pre")):
        if v[name] is None:
            assert grad not in got
            continue
        num = np.zeros_like(v[name])
        for i in np.ndindex(num.shape):
            u = {k: None if t is None else t.copy() for k, t in v.items()}
            u[name][i] += step
            up = loss(u)
            u[name][i] -= 2 * step
            num[i] = (up - loss(u)) / (2 * step)
        np.testing.assert_allclose(got[grad], num, rtol=1e-6, atol=1e-7)


def test_the_magnitudes_bound_the_values():
    rng = np.random.default_rng(3)
    v = _inputs(rng, "element", True)
    j = oj.Join(True, "element", True)
    f = oj.forward(j, **v)
    b = oj.backward(j, f["z"], v["y"], v["gate"], v["w_post"], v["w_pre"], *rng.standard_normal((2, 5, 8)))
    for d in (f, b):
        for k in d:
            if not k.startswith("mag_"):
                assert np.all(np.abs(d[k]) <= d["mag_" + k] * (1 + 1e-12)), k


def _desc(**over):
    a = dict(rows=4, hidden=64, post_norm=True, gate="channel", gate_act="sigmoid")
    a.update(over)
    return etd.make_join_desc(**a)


DESC_BAD = [
    (dict(rows=-1), "INVALID_ARG"), (dict(rows=1 << 31), "UNSUPPORTED"), (dict(hidden=0), "INVALID_ARG"),
    (dict(hidden=12), "INVALID_ARG"), (dict(hidden=16392), "UNSUPPORTED"), (dict(hidden=8200, dtype="f32"), "UNSUPPORTED"),
    (dict(dtype=4), "INVALID_ARG"), (dict(post_norm=2), "INVALID_ARG"), (dict(gate=4), "INVALID_ARG"),
    (dict(gate=-1), "INVALID_ARG"), (dict(gate_act=2), "INVALID_ARG"), (dict(eps=0.0), "INVALID_ARG"),
    (dict(eps=float("nan")), "INVALID_ARG"), (dict(weight_offset=float("inf")), "INVALID_ARG"),
    (dict(residual_scale=float("nan")), "INVALID_ARG"),
]


@pytest.mark.parametrize("over,code", DESC_BAD)
def test_descriptors_refused(over, code):
    j, lib, want = ctypes.byref(_desc(**over)), L.lib(), getattr(L, "MOE_ERR_" + code)
    n = ctypes.c_size_t()
    assert lib.moe_join_workspace_size(j, ctypes.byref(n)) == want
    assert lib.moe_block_join(j, 256, 256, 256, 256, 256, 256, 256, None) == want
    assert lib.moe_block_join_backward(j, *[256] * 13, 1 << 30, None) == want
    assert L.moe_last_error()


FWD = ("x", "y", "gate", "w_post", "w_pre", "z", "h")
FWD_BAD = [
    dict(x=None), dict(x=264), dict(y=264), dict(gate=None), dict(gate=264), dict(w_post=264), dict(w_pre=264),
    dict(z=None), dict(z=264), dict(h=264), dict(h=None), dict(y=None), dict(y=None, z=None),
]


@pytest.mark.parametrize("over", FWD_BAD)
def test_forward_arguments_refused(over):
    a = [over.get(n, 256) for n in FWD]
    assert L.lib().moe_block_join(ctypes.byref(_desc()), *a, None) == L.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("desc,over", [
    (dict(gate="none"), {}),                                        # a gate that no kind asks for
    (dict(post_norm=False), {}),                                    # a norm weight without its norm
    (dict(post_norm=False, gate="none"), dict(y=None, z=None, gate=None, w_post=None, h=None, w_pre=None)),
    (dict(post_norm=False, gate="none"), dict(y=None, gate=None, w_post=None)),    # z without y
    (dict(post_norm=False, gate="token"), dict(w_post=None, gate=258)),
])
def test_forward_arguments_refused_by_what_the_descriptor_says(desc, over):
    a = [over.get(n, 256) for n in FWD]
    assert L.lib().moe_block_join(ctypes.byref(_desc(**desc)), *a, None) == L.MOE_ERR_INVALID_ARG


BWD = ("z", "y", "gate", "w_post", "w_pre", "dz", "dh", "dx", "dy", "dgate", "dw_post", "dw_pre", "ws")
BWD_BAD = [
    dict(z=None), dict(y=None), dict(gate=None), dict(dz=264), dict(dh=None), dict(dz=None, dh=None, w_pre=None, dw_pre=None),
    dict(dx=None), dict(dx=264), dict(dy=None), dict(dgate=None), dict(dw_post=None), dict(dw_pre=None), dict(w_pre=None),
    dict(w_post=None), dict(dh=264), dict(dy=264), dict(dw_pre=264), dict(ws=264),
]


@pytest.mark.parametrize("over", BWD_BAD)
def test_backward_arguments_refused(over):
    a = [over.get(n, 256) for n in BWD]
    assert L.lib().moe_block_join_backward(ctypes.byref(_desc()), *a, 1 << 30, None) == L.MOE_ERR_INVALID_ARG


def test_backward_workspace():
    j = _desc(rows=100)
    need = etd.moe_join_workspace_size(j)
    assert need >= 3 * 64 * 4
    a = [256] * 13
    assert L.lib().moe_block_join_backward(ctypes.byref(j), *a, need - 1, None) == L.MOE_ERR_WORKSPACE
    a[-1] = None
    assert L.lib().moe_block_join_backward(ctypes.byref(j), *a, need, None) == L.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("dtype,H", [("bf16", 8), ("bf16", 2880), ("bf16", 16384), ("f32", 512), ("f32", 8192)])
def test_a_workspace_for_the_most_rows_is_enough_for_any(dtype, H):
    def size(rows):
        return etd.moe_join_workspace_size(etd.make_join_desc(rows, H, dtype, True, "channel"))
    most = size((1 << 31) - 1)
    assert 0 < most <= 3 * 4 * 262144 * 16
    assert all(size(r) <= most for r in [0, 1, 2, 63, 1000, 4095, 4096, 4097, 5000, 10 ** 6, 10 ** 6 + 7])
    assert size(0) == 0 and size(5) >= 5 * 3 * 4 * H


def test_no_rows_is_no_work():
    j = _desc(rows=0, gate="none", post_norm=False)
    assert L.lib().moe_block_join(ctypes.byref(j), *[None] * 7, None) == L.MOE_OK
    assert L.lib().moe_block_join_backward(ctypes.byref(j), *[None] * 13, 0, None) == L.MOE_OK


def test_the_binding_refuses_other_shapes_and_types():
    torch = pytest.importorskip("torch")
    j = _desc(gate="token")
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    g = torch.zeros(4)
    for bad in (dict(x=x[:3]), dict(y=x.float()), dict(z=x.T), dict(w_post=w[:32]), dict(w_pre=w.float()),
                dict(gate=g.bfloat16()), dict(gate=torch.zeros(64))):
        a = dict(x=x, y=x, gate=g, w_post=w, w_pre=w, z=x, h=x)
        a.update(bad)
        with pytest.raises(ValueError, match="of this join is"):
            etd.moe_block_join(j, **a)


@pytest.mark.parametrize("dgate", (None, 264))
def test_no_rows_and_a_refused_gate_gradient_enqueue_nothing(dgate):
    """The refusal comes before the weights' gradients are cleared (which has no device to run on here)."""
    a = [256] * 13
    a[BWD.index("dgate")] = dgate
    assert L.lib().moe_block_join_backward(ctypes.byref(_desc(rows=0)), *a, 1 << 30, None) == L.MOE_ERR_INVALID_ARG
    assert "dgate" in L.moe_last_error()
