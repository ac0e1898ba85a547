"""The join's gradients where a formula is easily evaluated badly: gates far from zero, infinities in a block's output that
is not normed, sums over many rows; and what a BlockJoin's calls share."""

import numpy as np
import pytest

from oracle import block_join as oj
from tests._harness import say
from tests.test_gpu_block_join import GATES, UNIT, check, dev, host, inputs, run_both

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import expert_token_dispatch_amd as etd  # noqa: E402
from expert_token_dispatch_amd import _lib as L  # noqa: E402

FAR = np.array([8.0, -8.0, 12.0, -12.0, 20.0, -20.0, 40.0, -40.0])  # bfloat16 values


def backward(jd, v, d, z=None):
    z = v["x"] if z is None else z

    def like(t):
        return None if t is None else torch.full_like(t, 7.0)
    out = {"dx": like(z), "dy": like(v["y"]), "dgate": like(v["gate"]), "dw_post": like(v["w_post"]), "dw_pre": like(v["w_pre"])}
    ws = torch.empty(max(etd.moe_join_workspace_size(jd), 1), dtype=torch.uint8, device="cuda").fill_(255)
    etd.moe_block_join_backward(jd, z, v["y"], v["gate"], v["w_post"], v["w_pre"], d["dz"], d["dh"], out["dx"], out["dy"],
                                out["dgate"], out["dw_post"], out["dw_pre"], ws)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("post", (True, False))
@pytest.mark.parametrize("gate", GATES[1:])
def test_sigmoid_gates_far_from_zero(gate, post, dtype):
    """s (1 - s) of the same relative precision on both sides.  Bound: as everywhere (twice 96 units of 2^-24, 38 of the
    sum over a row, the roundings of the sum over the rows), and the exponential's |g| = 40 units."""
    T, H = 24, 72
    say(f"[join] far gates {gate} post={post} {dtype}")
    v, d = inputs(T, H, dtype, gate, post, "full")
    g = FAR[np.arange(v["gate"].numel()) % len(FAR)].reshape(v["gate"].shape)
    v["gate"] = dev(g, "f32" if gate == "token" else dtype)
    jd = etd.make_join_desc(T, H, dtype, post, gate, "sigmoid", 1e-6, 0.0, 0.5)
    out = backward(jd, v, d)
    f64 = {k: host(t) for k, t in v.items()}
    ref = oj.backward(oj.Join(post, gate, True, 1e-6, 0.0, 0.5), f64["x"], f64["y"], f64["gate"], f64["w_post"], f64["w_pre"],
                      host(d["dz"]), host(d["dh"]))
    for name, t in out.items():
        if t is not None:
            units = 192 + 40 + (38 if name == "dgate" and gate == "token" else 0) + (161 if t.dim() == 1 else 0)
            check(t, ref[name], ref["mag_" + name], "f32" if t.dtype == torch.float32 else "bf16", units, f"{gate} {name}")


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("act", ("linear", "sigmoid"))
@pytest.mark.parametrize("gate", GATES)
def test_without_a_norm_the_blocks_gradient_does_not_ask_for_its_output(gate, act, dtype):
    """dy = scale g D: infinities and NaN in y leave it, and dx, as they are; a gate's gradient has them in their row."""
    T, H = 12, 520
    say(f"[join] infinite y {gate} {act} {dtype}")
    v, d = inputs(T, H, dtype, gate, False, "post")
    jd = etd.make_join_desc(T, H, dtype, False, gate, act, 1e-6, 0.0, 0.5)
    clean = backward(jd, v, d)
    y = v["y"].clone()
    y[3, 7], y[5, 500], y[8, 0] = float("inf"), float("-inf"), float("nan")
    bad = backward(jd, {**v, "y": y}, d)
    assert torch.isfinite(clean["dy"]).all()
    assert torch.equal(bad["dy"], clean["dy"]) and torch.equal(bad["dx"], clean["dx"])
    if gate in ("token", "element"):
        keep = [r for r in range(T) if r not in (3, 5, 8)]
        assert torch.equal(bad["dgate"][keep], clean["dgate"][keep])
        assert not torch.isfinite(bad["dgate"][[3, 5, 8]].reshape(3, -1)).all(dim=1).any()
    # and with the next norm's gradient, whose z is another tensor
    v, d = inputs(T, H, dtype, gate, False, "full")
    clean, bad = backward(jd, v, d), backward(jd, {**v, "y": y}, d)
    assert torch.equal(bad["dy"], clean["dy"]) and torch.equal(bad["dw_pre"], clean["dw_pre"])
