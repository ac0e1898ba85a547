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


@pytest.mark.parametrize("T,H", [(128, 512), (1024, 512), (2048, 512), (4096, 512), (1000, 4096), (4096, 64)])
def test_sums_over_rows_lose_what_a_tree_loses(T, H):
    """Rows of ones: zh and yh are 1 to the bit (eps is below a step of 1), so every sum over rows is one of given numbers.
    They lie less than 2^-17 / 2 past 1, so that adding them one after another drops the same again and again.  A term of
    the sums passes through a block's rows one by one, the blocks of a thread of the second step eight at a time as a tree
    (3) and those eights one by one, and 128 threads as a tree (7).  Each of these sums rounds by at most a unit of itself,
    and all have one sign."""
    say(f"[join] sums of {T} x {H}")
    n = H // 4  # vectors of a row
    most = 256 * max(1, 1024 // next((t for t in (64, 128, 192, 256, 384, 512, 768) if n <= t), 512 * ((n + 511) // 512)))
    rows = max(1, -(-T // most))
    blocks = -(-T // rows)
    units = rows + 3 + -(-blocks // 1024) + 7 + 1
    rng = np.random.default_rng(T + H)
    ones = torch.ones((T, H), device="cuda")
    col = 1.0 + 2.0 ** -17 * (0.45 + 0.04 * rng.random(H))
    grad = dev(np.broadcast_to(col, (T, H)).copy(), "f32")
    w = torch.ones(H, device="cuda")

    def off(got, terms):
        want = host(terms).sum(0)
        return float((np.abs(host(got) - want) / want).max() / UNIT)
    # dw_post = sum of dz, dgate the same
    jd = etd.make_join_desc(T, H, "f32", True, "channel", "linear", 1e-30)
    out = backward(jd, {"x": ones, "y": ones, "gate": w, "w_post": w, "w_pre": None}, {"dz": grad, "dh": None})
    assert off(out["dw_post"], grad) <= units and off(out["dgate"], grad) <= units
    # dw_pre = sum of dh
    jd = etd.make_join_desc(T, H, "f32", False, "none", "linear", 1e-30)
    out = backward(jd, {"x": ones, "y": None, "gate": None, "w_post": None, "w_pre": w}, {"dz": grad, "dh": grad})
    assert off(out["dw_pre"], grad) <= units


def test_a_blockjoins_calls_on_two_streams_and_in_two_graphs_share_no_sums(monkeypatch):
    T, H = 300, 520
    v, d = inputs(T, H, "bf16", "channel", True, "full")
    join = etd.BlockJoin(H, "bf16", v["w_post"], v["w_pre"], gate="channel", gate_act="sigmoid")
    used, real = [], L.moe_block_join_backward

    def recorded(*args):
        used.append((args[-1].data_ptr(), args[-1].data_ptr() + args[-1].numel()))
        real(*args)
    monkeypatch.setattr(L, "moe_block_join_backward", recorded)

    def step(grads=None):
        return join.backward(v["x"], v["y"], v["gate"], d["dz"], d["dh"], grads=grads)
    want = step()
    torch.cuda.synchronize()
    used.clear()  # a capture gives idle memory back, and may get it again
    sides, graphs, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [], []
    for _ in sides:
        outs.append({k: None if t is None else torch.empty_like(t) for k, t in want.items()})
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step(outs[-1])
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append(step())
    spans = sorted(used)
    assert len(used) == 4 and all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
    for _ in range(3):
        for o in outs[:2]:
            for t in o.values():
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, sides):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o in outs:
            for k, t in want.items():
                assert torch.equal(o[k], t), k


def test_gradients_of_the_norm_alone_into_buffers_of_its_own():
    """Without y the results are dx and dw_pre: the buffers for them are enough."""
    T, H = 20, 136
    v, d = inputs(T, H, "f32", "none", False, "enter")
    join = etd.BlockJoin(H, "f32", w_pre=v["w_pre"])
    want = join.backward(v["x"], dz=d["dz"], dh=d["dh"])
    grads = {"dx": torch.empty_like(v["x"]), "dw_pre": torch.empty_like(v["w_pre"])}
    got = join.backward(v["x"], dz=d["dz"], dh=d["dh"], grads=grads)
    torch.cuda.synchronize()
    assert got is grads and torch.equal(got["dx"], want["dx"]) and torch.equal(got["dw_pre"], want["dw_pre"])
    del grads["dw_pre"]
    with pytest.raises(L.MoeError, match="dw_pre"):
        join.backward(v["x"], dz=d["dz"], dh=d["dh"], grads=grads)
