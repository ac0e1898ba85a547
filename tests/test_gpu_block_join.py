"""The join with the residual stream on the GPU against the float64 oracle.

Tolerances.  An output is off by half a step of its type (bf16 2^-8, float32 2^-24 of its value) and by
the float32 evaluation.  A row's sum adds at most 16 products in a thread, then 6 steps of a wave and 16
waves: 38 roundings, so a mean and its reciprocal root are off by at most 20 + 3 units of 2^-24; a result
takes at most two of them, a sigmoid (whose exponential is off by 2 + |g| units, |g| < 6 here) and a
dozen products and sums: under 96 units of 2^-24 of the magnitudes that went into it.  A sum over rows adds
at most rows / 256 + 1 rows in a thread (and whatever each is off), up to 4096 / 128 blocks in a thread of
the second step and 128 threads.
"""

import numpy as np
import pytest

from oracle import block_join as oj
from tests._harness import say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import expert_token_dispatch_amd as etd  # noqa: E402
from expert_token_dispatch_amd import _lib as L  # noqa: E402

UNIT = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": UNIT}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(a, dtype):
    return None if a is None else torch.tensor(a, dtype=torch.float32, device="cuda").to(DT[dtype])


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def inputs(T, H, dtype, gate, post, form, seed=0, offset=0.0):
    """Tensors as a layer has them: a stream with a few large channels, and small gradients."""
    rng = np.random.default_rng(1000 * T + H + seed)
    stream = rng.standard_normal((T, H)) * np.where(rng.random(H) < 0.05, 10.0, 1.0)
    shape = {"none": None, "channel": (H,), "token": (T,), "element": (T, H)}[gate]
    g = None if shape is None else np.clip(rng.standard_normal(shape), -5, 5)
    v = {"x": dev(stream, dtype), "y": None if form == "enter" else dev(2 * rng.standard_normal((T, H)), dtype),
         "gate": dev(g, "f32" if gate == "token" else dtype),
         "w_post": dev(1 - offset + 0.1 * rng.standard_normal(H), dtype) if post else None,
         "w_pre": None if form == "post" else dev(1 - offset + 0.1 * rng.standard_normal(H), dtype)}
    d = {"dz": dev(rng.standard_normal((T, H)), dtype), "dh": None if form == "post" else dev(rng.standard_normal((T, H)), dtype)}
    return v, d


def check(got, ref, mag, dtype, units, what):
    got = host(got)
    assert got.shape == ref.shape, what
    allowed = HALF[dtype] * np.abs(ref) + units * UNIT * mag + 1e-38
    worst = float((np.abs(got - ref) / allowed).max())
    assert np.isfinite(got).all() and worst <= 1.0, f"{what}: {worst} of the allowed error"


def run_both(v, d, dtype, j, jd, form, what):
    T, H = v["x"].shape
    f64 = {k: host(t) for k, t in v.items()}
    ref = oj.forward(j, f64["x"], f64["y"], f64["gate"], f64["w_post"], f64["w_pre"], next_norm=form != "post")
    z = None if v["y"] is None else torch.full_like(v["x"], 7.0)
    h = None if form == "post" else torch.full_like(v["x"], 7.0)
    etd.moe_block_join(jd, v["x"], v["y"], v["gate"], v["w_post"], v["w_pre"], z, h)
    torch.cuda.synchronize()
    for name, t in (("z", z), ("h", h)):
        if t is not None:
            check(t, ref[name], ref["mag_" + name], dtype, 96, f"{what} {name}")
    zin = v["x"] if z is None else z

    def like(t):
        return None if t is None else torch.full_like(t, 7.0)
    out = {"dx": like(zin), "dy": like(v["y"]), "dgate": like(v["gate"]), "dw_post": like(v["w_post"]), "dw_pre": like(v["w_pre"])}
    ws = torch.empty(max(etd.moe_join_workspace_size(jd), 1), dtype=torch.uint8, device="cuda").fill_(255)
    etd.moe_block_join_backward(jd, zin, v["y"], v["gate"], v["w_post"], v["w_pre"], d["dz"], d["dh"], out["dx"], out["dy"],
                                out["dgate"], out["dw_post"], out["dw_pre"], ws)
    torch.cuda.synchronize()
    ref = oj.backward(j, host(zin), f64["y"], f64["gate"], f64["w_post"], f64["w_pre"], host(d["dz"]), host(d["dh"]))
    for name, t in out.items():
        if t is None:
            assert name not in ref
            continue
        over_rows = name in ("dw_post", "dw_pre") or (name == "dgate" and j.gate == "channel")
        out_dtype = "f32" if t.dtype == torch.float32 else "bf16"
        units = 96 * 2 + (T // 256 + 1 + 160 if over_rows else 0)
        if name == "dgate" and j.gate == "token":
            units += 38
        check(t, ref[name], ref["mag_" + name], out_dtype, units, f"{what} {name}")
    return z, h, out


GATES = ("none", "channel", "token", "element")
# rows, hidden: every width of the kernels and both sides of where it changes, odd numbers of rows
SIZES = [(1, 8), (3, 40), (5, 512), (7, 520), (1, 1024), (6, 1032), (4, 2048), (3, 2056), (2, 2880), (5, 4096),
         (2, 4104), (3, 8192), (2, 8200), (2, 16384)]


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("T,H", SIZES)
def test_sizes(T, H, dtype):
    if dtype == "f32" and H > 8192:
        pytest.skip("a float32 row of this length is refused")
    say(f"[join] {T} x {H} {dtype}")
    v, d = inputs(T, H, dtype, "channel", True, "full")
    j = oj.Join(True, "channel", True, 1e-6, 0.0, 0.5)
    jd = etd.make_join_desc(T, H, dtype, True, "channel", "sigmoid", 1e-6, 0.0, 0.5)
    run_both(v, d, dtype, j, jd, "full", f"{T} x {H} {dtype}")


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("form,post,sigmoid,offset", [("full", True, False, 1.0), ("full", True, True, 0.0),
                                                      ("full", False, True, 0.0), ("post", True, False, 0.0),
                                                      ("post", False, False, 0.0)])
def test_forms_and_gates(form, post, sigmoid, offset, gate, dtype):
    T, H = 37, 200
    say(f"[join] {form} post={post} {gate} sigmoid={sigmoid} {dtype}")
    v, d = inputs(T, H, dtype, gate, post, form, offset=offset)
    j = oj.Join(post, gate, sigmoid, 1e-5, offset, -0.75)
    jd = etd.make_join_desc(T, H, dtype, post, gate, "sigmoid" if sigmoid else "linear", 1e-5, offset, -0.75)
    run_both(v, d, dtype, j, jd, form, f"{form} {gate}")


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("weighted", (True, False))
def test_the_norm_before_a_first_block(weighted, dtype):
    T, H = 19, 264
    v, d = inputs(T, H, dtype, "none", False, "enter")
    if not weighted:
        v["w_pre"] = None
    say(f"[join] enter weighted={weighted} {dtype}")
    jd = etd.make_join_desc(T, H, dtype, eps=1e-5, weight_offset=0.5)
    run_both(v, d, dtype, oj.Join(eps=1e-5, offset=0.5), jd, "enter", "enter")
    d["dz"] = None
    run_both(v, d, dtype, oj.Join(eps=1e-5, offset=0.5), jd, "enter", "enter without dz")


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T,H,dtype", [(515, 4104, "f32"), (300, 8192, "f32"), (515, 6152, "bf16"), (259, 12288, "bf16"),
                                       (513, 4672, "bf16")])
def test_wide_rows_share_the_blocks(T, H, dtype, gate):
    """Several rows a block where a thread has several vectors."""
    say(f"[join] {T} x {H} {gate} {dtype}")
    v, d = inputs(T, H, dtype, gate, True, "full")
    jd = etd.make_join_desc(T, H, dtype, True, gate, "sigmoid", 1e-6, 0.0, 0.5)
    run_both(v, d, dtype, oj.Join(True, gate, True, 1e-6, 0.0, 0.5), jd, "full", f"{T} x {H} {gate} {dtype}")


@pytest.mark.parametrize("T", (511, 512, 513, 1700, 5000))
def test_many_rows_share_the_blocks(T):
    H = 72
    say(f"[join] {T} rows")
    v, d = inputs(T, H, "f32", "channel", True, "full")
    jd = etd.make_join_desc(T, H, "f32", True, "channel", "linear", 1e-6, 0.0, 1.0)
    run_both(v, d, "f32", oj.Join(True, "channel", False), jd, "full", f"{T} rows")


def test_norms_without_weights_and_gradients_of_one_result_alone():
    T, H = 9, 136
    v, d = inputs(T, H, "f32", "element", False, "full")
    v["w_pre"] = None
    j = oj.Join(True, "element", True)
    jd = etd.make_join_desc(T, H, "f32", True, "element", "sigmoid")
    run_both(v, d, "f32", j, jd, "full", "no weights")
    run_both(v, {"dz": None, "dh": d["dh"]}, "f32", j, jd, "full", "dh alone")
    run_both(v, {"dz": d["dz"], "dh": None}, "f32", j, jd, "full", "dz alone")


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_outputs_in_the_buffers_of_inputs_and_rows_around_them(dtype):
    """z on x, h on y, dx on dz, dy on y; the rows around the call's stay as they were."""
    T, H = 6, 1032
    say(f"[join] in place {dtype}")
    v, d = inputs(T, H, dtype, "token", True, "full")
    jd = etd.make_join_desc(T, H, dtype, True, "token", "sigmoid")
    z, h, out = run_both(v, d, dtype, oj.Join(True, "token", True), jd, "full", "apart")

    def framed(t):
        big = torch.full((T + 2, H), 3.0, dtype=t.dtype, device="cuda")
        big[1:-1] = t
        return big
    x, y, dz, dy = framed(v["x"]), framed(v["y"]), framed(d["dz"]), framed(v["y"])
    etd.moe_block_join(jd, x[1:-1], y[1:-1], v["gate"], v["w_post"], v["w_pre"], x[1:-1], y[1:-1])
    ws = torch.empty(etd.moe_join_workspace_size(jd), dtype=torch.uint8, device="cuda")
    small = {k: torch.empty_like(out[k]) for k in ("dgate", "dw_post", "dw_pre")}
    etd.moe_block_join_backward(jd, z, dy[1:-1], v["gate"], v["w_post"], v["w_pre"], dz[1:-1], d["dh"], dz[1:-1], dy[1:-1],
                                small["dgate"], small["dw_post"], small["dw_pre"], ws)
    torch.cuda.synchronize()
    for got, want in ((x, z), (y, h), (dz, out["dx"]), (dy, out["dy"])):
        assert torch.equal(got[1:-1], want)
        assert (got[0] == 3.0).all() and (got[-1] == 3.0).all()
    for k, t in small.items():
        assert torch.equal(t, out[k])


def test_a_rows_infinities_and_nan_stay_in_it():
    T, H = 12, 520
    v, _ = inputs(T, H, "bf16", "element", True, "full")
    jd = etd.make_join_desc(T, H, "bf16", True, "element", "sigmoid")

    def go():
        z, h = torch.empty_like(v["x"]), torch.empty_like(v["x"])
        etd.moe_block_join(jd, v["x"], v["y"], v["gate"], v["w_post"], v["w_pre"], z, h)
        return z, h
    clean = go()
    v["x"][3, 7], v["y"][5, 500], v["gate"][8, 0] = float("nan"), float("inf"), float("nan")
    bad = go()
    keep = [r for r in range(T) if r not in (3, 5, 8)]
    for a, b in zip(clean, bad):
        assert torch.equal(a[keep], b[keep])
    assert bad[1][3].isnan().all() and bad[0][8, 0].isnan()


def test_no_rows_zero_the_weights_gradients():
    H = 24
    jd = etd.make_join_desc(0, H, "bf16", True, "channel", "linear")
    x = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    w = [torch.full((H,), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(6)]
    etd.moe_block_join_backward(jd, x, x, w[0], w[1], w[2], x, x, x, x, w[3], w[4], w[5], None)
    torch.cuda.synchronize()
    assert all((t == 0).all() for t in w[3:]) and all((t == 5).all() for t in w[:3])


def test_on_a_stream_of_its_own_and_the_same_every_time():
    T, H = 700, 2880
    v, d = inputs(T, H, "bf16", "channel", True, "full")
    join = etd.BlockJoin(H, "bf16", v["w_post"], v["w_pre"], gate="channel", gate_act="sigmoid")
    z, h = join.forward(v["x"], v["y"], v["gate"])
    g = join.backward(z, v["y"], v["gate"], d["dz"], d["dh"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        z2, h2 = join.forward(v["x"], v["y"], v["gate"])
        g2 = join.backward(z2, v["y"], v["gate"], d["dz"], d["dh"])
    side.synchronize()
    assert torch.equal(z, z2) and torch.equal(h, h2)
    for k in g:
        assert torch.equal(g[k], g2[k]), k


def test_captured_and_replayed():
    T, H = 130, 520
    v, d = inputs(T, H, "bf16", "channel", True, "full")
    join = etd.BlockJoin(H, "bf16", v["w_post"], v["w_pre"], gate="channel", gate_act="sigmoid")
    z, h = torch.empty_like(v["x"]), torch.empty_like(v["x"])
    grads = join.backward(v["x"], v["y"], v["gate"], d["dz"], d["dh"])
    x = v["x"].clone()

    def step():
        join.forward(x, v["y"], v["gate"], z=z, h=h)
        join.backward(z, v["y"], v["gate"], d["dz"], d["dh"], grads=grads)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(3):
        x.copy_(v["x"] * (1 + r))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (z, h, *[t for t in grads.values() if t is not None])]
        ze, he = join.forward(x, v["y"], v["gate"])
        ge = join.backward(ze, v["y"], v["gate"], d["dz"], d["dh"])
        torch.cuda.synchronize()
        for a, b in zip(got, (ze, he, *[t for t in ge.values() if t is not None])):
            assert torch.equal(a, b), f"replay {r}"


def test_rows_past_the_first_dimension_of_a_launch():
    """More than 2^20 rows of a block each: the last ones are the first ones again."""
    T, H = (1 << 20) + 5, 1032
    g = torch.Generator(device="cuda").manual_seed(3)
    head = torch.randn((5, H), generator=g, device="cuda").bfloat16()
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[:5], x[-5:] = head, head
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).bfloat16()
    h = torch.full_like(x, 7.0)
    etd.moe_block_join(etd.make_join_desc(T, H), x, None, None, None, w, None, h)
    torch.cuda.synchronize()
    assert torch.equal(h[:5], h[-5:]) and (h[5:-5] == 0).all() and h[:5].abs().min() >= 0
    ref = oj.forward(oj.Join(), host(head), w_pre=host(w))
    check(h[-5:], ref["h"], ref["mag_h"], "bf16", 96, "last rows")


def test_a_training_step_of_a_block():
    """norm -> layer -> norm, gate, scale, sum and the next norm, forward and backward, against the gradients that
    differentiating the whole in 64 bits gives (at the layer's own choice of experts).  Each of the three stages is
    held to 1e-5 of its rows' largest entries; together they get five times that."""
    import synth
    from tests._harness import TOL_F32, layer_of
    s = synth.spec("tiny_fp32", T=60)
    layer, x = layer_of(synth.make_layer(s))
    T, H, k = s.T, s.H, s.k
    g = torch.Generator(device="cuda").manual_seed(1)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    w = [1 + 0.1 * rand(H) for _ in range(3)]
    gate, dz, dh2 = rand(T), rand(T, H), rand(T, H)
    first = etd.BlockJoin(H, "f32", w_pre=w[0])
    after = etd.BlockJoin(H, "f32", w_post=w[1], w_pre=w[2], gate="token", gate_act="sigmoid", residual_scale=0.7)
    _, h = first.forward(x)
    y, saved = layer.forward_train(h)
    z, h2 = after.forward(x, y, gate)
    ga = after.backward(z, y, gate, dz, dh2)
    gl = layer.backward(h, saved, ga["dy"])
    gf = first.backward(x, dz=ga["dx"], dh=gl["dx"])
    torch.cuda.synchronize()

    ids = saved._tensors["topk_ids"].long()
    P = [t.double().requires_grad_() for t in (x, w[0], w[1], w[2], gate, layer.w_router, layer.w_gate, layer.w_up, layer.w_down)]
    X, W0, W1, W2, G, WR, WG, WU, WD = P

    def norm(v, f):
        return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6) * f
    Hn = norm(X, W0)
    logits = Hn @ WR.T + (0 if layer.b_router is None else layer.b_router.double())
    wt = torch.softmax(torch.gather(logits, 1, ids), 1)
    Y = torch.zeros_like(X)
    for j in range(k):
        for e in range(s.E):
            rows = (ids[:, j] == e).nonzero()[:, 0]
            if len(rows):
                v = Hn[rows]
                a, b = (v @ WG[e].T, v @ WU[e].T) if s.weight_layout in ("out_in", 0) else (v @ WG[e], v @ WU[e])
                o = torch.nn.functional.silu(a) * b
                o = o @ WD[e].T if s.weight_layout in ("out_in", 0) else o @ WD[e]
                Y = Y.index_add(0, rows, wt[rows, j, None] * o)
    Z = X + 0.7 * torch.sigmoid(G)[:, None] * norm(Y, W1)
    loss = (Z * dz.double()).sum() + (norm(Z, W2) * dh2.double()).sum()
    ref = torch.autograd.grad(loss, P)
    got = (gf["dx"], gf["dw_pre"], ga["dw_post"], ga["dw_pre"], ga["dgate"], gl["dw_router"], gl["dw_gate"], gl["dw_up"], gl["dw_down"])
    for name, a, b in zip(("x", "w0", "w1", "w2", "gate", "router", "gates", "ups", "downs"), got, ref):
        assert (a.double() - b).abs().max() <= 5 * TOL_F32 * b.abs().max(), name
