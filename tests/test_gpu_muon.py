"""The weight update on the GPU: orthogonalisation by Newton-Schulz steps and the Muon step
against their formulas in 64 bits, and a training step, its update, packing and the packed
forward in a row."""

import math

import numpy as np
import pytest

import synth
from tests._harness import layer_of, np_of, say
from tests.test_gpu_packed_experts import values_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import expert_token_dispatch_amd as etd  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
USUAL = (3.4445, -4.7750, 2.0315)
# Frobenius error of a result over its norm.  bf16: half a step of the result (2^-8) and as much
# again for the float16 working values.  f32: an error of X_j grows by at most a = 3.45 a step
# (the map's slope), a^5 = 485 from X_0 on, whose norm is 1: 485 * 2^-24 = 2.9e-5, and the
# products' roundings of P, relative to X again, each as much over the remaining steps
# (a geometric sum, 1.41 times).
TOL = {"bf16": 2.0 ** -7, "f32": 4.1e-5}


def newton_schulz(u, steps=5, coefs=USUAL, eps=1e-7):
    a, b, c = coefs
    x = u / (np.linalg.norm(u) + eps) if np.linalg.norm(u) + eps > 0 else u * 0.0
    for _ in range(steps):
        g = x @ x.T if x.shape[0] <= x.shape[1] else x.T @ x
        x = a * x + ((b * g + c * (g @ g)) @ x if x.shape[0] <= x.shape[1] else x @ (b * g + c * (g @ g)))
    return x


def gradient(shape, seed, scale=1e-3):
    """A few strong directions over a broad floor."""
    rng = np.random.default_rng(seed)
    L, R, C = shape
    r = max(1, min(R, C) // 16)
    s = rng.standard_normal((L, R, r)) @ rng.standard_normal((L, r, C)) / math.sqrt(r)
    return (scale * (s + 0.25 * rng.standard_normal(shape))).astype(np.float32)


def orthogonalize(g, dtype, steps=5, out=None, **kw):
    m = etd.make_muon_desc(*g.shape, dtype=dtype, steps=steps, **kw)
    ws = torch.full((etd.moe_muon_workspace_size(m),), 255, dtype=torch.uint8, device="cuda")
    o = torch.empty_like(g) if out is None else out
    etd.moe_orthogonalize(m, g, o, ws)
    torch.cuda.synchronize()
    return o


def assert_near(got, ref, dtype, what=""):
    n = np.linalg.norm(ref)
    err = np.linalg.norm(got - ref) / n if n else np.abs(got).max()
    say(f"[muon]   {what} error {err:.2e}")
    assert err <= (TOL[dtype] if n else 0.0), f"{what}: {err}"


SHAPES = [(1, 1, 1), (3, 2, 7), (2, 9, 3), (2, 64, 64), (1, 65, 63), (4, 100, 260), (2, 260, 100), (1, 300, 290),
          (2, 257, 700), (2, 700, 257), (1, 128, 2048), (1, 640, 640),
          (1, 1090, 1300), (1, 1300, 1090), (9, 264, 520)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_orthogonalize(shape, dtype):
    say(f"[muon] orthogonalize {shape} {dtype}")
    g = torch.from_numpy(gradient(shape, sum(shape))).to(TYPES[dtype])
    o = np_of(orthogonalize(g.cuda(), dtype)).astype(np.float64)
    for z in range(shape[0]):
        assert_near(o[z], newton_schulz(g[z].double().numpy()), dtype, f"matrix {z}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6])
@pytest.mark.parametrize("shape", [(2, 96, 80), (1, 272, 320)])
def test_steps_and_coefficients(shape, steps, dtype):
    g = torch.from_numpy(gradient(shape, 5)).to(TYPES[dtype])
    for coefs in (USUAL, (1.875, -1.25, 0.375), (1.5, -0.5, 0.0)):
        o = np_of(orthogonalize(g.cuda(), dtype, steps=steps, coefs=coefs)).astype(np.float64)
        for z in range(shape[0]):
            assert_near(o[z], newton_schulz(g[z].double().numpy(), steps, coefs), dtype, f"{coefs} x {steps}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_zero_matrix_stays_zero_and_others_do_not_see_it(dtype):
    g = torch.from_numpy(gradient((4, 80, 300), 7)).to(TYPES[dtype]).cuda()
    whole = orthogonalize(g, dtype)
    g[1] = 0
    g[2, 3, 5] = float("nan")
    for eps in (1e-7, 0.0):
        o = orthogonalize(g, dtype, eps=eps)
        assert torch.all(o[1] == 0)
        assert torch.isnan(o[2]).all()
    o = orthogonalize(g, dtype)
    assert torch.equal(o[0], whole[0]) and torch.equal(o[3], whole[3])
    assert torch.equal(orthogonalize(g.clone(), dtype), o) or torch.equal(o[0], whole[0])


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e18, 1e34])
def test_scale_of_the_gradient_does_not_matter(scale):
    # squares of these leave float32's range; eps = 0 since the norm itself may be tiny
    for dtype in ("bf16", "f32"):
        g = torch.from_numpy(gradient((1, 70, 90), 9, scale)).to(TYPES[dtype])
        o = np_of(orthogonalize(g.cuda(), dtype, eps=0.0)).astype(np.float64)
        assert_near(o[0], newton_schulz(g[0].double().numpy(), eps=0.0), dtype, f"{dtype} {scale}")


def coherent_bound(coefs=USUAL, phases=(3, 2)):
    """Relative error of the one singular value of a bf16 matrix of rank one (1 after the norm), to
    first order and with every float16 rounding (u, half a step) off by the most and none averaged
    out, as where all entries of a product are alike: X's high half in A, then per step P' = p - a,
    T and the next A, the join Q' = Q - a^j (a^3 = 41 beside a Q of 0.7), X between the phases."""
    a, b, c = coefs
    u, s, ex = 2.0 ** -11, 1.0, 0.0
    for n in phases:
        t, ea, q, eq, q0 = s * s, 2 * (ex + u) + u, 1.0, 0.0, 1.0
        for j in range(n):
            p = a + b * t + c * t * t
            ep = abs((b * t + 2 * c * t * t) / p) * ea + u * abs((p - a) / p)
            q, q0 = q * p, q0 * a
            eq += ep + (u * abs((q - q0) / q) if j else 0.0)
            ea, t = ea + 2 * ep + 2 * u, t * p * p
        s, ex = s * q, ex + eq + u
    return ex + 2.0 ** -8


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["one-entry", "rank-one", "orthogonal"])
def test_special_matrices(kind, dtype):
    rng = np.random.default_rng(3)
    n = 300
    if kind == "one-entry":
        g = np.zeros((1, n, n + 20), np.float32)
        g[0, 17, 200] = -3.0
    elif kind == "rank-one":   # powers of two: rank one in either type
        g = (2.0 ** rng.integers(-3, 4, (1, n, 1)) * 2.0 ** rng.integers(-3, 4, (1, 1, n + 20))).astype(np.float32)
    else:
        g = np.linalg.qr(rng.standard_normal((n, n)))[0][None].astype(np.float32)
    t = torch.from_numpy(g).to(TYPES[dtype])
    o = np_of(orthogonalize(t.cuda(), dtype)).astype(np.float64)
    ref = newton_schulz(t[0].double().numpy())
    if kind == "orthogonal" or dtype == "f32":
        assert_near(o[0], ref, dtype, kind)
    else:
        err = np.linalg.norm(o[0] - ref) / np.linalg.norm(ref)
        say(f"[muon]   {kind} error {err:.2e} of {coherent_bound():.2e}")
        assert err <= coherent_bound()


def test_the_result_may_overwrite_the_gradient():
    g = torch.from_numpy(gradient((2, 200, 333), 11)).to(torch.bfloat16).cuda()
    want = orthogonalize(g, "bf16")
    got = orthogonalize(g, "bf16", out=g)
    assert torch.equal(got, want)


UPDATES = [
    # shape, dtype, master, nesterov, decay
    ((2, 96, 160), "bf16", True, True, 0.1),
    ((2, 96, 160), "bf16", False, True, 0.1),
    ((3, 7, 5), "bf16", True, False, 0.0),
    ((1, 300, 270), "bf16", True, True, 0.0),
    ((2, 321, 130), "f32", False, True, 0.1),
    ((2, 130, 321), "f32", True, False, 0.1),
    ((1, 1, 33), "f32", False, True, 0.0),
]


@pytest.mark.parametrize("shape,dtype,master,nesterov,decay", UPDATES)
def test_muon_update(shape, dtype, master, nesterov, decay):
    say(f"[muon] update {shape} {dtype} master={master} nesterov={nesterov}")
    rng = np.random.default_rng(sum(shape))
    # the factors as the descriptor holds them, in float32
    mu, lr, scale, decay = (float(np.float32(v)) for v in (0.95, 2e-3, 0.2 * math.sqrt(max(shape[1:])), decay))
    w = torch.from_numpy((rng.standard_normal(shape) / math.sqrt(shape[2])).astype(np.float32))
    ref_w = w.double().numpy() if master else w.to(TYPES[dtype]).double().numpy()
    ref_m = np.zeros(shape)
    weight, mom = w.to(TYPES[dtype]).cuda(), torch.zeros(shape, device="cuda")
    mast = w.cuda() if master else None
    m = etd.make_muon_desc(*shape, dtype=dtype, momentum=mu, nesterov=nesterov, lr=lr, update_scale=scale,
                           weight_decay=decay)
    ws = torch.full((etd.moe_muon_workspace_size(m),), 255, dtype=torch.uint8, device="cuda")
    slack, off_m = 0.0, 0.0
    for step in range(3):
        g = torch.from_numpy(gradient(shape, 100 + step)).to(TYPES[dtype])
        etd.moe_muon_update(m, g.cuda(), mom, weight, ws, master=mast)
        torch.cuda.synchronize()
        g64 = g.double().numpy()
        # the momentum: the last error mu times, and two float32 roundings, half a step each, of
        # values no larger than the sum of the terms (1.01: products of errors)
        off_m = mu * off_m + 1.01 * 2 * 2.0 ** -24 * (mu * np.abs(ref_m) + np.abs(g64))
        ref_m = mu * ref_m + g64
        far = np.abs(np_of(mom).astype(np.float64) - ref_m) > off_m
        assert not far.any()
        ref_w = ref_w * (1.0 - lr * decay)
        for z in range(shape[0]):
            o = newton_schulz(g64[z] + mu * ref_m[z] if nesterov else ref_m[z])
            ref_w[z] -= lr * scale * o
        # the update's error by the tolerance of O, and the roundings of W: float32 (three) or the type
        kept = 3 * 2.0 ** -24 if (master or dtype == "f32") else 2.0 ** -8
        o_norm = 1.3 * math.sqrt(min(shape[1:]) * shape[0])   # singular values of O are below 1.3
        slack += lr * scale * TOL[dtype] * o_norm + kept * np.linalg.norm(ref_w)
        got = np_of(mast if master else weight).astype(np.float64)
        err = np.linalg.norm(got - ref_w)
        assert err <= slack, f"step {step}: {err} > {slack}"
        if master:
            assert torch.equal(weight, mast.to(TYPES[dtype]))


def newton_schulz_f64(u, steps=5, coefs=USUAL, eps=1e-7):
    """The formula on float64 matrices of the GPU, for sides that are slow on the CPU."""
    a, b, c = coefs
    x = u / (u.norm() + eps)
    for _ in range(steps):
        g = torch.mm(x, x.t().contiguous()) if x.shape[0] <= x.shape[1] else torch.mm(x.t().contiguous(), x)
        p = b * g + c * torch.mm(g, g)
        x = a * x + (torch.mm(p, x) if x.shape[0] <= x.shape[1] else torch.mm(x, p))
    return x


# stacks that fill the card: products of many tiles in one launch, odd sides, long K
@pytest.mark.parametrize("shape", [(14, 990, 1010), (16, 1010, 996), (16, 950, 4100), (1, 4100, 4100), (2, 2100, 4100),
                                   (40, 200, 1000), (130, 300, 290), (200, 70, 65), (33, 250, 130)])
def test_stacks_that_fill_the_card(shape):
    say(f"[muon] stack {shape}")
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    L, R, C = shape
    r = max(1, min(R, C) // 16)
    strong = torch.stack([torch.mm(torch.randn((R, r), device="cuda", generator=gen),
                                   torch.randn((r, C), device="cuda", generator=gen)) for _ in range(L)])
    g = (1e-3 * (strong / math.sqrt(r) + 0.25 * torch.randn(shape, device="cuda", generator=gen))).bfloat16()
    o = orthogonalize(g, "bf16")
    lr, scale, decay = (float(np.float32(v)) for v in (2e-3, 0.2 * math.sqrt(max(R, C)), 0.1))
    m = etd.make_muon_desc(*shape, momentum=0.95, nesterov=False, lr=lr, update_scale=scale, weight_decay=decay)
    ws = torch.full((etd.moe_muon_workspace_size(m),), 255, dtype=torch.uint8, device="cuda")
    w0 = torch.randn(shape, device="cuda", generator=gen) / math.sqrt(C)
    mast, weight, mom = w0.clone(), w0.bfloat16(), torch.zeros(shape, device="cuda")
    etd.moe_muon_update(m, g, mom, weight, ws, master=mast)
    alone = w0.bfloat16()
    etd.moe_muon_update(m, g, torch.zeros(shape, device="cuda"), alone, ws)
    torch.cuda.synchronize()
    assert torch.equal(mom, g.float())                    # of a momentum that was zero
    assert torch.equal(weight, mast.bfloat16())
    for z in sorted({0, L // 2, L - 1}):
        ref = newton_schulz_f64(g[z].double())
        n = float(ref.norm())
        err = float((o[z].double() - ref).norm()) / n
        say(f"[muon]   matrix {z} error {err:.2e}")
        assert err <= TOL["bf16"]
        want = w0[z].double() * (1.0 - lr * decay) - lr * scale * ref
        slack = lr * scale * TOL["bf16"] * n + 3 * 2.0 ** -24 * float(want.norm())
        assert float((mast[z].double() - want).norm()) <= slack
        # without a master the weight is rounded before and after, half a step each
        slack += 2 * 2.0 ** -8 * float(w0[z].norm() + lr * scale * n)
        assert float((alone[z].double() - want).norm()) <= slack


def test_zero_gradient_only_decays_the_weight():
    shape = (2, 40, 72)
    w = torch.randn(shape, device="cuda")
    m = etd.make_muon_desc(*shape, dtype="f32", lr=0.5, weight_decay=0.5)
    ws = torch.full((etd.moe_muon_workspace_size(m),), 255, dtype=torch.uint8, device="cuda")
    got, mom = w.clone(), torch.zeros(shape, device="cuda")
    etd.moe_muon_update(m, torch.zeros(shape, device="cuda"), mom, got, ws)
    assert torch.equal(got, w * 0.75) and torch.all(mom == 0)


def test_update_in_a_graph_between_eager_work():
    shape = (2, 270, 290)
    gen = torch.Generator(device="cuda").manual_seed(1)
    w0 = torch.randn(shape, device="cuda", generator=gen) * 0.05
    gs = [torch.from_numpy(gradient(shape, 40 + i)).to(torch.bfloat16).cuda() for i in range(4)]
    m = etd.make_muon_desc(*shape, lr=1e-3)
    n = etd.moe_muon_workspace_size(m)

    def fresh():
        return dict(g=gs[0].clone(), mom=torch.zeros(shape, device="cuda"), mast=w0.clone(), w=w0.bfloat16(),
                    ws=torch.empty(n, dtype=torch.uint8, device="cuda"))

    def step(s):
        etd.moe_muon_update(m, s["g"], s["mom"], s["w"], s["ws"], master=s["mast"])

    eager, cap = fresh(), fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cap)                                  # warm-up on another stream: the first step
    torch.cuda.synchronize()
    step(eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cap)
    for g in gs[1:]:
        for s in (eager, cap):
            s["g"].copy_(g)
        graph.replay()
        step(eager)
        torch.cuda.synchronize()
        for k in ("mom", "mast", "w"):
            assert torch.equal(eager[k], cap[k]), k


def test_one_workspace_for_stacks_of_different_shapes():
    shapes = [(2, 300, 280), (1, 20, 500), (3, 280, 300)]
    descs = [etd.make_muon_desc(*s) for s in shapes]
    ws = torch.full((max(etd.moe_muon_workspace_size(d) for d in descs),), 255, dtype=torch.uint8, device="cuda")
    gs = [torch.from_numpy(gradient(s, 60 + i)).to(torch.bfloat16).cuda() for i, s in enumerate(shapes)]
    outs = [torch.empty_like(g) for g in gs]
    for d, g, o in zip(descs, gs, outs):
        etd.moe_orthogonalize(d, g, o, ws)
    for g, o in zip(gs, outs):
        assert torch.equal(orthogonalize(g, "bf16"), o)


@pytest.mark.parametrize("layout", ["out_in", "in_out"])
def test_train_update_pack_and_serve(layout):
    """A training step, the update of the experts, their 4-bit copy and a forward on it."""
    s = synth.spec("gptoss_ep8_share", T=300, H=320, I=288, E=8, k=2, L=8, weight_layout=layout)
    inp = synth.make_layer(s)
    layer, x = layer_of(inp)
    before = {n: getattr(layer, n).double().cpu().numpy() for n in layer.MUON_WEIGHTS}
    state = layer.muon_state()
    y, saved = layer.forward_train(x)
    grads = layer.backward(x, saved, torch.randn_like(y))
    layer.muon_update(grads, state, lr=1e-2)
    packed = layer.pack_experts()
    served = layer.forward_packed(x, packed)
    torch.cuda.synchronize()
    for n in layer.MUON_WEIGHTS:
        g = grads["d" + n].double().cpu().numpy()
        got = np_of(state["master"][n]).astype(np.float64)
        scale = 0.2 * math.sqrt(max(g.shape[1:]))
        ref = np.stack([before[n][z] - 1e-2 * scale * newton_schulz(1.95 * g[z]) for z in range(len(g))])
        o_norm = 1.3 * math.sqrt(min(g.shape[1:]) * len(g))
        assert np.linalg.norm(got - ref) <= 1e-2 * scale * TOL["bf16"] * o_norm + 3 * 2.0 ** -24 * np.linalg.norm(ref)
        assert torch.equal(getattr(layer, n), state["master"][n].bfloat16())
        w = got.transpose(0, 2, 1) if layout == "in_out" else got
        t = packed._tensors
        v = values_of(t[n[2:] + "_codes"].cpu().numpy(), t[n[2:] + "_scales"].cpu().numpy())
        assert np.linalg.norm(v - w) < 0.2 * np.linalg.norm(w)   # half a step of a code is at most a quarter of it
    # the forward on the codes equals the forward on the weights they stand for
    for n in layer.MUON_WEIGHTS:
        t = packed._tensors
        etd.moe_unpack_weights(t[n[2:] + "_codes"], t[n[2:] + "_scales"], getattr(layer, n), weight_layout=layout)
    plain = layer.forward(x)
    a, b = np_of(served).astype(np.float64), np_of(plain).astype(np.float64)
    assert np.linalg.norm(a - b) <= 2 * 2.0 ** -7 * np.linalg.norm(b)   # each: h and y rounded once


@pytest.mark.parametrize("shape", [(14, 990, 1010), (4, 300, 290), (5, 60, 200)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_gradient_that_is_not_finite_spoils_its_own_matrix_only(shape, bad):
    gen = torch.Generator(device="cuda").manual_seed(11)
    g = (1e-3 * torch.randn(shape, device="cuda", generator=gen)).bfloat16()
    w0 = torch.randn(shape, device="cuda", generator=gen)
    m = etd.make_muon_desc(*shape, lr=1e-2)
    ws = torch.full((etd.moe_muon_workspace_size(m),), 255, dtype=torch.uint8, device="cuda")

    def step(grad):
        mast, w, mom = w0.clone(), w0.bfloat16(), torch.zeros(shape, device="cuda")
        etd.moe_muon_update(m, grad, mom, w, ws, master=mast)
        return mast, w, mom

    ref = step(g)
    broken = g.clone()
    broken[2, shape[1] - 1, 1] = bad
    got = step(broken)
    torch.cuda.synchronize()
    others = [z for z in range(shape[0]) if z != 2]
    for a, b in zip(got, ref):
        assert torch.equal(a[others], b[others])
    assert not torch.isfinite(got[0][2]).any()


def test_two_updates_at_once_on_two_streams():
    shapes = [(6, 520, 600), (14, 990, 1010)]
    gen = torch.Generator(device="cuda").manual_seed(12)
    sets = []
    for s in shapes:
        m = etd.make_muon_desc(*s, lr=1e-2)
        sets.append((m, (1e-3 * torch.randn(s, device="cuda", generator=gen)).bfloat16(),
                     torch.randn(s, device="cuda", generator=gen)))

    def run(m, g, w0, stream):
        ws = torch.empty(etd.moe_muon_workspace_size(m), dtype=torch.uint8, device="cuda")
        mast, w, mom = w0.clone(), w0.bfloat16(), torch.zeros_like(w0)
        torch.cuda.synchronize()
        return mast, lambda: etd.moe_muon_update(m, g, mom, w, ws, master=mast, stream=stream)

    want = []
    for s in sets:
        mast, call = run(*s, None)
        for _ in range(3):
            call()
        want.append(mast)
    streams = [torch.cuda.Stream() for _ in sets]
    pairs = [run(*s, st) for s, st in zip(sets, streams)]
    for _ in range(3):
        for _, call in pairs:
            call()
    torch.cuda.synchronize()
    for (mast, _), ref in zip(pairs, want):
        assert torch.equal(mast, ref)


def test_a_stack_of_more_than_2_to_31_elements():
    shape = (2100, 1024, 1024)
    gen = torch.Generator(device="cuda").manual_seed(13)
    g = torch.randn(shape, device="cuda", generator=gen, dtype=torch.bfloat16)
    w = torch.zeros(shape, device="cuda", dtype=torch.bfloat16)
    mom = torch.zeros(shape, device="cuda")
    m = etd.make_muon_desc(*shape, momentum=0.5, nesterov=False, lr=1.0, update_scale=-1.0)
    ws = torch.empty(etd.moe_muon_workspace_size(m), dtype=torch.uint8, device="cuda")
    etd.moe_muon_update(m, g, mom, w, ws)       # from zero weights: W is the orthogonalised gradient
    torch.cuda.synchronize()
    for z in (0, 1050, 2047, 2048, 2099):
        assert torch.equal(mom[z], g[z].float())
        ref = newton_schulz_f64(g[z].double())
        assert float((w[z].double() - ref).norm() / ref.norm()) <= TOL["bf16"]
