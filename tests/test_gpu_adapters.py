"""The experts with adapters of many requests on the GPU against the float64 oracle, by the framework's
measures of a row (float32 1e-5 of its largest entry, bf16 2e-2 of its norm), and what has to be equal bit for bit:
a row does not depend on the other rows' adapters, and where the plain experts take the same kernels, rows
without an adapter are theirs."""

import numpy as np
import pytest

from oracle import adapters as oa
from tests._harness import row_error, say, tol

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import expert_token_dispatch_amd as etd  # noqa: E402
from expert_token_dispatch_amd import _lib as L  # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ALL = ("gate", "up", "down")


def counts_of(rng, Lc, P, spread):
    if spread == "even":
        return np.bincount(rng.integers(0, Lc, P), minlength=Lc)
    if spread == "one":      # every row to one expert in the middle
        return np.eye(Lc, dtype=np.int64)[Lc // 2] * P
    w = 1.0 / (1 + np.arange(Lc))
    return np.bincount(rng.choice(Lc, P, p=w / w.sum()), minlength=Lc)


class Case:
    """Tensors of one call, k = 1: row q's token is pairs[q]."""

    def __init__(self, H, I, Lc, P, R, n, dtype="bf16", layout="out_in", spread="even", kind="mixed", has=ALL, scale=True,
                 seed=0, behind=0):
        g = torch.Generator(device="cuda").manual_seed(seed + 7 * P + H)
        rng = np.random.default_rng(seed + 3 * P + I)
        self.dims, self.dtype, self.P = (H, I, Lc, R, n), dtype, P
        self.d = etd.make_desc(P + behind, H, I, Lc, 1, dtype=dtype, weight_layout=layout)
        self.counts = counts_of(rng, Lc, P, spread)
        self.off = np.concatenate([[0], self.counts.cumsum()])
        self.offsets = torch.tensor(self.off, dtype=torch.int32, device="cuda")
        pairs = np.concatenate([rng.permutation(P), np.arange(P, P + behind)])
        for e in range(Lc):  # ascending in every segment, as the dispatch leaves them
            pairs[self.off[e]:self.off[e + 1]].sort()
        self.pairs = torch.tensor(pairs, dtype=torch.int32, device="cuda")
        T = P + behind
        if kind == "mixed":
            ids = rng.integers(-1, n, T)
        elif kind == "runs":
            ids = np.sort(rng.integers(0, n, T))
        elif kind == "none":
            ids = np.full(T, -1)
        else:
            ids = np.full(T, kind)
        self.set_ids(ids)

        def rand(*shape):
            return torch.randn(shape, generator=g, device="cuda")
        self.x = rand(T, H).to(DT[dtype])
        self.w, t = {}, {}
        for name, N, K in (("gate", I, H), ("up", I, H), ("down", H, I)):
            w = (rand(Lc, N, K) * K ** -0.5).to(DT[dtype])
            self.w[name] = w if layout == "out_in" else w.transpose(1, 2).contiguous()
            if name in has:
                t[name + "_a"] = (rand(n, Lc, R, K) * K ** -0.5).to(DT[dtype])
                t[name + "_b"] = (rand(n, Lc, N, R) * 0.5 * R ** -0.5).to(DT[dtype])
        if scale:
            t["scale"] = 0.5 + torch.rand(n, generator=g, device="cuda")
        self.t, self.layout = t, layout

    def set_ids(self, ids):
        self.ids = np.asarray(ids)
        self.adapter_ids = torch.tensor(self.ids, dtype=torch.int32, device="cuda")

    def run(self, ws=None, stream=None):
        y = torch.full_like(self.x, 7.0)
        ad = etd.make_adapters(self.t)
        if ws is None:
            ws = torch.empty(etd.moe_adapted_workspace_size(self.d, ad, L.MOE_STAGE_FFN), dtype=torch.uint8, device="cuda").fill_(255)
        etd.moe_grouped_ffn_adapted(self.d, self.x, self.offsets, self.pairs, self.adapter_ids, self.w["gate"], self.w["up"],
                                    self.w["down"], ad, y, ws, stream=stream)
        torch.cuda.synchronize()
        return y

    def plain(self):
        y = torch.full_like(self.x, 7.0)
        n = etd.moe_workspace_size(self.d, L.MOE_STAGE_FFN)
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        etd.moe_grouped_ffn(self.d, self.x, self.offsets, self.w["gate"], self.w["up"], self.w["down"], y, ws=ws)
        torch.cuda.synchronize()
        return y

    def reference(self, rows=None):
        """Of all rows, or of some alone."""
        def h(t):
            return t.double().cpu().numpy()
        H, I, Lc, R, n = self.dims
        w = {k: h(v) if self.layout == "out_in" else h(v).transpose(0, 2, 1) for k, v in self.w.items()}
        ad = {k: h(v) for k, v in self.t.items() if k != "scale"}
        scale = h(self.t["scale"]) if "scale" in self.t else np.ones(n)
        pairs = self.pairs.cpu().numpy()
        x, ids, off = h(self.x)[:self.P], self.ids[pairs][:self.P], self.off
        if rows is not None:
            x, ids, off = x[rows], ids[rows], np.searchsorted(rows, self.off)
        return oa.grouped_ffn(x, off, ids, w, ad, scale)

    def check(self, what, rows=None):
        say(f"[adapters] {what}: H I L R n {self.dims} P {self.P} {self.dtype} {self.layout}")
        y = self.run().double().cpu().numpy()
        ref = self.reference(rows)
        got = y[:self.P] if rows is None else y[rows]
        e = row_error(got, ref, self.dtype)
        assert np.isfinite(got).all() and e <= tol(self.dtype), f"{what}: row error {e}"
        assert (y[self.P:] == 7.0).all(), "a row behind the last segment was written"


# H, I, L, P, R, n: few rows and many, on and off the tiles' sizes
SHAPES = [
    (8, 8, 1, 1, 8, 1), (64, 64, 1, 1, 16, 1), (64, 96, 4, 3, 16, 5), (40, 72, 3, 50, 24, 4), (256, 128, 8, 17, 16, 3),
    (96, 160, 5, 130, 32, 7), (512, 256, 8, 200, 8, 5), (320, 320, 2, 64, 128, 3), (128, 384, 16, 333, 40, 33),
    (136, 264, 3, 500, 16, 9), (64, 64, 2, 700, 8, 2), (256, 512, 4, 1100, 16, 6), (576, 320, 2, 900, 64, 3),
    (1000, 72, 4, 60, 16, 3), (104, 1096, 5, 9, 8, 2), (2056, 24, 2, 2, 24, 2), (88, 520, 50, 70, 16, 4),
    (192, 448, 3, 1500, 128, 2), (72, 1000, 8, 200, 16, 5), (264, 200, 1, 65, 40, 3), (520, 136, 3, 900, 24, 4),
    (136, 2056, 2, 1300, 72, 3), (64, 2944, 4, 2100, 16, 6), (40, 8, 300, 6000, 8, 3), (40, 72, 300, 10000, 8, 3), (128, 64, 40, 600, 48, 12), (256, 256, 1, 2000, 104, 5),
]


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("layout", ("out_in", "in_out"))
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, layout, dtype):
    H, I, Lc, P, R, n = shape
    Case(H, I, Lc, P, R, n, dtype, layout, behind=P % 3).check("shape")


@pytest.mark.parametrize("spread", ("one", "skew"))
@pytest.mark.parametrize("kind", ("mixed", "runs"))
@pytest.mark.parametrize("P", (40, 333, 1200))
def test_spreads(P, kind, spread):
    Case(128, 192, 8, P, 16, 20, spread=spread, kind=kind).check(f"{spread} {kind}")


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("P", (9, 300, 1000))
@pytest.mark.parametrize("has", (("gate",), ("up",), ("down",), ("gate", "down"), ("up", "down"), ("gate", "up")))
def test_projections_without_adapters(has, P, dtype):
    Case(128, 192, 2, P, 16, 3, dtype, has=has, scale=P != 300).check(str(has))


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("layout", ("out_in", "in_out"))
@pytest.mark.parametrize("shape", [(2048, 768, 100, 300), (2048, 768, 128, 512), (136, 264, 3, 200), (256, 4096, 4, 2400),
                                   (4096, 4096, 2, 2200)])
def test_without_an_adapter_a_row_is_the_plain_experts(shape, layout, dtype):
    """At sizes where the plain experts take the kernels that the adapted ones take."""
    H, I, Lc, P = shape
    if (dtype, layout) == ("f32", "out_in") and P <= 32 * Lc or (dtype, layout) == ("bf16", "out_in") and H % 64:
        pytest.skip("rows of this number and type take a kernel that the plain experts do not have")
    c = Case(H, I, Lc, P, 16, 3, dtype, layout, kind="none")
    say(f"[adapters] none {shape} {layout} {dtype}")
    plain = c.plain()
    assert torch.equal(c.run(), plain)
    odd = np.array([-1, 3, 1 << 30, -(1 << 31), (1 << 31) - 1])  # outside [0, count)
    c.set_ids(odd[np.arange(P) % 5])
    assert torch.equal(c.run(), plain)
    ids = np.full(P, -1)
    ids[::7] = 1
    c.set_ids(ids)
    rows = ids[c.pairs.cpu().numpy()] < 0
    y = c.run()
    assert torch.equal(y[torch.tensor(rows, device="cuda")], plain[torch.tensor(rows, device="cuda")])


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("layout", ("out_in", "in_out"))
@pytest.mark.parametrize("I", (192, 200))
@pytest.mark.parametrize("P", (30, 200, 1200))
def test_a_row_depends_on_no_other_request(P, I, layout, dtype):
    """Other requests' adapters change, and one of them holds NaN and infinities: not a bit of the others' rows."""
    H, Lc, R, n = 128, 2, 24, 6
    c = Case(H, I, Lc, P, R, n, dtype, layout)
    say(f"[adapters] isolation P={P} I={I} {layout} {dtype}")
    base = c.run()
    keep = c.ids % 2 == 0                    # adapters 0, 2, 4 stay
    c.set_ids(np.where(keep, c.ids, 5))
    rows = torch.tensor(keep[c.pairs.cpu().numpy()], device="cuda")
    for k, v in c.t.items():
        if k != "scale":
            v[5] = float("nan") if k.endswith("_a") else float("inf")
    y = c.run()
    assert torch.equal(y[rows], base[rows])
    assert not torch.isfinite(y[~rows]).any()
    assert torch.isfinite(base).all()


@pytest.mark.parametrize("I", (192, 200))
@pytest.mark.parametrize("P", (30, 200, 1200))
@pytest.mark.parametrize("R,n,broken", [(8, 7, 3), (16, 8, 0), (16, 2, 1), (40, 5, 4)])
def test_a_broken_adapter_beside_each_of_the_others(R, n, broken, P, I):
    """Every tile has all adapters in changing orders, one of them with NaN in its B alone: the rows of the others
    are what they are without it."""
    c = Case(128, I, 2, P, R, n, seed=R)
    say(f"[adapters] one broken of {n}, rank {R}, P={P} I={I}")
    c.check("whole")
    base = c.run()
    rows = torch.tensor((c.ids != broken)[c.pairs.cpu().numpy()], device="cuda")
    for k, v in c.t.items():
        if k.endswith("_b"):
            v[broken, :, ::3] = float("nan")
    y = c.run()
    assert torch.equal(y[rows], base[rows])
    assert torch.isnan(y[~rows]).any(dim=1).all()


def test_the_same_every_time_on_other_streams_and_two_at_once():
    a, b = Case(256, 512, 4, 1100, 16, 6), Case(128, 192, 8, 60, 8, 9, seed=5)
    ya, yb = a.run(), b.run()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        outs = []
        for c, s in ((a, sa), (b, sb)):
            ad = etd.make_adapters(c.t)
            ws = torch.empty(etd.moe_adapted_workspace_size(c.d, ad, L.MOE_STAGE_FFN), dtype=torch.uint8, device="cuda").fill_(255)
            y = torch.empty_like(c.x)
            s.wait_stream(torch.cuda.current_stream())
            etd.moe_grouped_ffn_adapted(c.d, c.x, c.offsets, c.pairs, c.adapter_ids, c.w["gate"], c.w["up"], c.w["down"], ad, y,
                                        ws, stream=s)
            outs.append((y, ws))
        torch.cuda.synchronize()
        assert torch.equal(outs[0][0], ya) and torch.equal(outs[1][0], yb)


def test_adapters_past_32_bit_offsets():
    """The last of the adapters starts past 2^31 elements of every stack."""
    H, I, Lc, R, n = 4096, 4096, 16, 128, 280
    c = Case(H, I, Lc, 6, R, 1, kind="none", has=())
    say("[adapters] stacks past 32-bit offsets")
    g = torch.Generator(device="cuda").manual_seed(1)
    small = {}
    for name in ALL:
        for side, shape in (("_a", (n, Lc, R, H)), ("_b", (n, Lc, H, R))):
            t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
            t[-1] = (torch.randn(shape[1:], generator=g, device="cuda") * 0.02).bfloat16()
            c.t[name + side], small[name + side] = t, t[-1:].contiguous()
    assert n * Lc * R * H > 1 << 31
    c.t["scale"] = torch.ones(n, device="cuda")
    c.set_ids([n - 1] * 6)
    y = c.run()
    c.t = {**small, "scale": torch.ones(1, device="cuda")}
    c.dims = (H, I, Lc, R, 1)
    c.set_ids([0] * 6)
    assert torch.equal(c.run(), y)
    assert not torch.equal(c.plain(), y)


def layer_case(T, H, I, E, k, dtype="bf16", cap=0.0, lo=0, Lc=None, n=5, R=16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    Lc = E if Lc is None else Lc

    def rand(*shape, s=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * s).to(DT[dtype])
    d = etd.make_desc(T, H, I, E, k, lo, Lc, cap, dtype)
    layer = etd.MoELayer(d, rand(E, H, s=H ** -0.5), None, rand(Lc, I, H, s=H ** -0.5), rand(Lc, I, H, s=H ** -0.5),
                         rand(Lc, H, I, s=I ** -0.5))
    t = {}
    for name, N, K in (("gate", I, H), ("up", I, H), ("down", H, I)):
        t[name + "_a"], t[name + "_b"] = rand(n, Lc, R, K, s=K ** -0.5), rand(n, Lc, N, R, s=0.1)
    t["scale"] = torch.rand(n, generator=g, device="cuda") + 0.5
    ids = torch.randint(-1, n, (T,), generator=g, device="cuda").to(torch.int32)
    return layer, etd.make_adapters(t), ids, rand(T, H)


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("T,cap,lo,Lc", [(1, 0.0, 0, None), (5, 0.0, 0, None), (700, 0.0, 0, None), (700, 0.8, 2, 4)])
def test_the_layer_is_its_stages(T, cap, lo, Lc, dtype):
    layer, ad, ids, x = layer_case(T, 128, 192, 8, 2, dtype, cap, lo, Lc)
    say(f"[adapters] layer T={T} cap={cap} {dtype}")
    dropped = torch.zeros(1, dtype=torch.int64, device="cuda")
    counts = torch.zeros(8, dtype=torch.int32, device="cuda")
    y = layer.forward_adapted(x, ad, ids, counts_out=counts, num_dropped_out=dropped)
    r = layer.route(x, want_topk_logit=True)
    dd = layer.dispatch(x, r["topk_ids"], r["topk_logit"])
    ys = layer.grouped_ffn_adapted(dd["x_sorted"], dd["offsets"], dd["sorted_pairs"], ad, ids)
    z = layer.combine(ys, dd["pair_row"], r["topk_w"])
    torch.cuda.synchronize()
    assert torch.equal(y, z) and torch.equal(counts, dd["counts"]) and torch.equal(dropped, dd["num_dropped"])
    # and against 64 bits, pair by pair
    h = lambda t: t.double().cpu().numpy()  # noqa: E731
    n = int(dd["offsets"][-1])
    pairs = dd["sorted_pairs"].cpu().numpy()[:n]
    ref = oa.grouped_ffn(h(dd["x_sorted"])[:n], dd["offsets"].cpu().numpy(), ids.cpu().numpy()[pairs // 2],
                         {"gate": h(layer.w_gate), "up": h(layer.w_up), "down": h(layer.w_down)},
                         {k: h(v) for k, v in ad._tensors.items()}, h(ad._tensors["scale"]))
    assert row_error(h(ys)[:n], ref, dtype) <= tol(dtype)
    assert not torch.equal(y, layer.forward(x))


@pytest.mark.parametrize("T", (4, 600))
def test_captured_and_replayed(T):
    layer, ad, ids, x = layer_case(T, 256, 320, 8, 2)
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward_adapted(x, ad, ids, y=y)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward_adapted(x, ad, ids, y=y)
    for r in range(4):
        x.mul_(0.9)
        ids.copy_(torch.roll(ids, r))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, layer.forward_adapted(x, ad, ids)), f"replay {r}"


def test_a_block_of_a_model_served_to_many_requests():
    """norm -> the layer with every token's adapter -> norm, gate, sum and the next norm, as a model runs them."""
    T, H = 50, 128
    layer, ad, ids, x = layer_case(T, H, 192, 8, 2, "f32")
    w = [1 + 0.1 * torch.randn(H, device="cuda") for _ in range(3)]
    gate = torch.randn(T, device="cuda")
    first = etd.BlockJoin(H, "f32", w_pre=w[0])
    after = etd.BlockJoin(H, "f32", w_post=w[1], w_pre=w[2], gate="token", gate_act="sigmoid", residual_scale=0.5)
    _, h = first.forward(x)
    y = layer.forward_adapted(h, ad, ids)
    z, h2 = after.forward(x, y, gate)
    torch.cuda.synchronize()

    def norm(v, f):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * f
    X, W = x.double(), [t.double() for t in w]
    Z = X + 0.5 * torch.sigmoid(gate.double())[:, None] * norm(y.double(), W[1])
    for got, want in ((h, norm(X, W[0])), (z, Z), (h2, norm(Z, W[2]))):
        assert (got.double() - want).abs().max() <= 1e-5 * want.abs().max()
