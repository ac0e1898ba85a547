"""Every product kernel of the experts with adapters, by shapes that are known to take it: values, isolation, the low
part of what stands between the two low products, and infinities in an adapter."""

import numpy as np
import pytest

from tests._adapted_paths import CASES, kernel_of
from tests._harness import say
from tests.test_gpu_adapters import Case, layer_case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import expert_token_dispatch_amd as etd  # noqa: E402

LARGE = [c for c in CASES if c[0] == "large" and c[5] == "out_in"]


def some_rows(c):
    """The first and last rows of every segment and those around the tiles' borders."""
    rows = set()
    for a, b in zip(c.off[:-1], c.off[1:]):
        for at in range(0, b - a, 128):
            rows.update(range(a + max(at - 2, 0), min(a + at + 3, b)))
        rows.update(range(max(a, b - 20), b))
    return np.array(sorted(rows))


@pytest.mark.parametrize("R", (8, 16, 72))
@pytest.mark.parametrize("kind", ("mixed", "runs"))
@pytest.mark.parametrize("kernel,H,I,Lc,P,layout,spread", LARGE)
def test_values_of_the_large_tile_with_weights_along_k(kernel, H, I, Lc, P, layout, spread, kind, R):
    assert kernel_of(H, I, Lc, P, layout, R) == kernel
    c = Case(H, I, Lc, P, R, 5, layout=layout, spread=spread, kind=kind, seed=R)
    c.check(f"large tile {kind}", rows=some_rows(c))


@pytest.mark.parametrize("R,n,broken", [(16, 7, 3), (40, 5, 0)])
@pytest.mark.parametrize("kernel,H,I,Lc,P,layout,spread", LARGE)
def test_a_broken_adapter_in_the_large_tile(kernel, H, I, Lc, P, layout, spread, R, n, broken):
    c = Case(H, I, Lc, P, R, n, layout=layout, spread=spread, seed=R)
    say(f"[adapters] large tile, one broken of {n}: {(H, I, Lc, P)}")
    base = c.run()
    rows = torch.tensor((c.ids != broken)[c.pairs.cpu().numpy()], device="cuda")
    for k, v in c.t.items():
        if k.endswith("_b"):
            v[broken, :, ::3] = float("nan")
        elif k.endswith("_a"):
            v[broken, :, ::2, 1] = float("inf")
    y = c.run()
    assert torch.isfinite(base).all() and torch.equal(y[rows], base[rows])
    assert torch.isnan(y[~rows]).any(dim=1).all()


@pytest.mark.parametrize("layout,dtype", [("out_in", "bf16"), ("in_out", "bf16"), ("out_in", "f32")])
@pytest.mark.parametrize("spread", ("one", "skew"))
@pytest.mark.parametrize("P", (65, 250))
@pytest.mark.parametrize("H,I,Lc", [(128, 200, 8), (64, 2048, 32), (2048, 64, 64)])
def test_more_than_64_rows_on_an_expert_in_the_decode_kernel(H, I, Lc, P, spread, layout, dtype):
    """Its rows go 64 at a time: with waves that split K (the first shape) and whole ones (the others' wide product)."""
    assert kernel_of(H, I, Lc, P, layout, dtype=dtype) == "decode"
    c = Case(H, I, Lc, P, 16, 20, dtype, layout, spread)
    assert c.counts.max() > 64 or spread == "skew"
    c.check(f"decode kernel, {c.counts.max()} rows on one expert")


def one_hot(Lc, N, K, of, value=1.0):
    """[Lc, N, K] with `value` at column of(n) of row n."""
    w = torch.zeros(Lc, N, K, dtype=torch.bfloat16, device="cuda")
    w[:, torch.arange(N), of(torch.arange(N))] = value
    return w


class Picking:
    """Weights and adapters that pick columns, so that results are known without a product's rounding.  With an adapter,
    projection `p` in `has` is  sum_r s v[col(r)] [r = n mod R] - v[col(n mod R)] = (s - 1) v[col(n mod R)]  at output n;
    without one, -v[col(n mod R)].  s - 1 is 0 or +-2^-10..2^-12 and v a bfloat16: the high part of s v is v, the low part
    (s - 1) v, both exact.  The other projections are v at some column."""

    def __init__(self, H, I, Lc, P, layout, spread, R, has, scales):
        n = len(scales)
        c = self.c = Case(H, I, Lc, P, R, n, layout=layout, spread=spread, has=has)
        g = torch.Generator(device="cuda").manual_seed(R)
        sign = torch.where(torch.rand((P, H), generator=g, device="cuda") < 0.5, -1.0, 1.0)
        c.x = (sign * (0.5 + torch.rand((P, H), generator=g, device="cuda"))).bfloat16()
        c.t["scale"] = torch.tensor(scales, device="cuda")
        self.cols = {}
        for i, (name, N, K) in enumerate((("gate", I, H), ("up", I, H), ("down", H, I))):
            if name in has:
                def of(m, K=K, i=i):
                    return (7 * (m % R) + 3 + 2 * i) % K
                w = one_hot(Lc, N, K, of, -1.0)
                c.t[name + "_a"] = one_hot(Lc, R, K, of).expand(n, Lc, R, K).contiguous()
                c.t[name + "_b"] = one_hot(Lc, N, R, lambda m: m % R).expand(n, Lc, N, R).contiguous()
            else:
                def of(m, K=K, i=i):
                    return (3 * m + i) % K
                w = one_hot(Lc, N, K, of)
            self.cols[name] = of(torch.arange(N))
            c.w[name] = w if layout == "out_in" else w.transpose(1, 2).contiguous()
        self.has = has
        self.ids = torch.tensor(c.ids[c.pairs.cpu().numpy()], device="cuda")
        self.factor = torch.where(self.ids < 0, -1.0, c.t["scale"].double()[self.ids.clamp(min=0)] - 1.0)[:, None]

    def project(self, name, v):
        v = v[:, self.cols[name].cuda()]
        return self.factor * v if name in self.has else v

    def h(self):
        x = self.c.x.double()
        g, u = self.project("gate", x), self.project("up", x)
        return g / (1.0 + torch.exp(-g)) * u

    def y(self):
        return self.project("down", self.h())


# h is rounded once (2^-8 of it) after the gate's exponential, reciprocal and three products, under 32 units of
# 2^-24; y is h, or h times a power of two, or their negative: exact.
PICKED = 2.0 ** -8 + 32 * 2.0 ** -24


@pytest.mark.parametrize("R", (8, 72))
@pytest.mark.parametrize("has", [("gate",), ("up",), ("down",), ("gate", "up")])
@pytest.mark.parametrize("kernel,H,I,Lc,P,layout,spread", CASES)
def test_the_low_part_of_the_first_products(kernel, H, I, Lc, P, layout, spread, has, R):
    """Where the high parts cancel against the shared weights, the low parts alone are the result."""
    assert kernel_of(H, I, Lc, P, layout, R) == kernel
    say(f"[adapters] low part of {has}: {kernel} {(H, I, Lc, P, R)} {layout}")
    p = Picking(H, I, Lc, P, layout, spread, R, has, [1 + 2.0 ** -10, 1 - 2.0 ** -11, 1 + 2.0 ** -12])
    got, want = p.c.run().double(), p.y()
    assert (want != 0).all()
    worst = ((got - want).abs() / want.abs()).max()
    assert worst <= PICKED, f"off by {worst}"
    if "down" not in has:
        return
    rows = (p.ids == 1).nonzero()[:, 0]  # the same numbers to the bit from 2^11 times as much of h
    exact = -(2.0 ** -11) * p.c.plain().double()[rows] * -1.0
    assert torch.equal(got[rows], exact)


@pytest.mark.parametrize("kernel,H,I,Lc,P,layout,spread", CASES)
def test_infinities_in_an_adapter_give_what_the_sum_gives(kernel, H, I, Lc, P, layout, spread):
    """u B^T with an infinity in B is that infinity times u's sign, whatever the low part of u is (none, of u's sign, of
    the other); the adapter's other columns and the other adapters' rows are what they were."""
    assert kernel_of(H, I, Lc, P, layout, 24) == kernel
    say(f"[adapters] infinities: {kernel} {(H, I, Lc, P)} {layout}")
    p = Picking(H, I, Lc, P, layout, spread, 24, ("down",), [1.0, 1 + 2.0 ** -10, 1 - 2.0 ** -10, 1.0])
    base = p.c.run().double()
    b = p.c.t["down_b"]
    n = torch.arange(0, H, 3, device="cuda")
    b[:3, :, n, n % 24] = float("inf")
    y, h = p.c.run().double(), p.h()
    broken = ((p.ids >= 0) & (p.ids < 3))[:, None] & (torch.arange(H, device="cuda") % 3 == 0)
    assert broken.any() and torch.equal(y[~broken], base[~broken])
    want = torch.sign(h[:, p.cols["down"].cuda()]) * float("inf")
    assert torch.equal(y[broken], want[broken])


@pytest.mark.parametrize("spread", ("one", "skew"))
@pytest.mark.parametrize("kernel,H,I,Lc,P,layout,_", CASES)
def test_uneven_segments_in_every_kernel(kernel, H, I, Lc, P, layout, _, spread):
    c = Case(H, I, Lc, P, 16, 5, layout=layout, spread=spread)
    c.check(f"{kernel} {spread}", rows=some_rows(c))


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("kernel,H,I,Lc,P,layout,_", CASES)
def test_no_row_for_any_of_a_ranks_experts(kernel, H, I, Lc, P, layout, _, dtype):
    """The descriptor allows P rows, the batch sends none: nothing is read as a row, nothing written."""
    say(f"[adapters] no rows: {(H, I, Lc, P)} {layout} {dtype}")
    c = Case(H, I, Lc, P, 16, 5, dtype, layout)
    c.offsets.zero_()
    assert (c.run() == 7.0).all()


def test_the_most_adapters_and_the_highest_rank():
    say("[adapters] 65535 adapters; rank 128")
    c = Case(16, 8, 2, 40, 8, 65535)
    ids = np.arange(40) * 1679 % 65535
    ids[::5] = 65534
    ids[1::5] = 65535  # past the last: none
    c.set_ids(ids)
    c.check("65535 adapters")
    Case(264, 136, 2, 700, 128, 3, kind="mixed").check("rank 128")


def test_the_layer_with_route_options_is_its_stages():
    T, E, k = 300, 16, 4
    layer, ad, ids, x = layer_case(T, 128, 192, E, k)
    bias = torch.linspace(-1, 1, E, device="cuda")
    opts = etd.make_route_opts(bias, 4, 2)
    y = layer.forward_adapted(x, ad, ids, opts=opts)
    r = layer.route(x, opts=opts)
    dd = layer.dispatch(x, r["topk_ids"])
    ys = layer.grouped_ffn_adapted(dd["x_sorted"], dd["offsets"], dd["sorted_pairs"], ad, ids)
    z = layer.combine(ys, dd["pair_row"], r["topk_w"])
    torch.cuda.synchronize()
    assert torch.equal(y, z) and not torch.equal(y, layer.forward_adapted(x, ad, ids))
