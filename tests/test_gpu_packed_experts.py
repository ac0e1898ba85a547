"""Expert weights in 4 bits on the GPU: packing and unpacking against the format's
definition in 64 bits, the packed feed-forward against the 64-bit formula on the unpacked
values, the packed layer against the oracle on those values."""

import numpy as np
import pytest

import oracle
import synth
from tests._harness import layer_of, np_of, row_error, say, tol

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import expert_token_dispatch_amd as etd  # noqa: E402

MAG = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def values_of(codes, scales):
    """The weights that uint8 codes [..., K/2] and scales [..., K/32] stand for, float64."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.where(c & 8, -1.0, 1.0) * MAG[c & 7]
    e = np.repeat(scales.astype(np.int64), 32, -1)
    return np.where(e == 255, np.nan, np.ldexp(v, np.where(e == 255, 0, e - 127)))


def packed_by_definition(w):
    """float64 w [..., K] -> values after packing: nearest of the 16 codes, ties to the even one."""
    g = w.reshape(*w.shape[:-1], -1, 32)
    top = np.abs(g).max(-1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.clip(np.frexp(top)[1] - 1 - 2, -127, 127)
        q = np.abs(np.ldexp(g, -e))
        d = np.abs(np.minimum(q, 6.0)[..., None] - MAG)
        near = d == d.min(-1, keepdims=True)
    code = np.where(near[..., ::2].any(-1), 2 * near[..., ::2].argmax(-1), near.argmax(-1))
    v = np.ldexp(MAG[code], e) * np.where(np.signbit(g), -1.0, 1.0)
    return np.where(np.isfinite(top), v, np.nan).reshape(w.shape)


def stack_with_edges(shape, dtype, seed):
    """A stack [count, out, in]; some groups are zero, tied, tiny, huge or not finite."""
    rng = np.random.default_rng(seed)
    w = rng.standard_normal(shape).astype(np.float32)
    flat = w.reshape(-1, 32)
    n = len(flat)
    edge = [np.zeros(32), np.full(32, -0.0), np.resize([4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5, -0.25], 32),
            flat[0] * 2.0 ** -100, flat[0] * 2.0 ** 100, np.r_[7.9, flat[0][1:]], np.full(32, 2.0 ** -120)]
    for i, v in enumerate(edge):
        if n > 8:
            flat[(i * 5 + 1) % n] = v
    if n > 40:
        flat[37, 3], flat[39, 31] = np.nan, -np.inf
    return torch.from_numpy(w).to(TYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["out_in", "in_out"])
@pytest.mark.parametrize("shape", [(1, 8, 32), (3, 40, 96), (2, 264, 160), (5, 72, 2880)])
def test_pack_and_unpack(shape, layout, dtype):
    say(f"[pack] {shape} {layout} {dtype}")
    w = stack_with_edges(shape, dtype, 1)
    want = packed_by_definition(w.double().numpy())
    stored = w if layout == "out_in" else w.transpose(1, 2).contiguous()
    dev = stored.cuda()
    codes = torch.empty((*shape[:2], shape[2] // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((*shape[:2], shape[2] // 32), dtype=torch.uint8, device="cuda")
    etd.moe_pack_weights(dev, codes, scales, weight_layout=layout)
    back = torch.full_like(dev, 7.0)
    etd.moe_unpack_weights(codes, scales, back, weight_layout=layout)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(values_of(codes.cpu().numpy(), scales.cpu().numpy()), want)
    got = back.cpu() if layout == "out_in" else back.cpu().transpose(1, 2)
    np.testing.assert_array_equal(got.double().numpy(), want)   # exact: two significant bits


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_code_and_scale(dtype):
    # all 256 code bytes under scale bytes whose values are normal in the type
    codes = torch.arange(256, dtype=torch.uint8).reshape(1, 16, 16).repeat(1, 16, 1)
    scales = torch.arange(256, dtype=torch.uint8).reshape(1, 256, 1).clamp(min=2, max=252)
    scales[0, -1] = 255
    w = torch.empty((1, 256, 32), dtype=TYPES[dtype], device="cuda")
    etd.moe_unpack_weights(codes.cuda(), scales.cuda(), w)
    np.testing.assert_array_equal(w.cpu().double().numpy(), values_of(codes.numpy(), scales.numpy()))


def packed_stack(rng, L, N, K):
    """A random packed stack of weights around N(0, 1/K): (device tensors, float64 values)."""
    codes = rng.integers(0, 256, (L, N, K // 2), dtype=np.uint8)
    scales = (127 - 3 - int(round(np.log2(K) / 2)) + rng.integers(0, 3, (L, N, K // 32))).astype(np.uint8)
    return torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), values_of(codes, scales)


def ffn_reference(x, w, dtype):
    """y and a bound on the error of float32 sums, h rounded once and y rounded once, float64."""
    wg, wu, wd = w
    u32 = 2.0 ** -24
    a, b = x @ wg.T, x @ wu.T
    sa, sb = np.abs(x) @ np.abs(wg).T, np.abs(x) @ np.abs(wu).T
    sg = 1.0 / (1.0 + np.exp(-a))
    h = a * sg * b
    K, I = x.shape[1], h.shape[1]
    # sums of K products in float32; |silu'| <= 1.1; exp, reciprocal and products: 8 ulp
    dh = K * u32 * (1.1 * sa * np.abs(b) + np.abs(a * sg) * sb) + (HALF_STEP[dtype] + 8 * u32) * np.abs(h)
    y = h @ wd.T
    return y, (dh + I * u32 * np.abs(h)) @ np.abs(wd).T + HALF_STEP[dtype] * np.abs(y) + 1e-30


FFN = [
    # (H, I, rows of each expert, dtype)
    (32, 32, (1,), "bf16"),
    (64, 96, (0, 3, 0, 1), "bf16"),
    (160, 352, (5, 0, 17), "bf16"),
    (512, 288, (16, 1, 33, 0, 2, 64), "bf16"),
    (2048, 768, (1, 0, 2, 1), "bf16"),
    (2880, 480, (0, 7, 20), "bf16"),
    (96, 2880, (2, 31), "bf16"),
    (256, 320, (70, 130, 9), "bf16"),
    (256, 320, (300, 0, 200), "bf16"),
    (256, 320, (700, 90), "bf16"),
    (4096, 64, (1, 1), "bf16"),
    (96, 160, (70, 40), "bf16"),
    (352, 96, (150,), "bf16"),
    (96, 1184, (130, 0, 300), "bf16"),
    (64, 32, tuple(33 + i % 5 for i in range(70)), "bf16"),
    (2880, 352, (128, 0, 257), "bf16"),
    (64, 2080, (8000, 0, 101), "bf16"),
    (4096, 64, (127, 8000), "bf16"),
    (96, 64, (0, 9, 40), "f32"),
    (512, 256, (1, 64, 0), "f32"),
]


@pytest.mark.parametrize("H,I,rows,dtype", FFN)
@pytest.mark.parametrize("spare", [0, 40])
def test_grouped_ffn_packed(H, I, rows, dtype, spare):
    """spare: rows of the buffers behind the last segment, which stay as they were."""
    say(f"[packed ffn] H={H} I={I} rows={rows} {dtype} spare={spare}")
    rng = np.random.default_rng(H + I + sum(rows))
    L, P = len(rows), sum(rows)
    pm = P + spare
    x = torch.from_numpy(rng.standard_normal((pm, H)).astype(np.float32)).to(TYPES[dtype])
    stacks = {n: packed_stack(rng, L, N, K) for n, N, K in (("gate", I, H), ("up", I, H), ("down", H, I))}
    packed = etd.make_packed_experts({f"{n}_{k}": s[i] for n, s in stacks.items() for i, k in ((0, "codes"), (1, "scales"))})
    off = np.r_[0, np.cumsum(rows)].astype(np.int32)
    d = etd.make_desc(pm, H, I, L, 1, dtype=dtype, weight_layout="in_out")  # the layout does not matter here
    ws = torch.full((etd.moe_packed_workspace_size(d, etd.MOE_STAGE_FFN),), 255, dtype=torch.uint8, device="cuda")
    y = torch.full((pm, H), 3.0, dtype=TYPES[dtype], device="cuda")
    etd.moe_grouped_ffn_packed(d, x.cuda(), torch.from_numpy(off).cuda(), packed, y, ws=ws)
    again = torch.full_like(y, 3.0)
    etd.moe_grouped_ffn_packed(d, x.cuda(), torch.from_numpy(off).cuda(), packed, again, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(y, again)
    got, xs = np_of(y).astype(np.float64), x.double().numpy()
    assert np.all(got[P:] == 3.0)
    for e in range(L):
        r = slice(off[e], off[e + 1])
        if rows[e]:
            ref, bound = ffn_reference(xs[r], [stacks[n][2][e] for n in ("gate", "up", "down")], dtype)
            over = np.abs(got[r] - ref) / bound
            assert over.max() <= 1.0, f"expert {e}: {over.max()} of the bound"


def unpacked_input(inp, layer, packed):
    """inp with the expert weights that `packed` stands for, as the oracle takes them."""
    s = inp["spec"]
    out = dict(inp)
    for n in ("gate", "up", "down"):
        t = packed._tensors
        v = values_of(t[n + "_codes"].cpu().numpy(), t[n + "_scales"].cpu().numpy()).astype(np.float32)
        if s.weight_layout == "in_out":
            v = np.ascontiguousarray(v.transpose(0, 2, 1))
        out["w_" + n] = synth.f32_to_bf16_bits(v) if s.dtype == "bf16" else v
    return out


LAYERS = {
    "decode": synth.spec("decode_small", T=16, H=512, I=288, E=32, k=4, L=32),
    "one-token": synth.spec("decode_small", T=1, H=256, I=160, E=16, k=2, L=16),
    "share": synth.spec("gptoss_ep8_share", T=96, H=320, I=320, E=32, k=4, local_begin=8, L=8),
    "math-form": synth.spec("mixtral_like", T=700, H=256, I=384, E=4, k=2, L=4, weight_layout="in_out"),
    "capacity": synth.spec("skewed_capacity", T=512, H=128, I=192, E=16, k=3, L=16),
    "f32": synth.spec("tiny_fp32", T=200),
}


@pytest.mark.parametrize("name", list(LAYERS))
def test_layer_forward_packed(name):
    s = LAYERS[name]
    say(f"[packed layer] {name}: {s}")
    inp = synth.make_layer(s)
    layer, x = layer_of(inp)
    packed = layer.pack_experts()
    logits = np_of(layer.route(x, want_logits=True)["logits"])
    counts = torch.empty((s.E,), dtype=torch.int32, device="cuda")
    y = layer.forward_packed(x, packed, counts_out=counts)
    g = layer.staged(x)
    ys = layer.grouped_ffn_packed(g["x_sorted"], g["offsets"], packed)
    staged = layer.combine(ys, g["pair_row"], g["topk_w"])
    torch.cuda.synchronize()
    assert torch.equal(y, staged)
    assert torch.equal(counts, g["counts"])
    ref = oracle.layer_forward(unpacked_input(inp, layer, packed), logits=logits)
    err = row_error(np_of(y).astype(np.float64), ref["y"], s.dtype)
    say(f"[packed layer]   row error {err:.2e}")
    assert err <= tol(s.dtype)


@pytest.mark.parametrize("name", ["decode", "math-form"])
def test_packed_layer_in_a_graph_and_on_another_stream(name):
    s = LAYERS[name]
    inp = synth.make_layer(s)
    layer, x = layer_of(inp)
    packed = layer.pack_experts()
    ref = layer.forward_packed(x, packed)
    other, _ = layer_of(inp)                       # a second layer: a workspace of its own
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y_side = torch.empty_like(ref)
    with torch.cuda.stream(side):
        for _ in range(3):
            other.forward_packed(x, packed, y=y_side)
    for _ in range(3):
        y = layer.forward_packed(x, packed)
    torch.cuda.synchronize()
    assert torch.equal(y, ref) and torch.equal(y_side, ref)
    y_g = torch.empty_like(ref)
    with torch.cuda.stream(side):
        layer.forward_packed(x, packed, y=y_g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward_packed(x, packed, y=y_g)
    for r in range(3):
        y_g.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y_g, ref), f"replay {r}"
        assert torch.equal(layer.forward_packed(x, packed), ref)
        torch.cuda.synchronize()


def ffn_packed(x, rows, stacks, dtype="bf16", y=None):
    """y of the packed feed-forward on segments of `rows`; stacks: {name: (codes, scales)}."""
    H, I = x.shape[1], stacks["gate"][0].shape[1]
    packed = etd.make_packed_experts({f"{n}_{k}": s[i] for n, s in stacks.items() for i, k in ((0, "codes"), (1, "scales"))})
    d = etd.make_desc(x.shape[0], H, I, len(rows), 1, dtype=dtype)
    ws = torch.full((etd.moe_packed_workspace_size(d, etd.MOE_STAGE_FFN),), 255, dtype=torch.uint8, device="cuda")
    off = torch.from_numpy(np.r_[0, np.cumsum(rows)].astype(np.int32)).cuda()
    y = torch.full_like(x, 3.0) if y is None else y
    etd.moe_grouped_ffn_packed(d, x, off, packed, y, ws=ws)
    torch.cuda.synchronize()
    return y


# few rows, few rows with K split over waves, tiles of 128 weight rows, of 256, float32
NAN_GROUPS = [(96, 160, (3, 0, 2), "bf16"), (1088, 1056, (1, 2), "bf16"), (320, 288, (70, 9, 140), "bf16"),
              (288, 4128, (260, 900, 130), "bf16"), (96, 64, (9, 0, 40), "f32")]


@pytest.mark.parametrize("H,I,rows,dtype", NAN_GROUPS)
def test_a_nan_group_reaches_only_the_outputs_that_it_weighs(H, I, rows, dtype):
    say(f"[packed ffn] NaN groups H={H} I={I} rows={rows} {dtype}")
    rng = np.random.default_rng(7)
    L, P = len(rows), sum(rows)
    x = torch.from_numpy(rng.standard_normal((P, H)).astype(np.float32)).to(TYPES[dtype]).cuda()
    clean = {n: packed_stack(rng, L, N, K)[:2] for n, N, K in (("gate", I, H), ("up", I, H), ("down", H, I))}
    ref = ffn_packed(x, rows, clean, dtype)
    assert torch.isfinite(ref).all()
    last = slice(P - rows[-1], P)
    for o in (0, 17, H - 1):                      # a down row: one column of its expert's rows
        s = clean["down"][1].clone()
        s[L - 1, o, (o * 5) % (I // 32)] = 255
        y = ffn_packed(x, rows, {**clean, "down": (clean["down"][0], s)}, dtype)
        assert torch.isnan(y[last, o]).all()
        y[last, o] = ref[last, o]
        assert torch.equal(y, ref)
    for name, i in (("gate", 0), ("up", I - 1)):  # an entry of h: every output of its expert's rows
        s = clean[name][1].clone()
        s[0, i, (H // 32) - 1] = 255
        y = ffn_packed(x, rows, {**clean, name: (clean[name][0], s)}, dtype)
        assert torch.isnan(y[:rows[0]]).all() and torch.equal(y[rows[0]:], ref[rows[0]:])


@pytest.mark.parametrize("H,I,L,P,dtype", [(64, 96, 5, 20, "bf16"), (64, 96, 2, 500, "bf16"), (96, 2048, 4, 9000, "bf16"),
                                           (64, 96, 3, 40, "f32")])
def test_segments_without_rows_write_nothing(H, I, L, P, dtype):
    rng = np.random.default_rng(8)
    stacks = {n: packed_stack(rng, L, N, K)[:2] for n, N, K in (("gate", I, H), ("up", I, H), ("down", H, I))}
    y = ffn_packed(torch.randn((P, H), device="cuda").to(TYPES[dtype]), [0] * L, stacks, dtype)
    assert torch.all(y == 3.0)


@pytest.mark.parametrize("hot", [0, 19, 39])
def test_one_expert_with_all_the_rows_of_a_decode_step(hot):
    rng = np.random.default_rng(9)
    H, I, L, n = 256, 160, 40, 333                # 333 rows on 40 experts: the kernel for few rows
    rows = [n if e == hot else 0 for e in range(L)]
    full = {k: packed_stack(rng, L, N, K) for k, N, K in (("gate", I, H), ("up", I, H), ("down", H, I))}
    x = torch.from_numpy(rng.standard_normal((n, H)).astype(np.float32)).bfloat16()
    y = ffn_packed(x.cuda(), rows, {k: v[:2] for k, v in full.items()})
    ref, bound = ffn_reference(x.double().numpy(), [full[k][2][hot] for k in ("gate", "up", "down")], "bf16")
    assert (np.abs(np_of(y).astype(np.float64) - ref) <= bound).all()


def test_zero_capacity_gives_a_zero_packed_layer():
    s = synth.spec("skewed_capacity", T=1000, H=64, I=64, E=8, k=2, L=8, capacity_factor=0.001)
    layer, x = layer_of(synth.make_layer(s))
    dropped = torch.empty((1,), dtype=torch.int64, device="cuda")
    y = layer.forward_packed(x, layer.pack_experts(), y=torch.full_like(x, 3.0), num_dropped_out=dropped)
    torch.cuda.synchronize()
    assert int(dropped) == s.T * s.k and torch.all(y == 0)


def test_stacks_past_4_gib_are_reached():
    """The last expert of a stack whose codes lie past 32-bit offsets, in both kernels."""
    H, I, L = 4096, 8192, 300                     # 5.03 GB of codes a stack; one tensor serves all three
    codes = torch.zeros((L, I, H // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((L, I, H // 32), 127, dtype=torch.uint8, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    codes[-1] = torch.randint(0, 256, codes[-1].shape, dtype=torch.uint8, device="cuda", generator=gen)
    scales[-1] = 120 + torch.randint(0, 3, scales[-1].shape, dtype=torch.uint8, device="cuda", generator=gen)
    stacks = {"gate": (codes, scales), "up": (codes, scales),
              "down": (codes.view(L, H, I // 2), scales.view(L, H, I // 32))}
    for n, spare in ((3, 0), (200, 64 * L)):      # spare rows: more than 32 an expert
        x = torch.randn((n + spare, H), device="cuda", generator=gen).bfloat16()
        y = ffn_packed(x, [0] * (L - 1) + [n], stacks)
        alone = ffn_packed(x, [n], {k: (c[-1:].clone(), s[-1:].clone()) for k, (c, s) in stacks.items()})
        assert torch.all(y[n:] == 3.0) and float(y[:n].float().abs().max()) > 0
        # tiles and waves along K may differ between the two calls: the sums' order, not the values
        a, b = y[:n].double(), alone[:n].double()
        assert float((a - b).norm() / b.norm()) <= 2.0 ** -7


# one step of K or several, K cut inside a step, waves along K 1, 2 and 4, 16 or 32 rows a pass
F32_ROWS = [(32, 32, (1,)), (32, 96, (0, 5, 16)), (288, 160, (17, 0, 3, 40)), (512, 1056, (1, 1)), (2080, 544, (2, 0, 9)),
            (1024, 2048, (1,)), (160, 1312, (31, 33, 32)), (96, 64, (1, 0, 0, 0, 90, 2)), (544, 96, (7,) * 70)]


@pytest.mark.parametrize("H,I,rows", F32_ROWS)
def test_float32_rows_on_packed_experts(H, I, rows):
    say(f"[packed ffn] float32 H={H} I={I} rows={rows}")
    rng = np.random.default_rng(H + I)
    L, P, spare = len(rows), sum(rows), 3
    full = {k: packed_stack(rng, L, N, K) for k, N, K in (("gate", I, H), ("up", I, H), ("down", H, I))}
    x = torch.from_numpy(rng.standard_normal((P + spare, H)).astype(np.float32))
    y = ffn_packed(x.cuda(), rows, {k: v[:2] for k, v in full.items()}, "f32")
    assert torch.all(y[P:] == 3.0)
    got, off = np_of(y).astype(np.float64), np.r_[0, np.cumsum(rows)]
    for e in range(L):
        r = slice(off[e], off[e + 1])
        if rows[e]:
            ref, bound = ffn_reference(x[r].double().numpy(), [full[k][2][e] for k in ("gate", "up", "down")], "f32")
            over = np.abs(got[r] - ref) / bound
            assert over.max() <= 1.0, f"expert {e}: {over.max()} of the bound"


# products of so many tiles that codes go two steps a load, one stage of K or several
MANY_TILES = [(256, 2176, (8200, 0, 100)), (4224, 128, (31, 8300)), (4224, 384, (4000, 4301))]


@pytest.mark.parametrize("H,I,rows", MANY_TILES)
def test_products_of_many_tiles(H, I, rows):
    say(f"[packed ffn] many tiles H={H} I={I} rows={rows}")
    rng = np.random.default_rng(H + I)
    L, P = len(rows), sum(rows)
    full = {k: packed_stack(rng, L, N, K) for k, N, K in (("gate", I, H), ("up", I, H), ("down", H, I))}
    x = torch.from_numpy(rng.standard_normal((P, H), dtype=np.float32)).bfloat16()
    y = ffn_packed(x.cuda(), rows, {k: v[:2] for k, v in full.items()})
    got, off = np_of(y), np.r_[0, np.cumsum(rows)]
    for e in range(L):
        if rows[e]:
            some = np.unique(np.r_[off[e]:min(off[e] + 130, off[e + 1]), max(off[e], off[e + 1] - 130):off[e + 1],
                                   rng.integers(off[e], off[e + 1], 100)])
            ref, bound = ffn_reference(x[some].double().numpy(), [full[k][2][e] for k in ("gate", "up", "down")], "bf16")
            over = np.abs(got[some].astype(np.float64) - ref) / bound
            assert over.max() <= 1.0, f"expert {e}: {over.max()} of the bound"
