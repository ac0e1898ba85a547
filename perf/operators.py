"""What the operators on stacked expert weights cost, case by case.

Four kinds of pass over one stack of expert matrices or one layer's experts:

  ffn    the local experts' SwiGLU on rows sorted by expert, weights in 4 bits
         with a power-of-two scale per 32 inputs (moe_grouped_ffn_packed)
  pack   a weight stack into 4 bits and back to its type (moe_pack_weights, then
         moe_unpack_weights): the values the codes stand for
  orth   every matrix of a stack orthogonalised by Newton-Schulz steps (moe_orthogonalize)
  muon   momentum, orthogonalised update and decayed weight of a stack, in place
         (moe_muon_update)

With `own` false a pass is computed by elementary torch operations in 32 bits.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
COEF = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
MU = 0.95
GROUP = 32


def listed():
    return [
        # one token of the decode-sized layer: 8 of its 128 experts get one row each
        dict(name="ffn_decode_one", kind="ffn", H=2048, I=768, L=128, P=8, spread="one", dtype="bf16"),
        # its whole batch of 64 tokens, 8 experts each
        dict(name="ffn_decode_batch", kind="ffn", H=2048, I=768, L=128, P=512, spread="even", dtype="bf16"),
        # a rank that holds 16 of 128 experts, decoding a few tokens; some experts get nothing
        dict(name="ffn_share_decode", kind="ffn", H=2880, I=2880, L=16, P=40, spread="skew", dtype="bf16"),
        # the same rank on a chunk of a prompt, between decode and prefill
        dict(name="ffn_share_chunk", kind="ffn", H=2880, I=2880, L=16, P=2047, spread="skew", dtype="bf16"),
        # prefill of 8192 tokens, two experts each, through the widest experts
        dict(name="ffn_prefill", kind="ffn", H=4096, I=14336, L=8, P=16384, spread="even", dtype="bf16"),
        # a float32 layer's experts on a small batch
        dict(name="ffn_f32", kind="ffn", H=512, I=256, L=8, P=64, spread="even", dtype="f32"),
        # a rank's stack before serving, stored as the math form has it
        dict(name="pack_share", kind="pack", L=16, N=2880, K=2880, layout="in_out", dtype="bf16"),
        # a small float32 stack, stored as linear layers store it
        dict(name="pack_f32", kind="pack", L=8, N=256, K=512, layout="out_in", dtype="f32"),
        # the small float32 layer's gradient: where launches count
        dict(name="orth_f32", kind="orth", L=8, R=256, C=512, dtype="f32"),
        # 128 experts' gate gradients of the decode-sized layer
        dict(name="orth_many", kind="orth", L=128, R=768, C=2048, dtype="bf16"),
        # a training step of a rank's stack, square matrices, float32 masters
        dict(name="muon_share", kind="muon", L=16, R=2880, C=2880, dtype="bf16"),
        # the widest experts' gate stack in the math form's orientation transposed: tall matrices
        dict(name="muon_wide", kind="muon", L=8, R=14336, C=4096, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("ffn", "ffn", "pack", "orth", "muon"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if kind == "ffn":
        H, I = 32 * _log(rng, 2, 128), 32 * _log(rng, 2, 128)
        L = _log(rng, 1, 64)
        while 3 * L * H * I > 6e8:
            L = max(1, L // 2)
        P = _log(rng, 1, 8192 if dtype == "bf16" else 512)
        return dict(kind=kind, H=H, I=I, L=L, P=P, spread=rng.choice(("even", "skew")), dtype=dtype)
    if kind == "pack":
        N, K, L = 8 * _log(rng, 4, 512), 32 * _log(rng, 1, 128), _log(rng, 1, 32)
        return dict(kind=kind, L=L, N=N, K=K, layout=rng.choice(("out_in", "in_out")), dtype=dtype)
    R, C, L = _log(rng, 64, 3000), _log(rng, 64, 3000), _log(rng, 1, 64)
    cap = 1.5e12 if dtype == "bf16" else 2e11
    while L > 1 and 10 * L * min(R, C) ** 2 * max(R, C) > cap:
        L //= 2
    return dict(kind=kind, L=L, R=R, C=C, dtype=dtype)


# ---- the 4-bit format: e2m1 codes, low half of a byte first, and one e8m0 scale per 32 inputs ----
def _codes_of(q):
    """Codes 0..15 of values already divided by their scale: nearest e2m1, ties to the even code, at most 6."""
    a = q.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
            + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8)
            + (a > 5.0).to(torch.uint8))
    return code + 8 * torch.signbit(q).to(torch.uint8)


def _quantize(w):
    """w [..., K] float32 -> codes [..., K] 0..15, scale bytes [..., K / 32]."""
    g = w.reshape(*w.shape[:-1], w.shape[-1] // GROUP, GROUP)
    _, e = torch.frexp(g.abs().amax(-1))
    e = (e - 3).clamp(-127, 127)
    code = _codes_of(torch.ldexp(g, -e[..., None]))
    return code.reshape(w.shape), (e + 127).to(torch.uint8)


_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pair_table(dtype, device):
    """[256, 2]: the two values of a byte of codes, low half first."""
    v = torch.tensor(_MAGNITUDES + tuple(-x for x in _MAGNITUDES), dtype=dtype, device=device)
    b = torch.arange(256, device=device)
    return torch.stack([v[b & 15], v[b >> 4]], dim=-1)


def _unpack(codes, scales, dtype=torch.float32):
    """codes [..., K / 2] bytes, scales [..., K / 32] bytes -> values [..., K]."""
    v = _pair_table(dtype, codes.device)[codes.to(torch.int32)]
    v = v.reshape(*scales.shape, GROUP)
    s = torch.exp2(scales.to(dtype) - 127.0)
    return (v * s[..., None]).reshape(*codes.shape[:-1], codes.shape[-1] * 2)


# ---- what a program has in hand -----------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _packed_stack(L, N, K, g):
    """A trained-looking stack N(0, 1/K) in 4 bits, expert by expert."""
    codes = torch.empty((L, N, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((L, N, K // GROUP), dtype=torch.uint8, device=DEV)
    for e in range(L):
        c, s = _quantize(torch.randn((N, K), generator=g, device=DEV) * K ** -0.5)
        codes[e] = c[:, 0::2] | (c[:, 1::2] << 4)
        scales[e] = s
    return codes, scales


def _popularity(case):
    """Share of the rows that each expert draws: all alike, or falling off as 1 / rank."""
    return [1.0 if case["spread"] != "skew" else 1.0 / (1 + e) for e in range(case["L"])]


def _counts(case, rng):
    """Rows of each local expert, sum P."""
    L, P = case["L"], case["P"]
    order = torch.randperm(L, generator=rng)
    if case["spread"] == "one":  # every row to an expert of its own
        return torch.zeros(L, dtype=torch.int64).index_fill_(0, order[:P], 1)
    w = torch.tensor(_popularity(case))[order]
    return torch.bincount(torch.multinomial(w, P, replacement=True, generator=rng), minlength=L)


def _gradient(shape, g):
    """A weight gradient as a batch leaves it: a few dozen strong directions over a broad floor."""
    L, R, C = shape
    r = max(1, min(R, C) // 16)
    s = torch.randn((L, R, r), generator=g, device=DEV) @ torch.randn((L, r, C), generator=g, device=DEV) * r ** -0.5
    return (s + 0.25 * torch.randn(shape, generator=g, device=DEV)) * 1e-3


def prepare(case, seed):
    g = _gen(seed)
    dt = TYPES[case["dtype"]]
    st = dict(case)
    if case["kind"] == "ffn":
        H, I, L, P = case["H"], case["I"], case["L"], case["P"]
        n = _counts(case, torch.Generator().manual_seed(int(seed) + 5))
        st["counts"] = n.tolist()
        st["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).to(torch.int32).to(DEV)
        st["x"] = torch.randn((P, H), generator=g, device=DEV).to(dt)
        st["y"] = torch.zeros((P, H), dtype=dt, device=DEV)
        for name, N, K in (("gate", I, H), ("up", I, H), ("down", H, I)):
            st[name + "_codes"], st[name + "_scales"] = _packed_stack(L, N, K, g)
    elif case["kind"] == "pack":
        L, N, K = case["L"], case["N"], case["K"]
        shape = (L, N, K) if case["layout"] == "out_in" else (L, K, N)
        st["w"] = (torch.randn(shape, generator=g, device=DEV) * K ** -0.5).to(dt)
        st["codes"] = torch.empty((L, N, K // 2), dtype=torch.uint8, device=DEV)
        st["scales"] = torch.empty((L, N, K // GROUP), dtype=torch.uint8, device=DEV)
        st["back"] = torch.empty_like(st["w"])
    else:
        shape = (case["L"], case["R"], case["C"])
        st["g"] = _gradient(shape, g).to(dt)
        if case["kind"] == "orth":
            st["o"] = torch.empty_like(st["g"])
        else:
            st["lr"], st["decay"] = 2e-4, 0.1
            st["scale"] = 0.2 * math.sqrt(max(case["R"], case["C"]))
            st["momentum"] = _gradient(shape, g) * 5.0
            st["master"] = torch.randn(shape, generator=g, device=DEV) * case["C"] ** -0.5
            st["w"] = st["master"].to(dt)
    return st


# ---- the plain forms ------------------------------------------------------------------------------
def _ffn_plain(st):
    H, L, P = st["H"], st["L"], st["P"]
    on = [e for e in range(L) if st["counts"][e]]
    active = torch.tensor(on, device=DEV)
    most = max(st["counts"])
    first = st["offsets"][active].long()
    n = st["offsets"][active + 1].long() - first
    slot = torch.arange(most, device=DEV)
    row = first[:, None] + slot[None, :]                      # [experts with rows, most]
    there = slot[None, :] < n[:, None]
    xe = st["x"].float()[row.clamp(max=P - 1)] * there[..., None]
    w = {k: _unpack(st[k + "_codes"][active], st[k + "_scales"][active]) for k in ("gate", "up")}
    a, b = xe @ w["gate"].transpose(1, 2), xe @ w["up"].transpose(1, 2)
    h = a / (1.0 + torch.exp(-a)) * b
    del w, a, b, xe
    y = h @ _unpack(st["down_codes"][active], st["down_scales"][active]).transpose(1, 2)
    st["y"][row[there]] = y[there].to(st["y"].dtype)
    return st["y"]


def _pack_plain(st):
    w = st["w"].float()
    rows = w if st["layout"] == "out_in" else w.transpose(1, 2).contiguous()
    code, scale = _quantize(rows)
    v = _unpack(code[..., 0::2] | (code[..., 1::2] << 4), scale)
    st["back"].copy_(v if st["layout"] == "out_in" else v.transpose(1, 2))
    return st["back"]


def _orth_plain(u, steps=5):
    a, b, c = COEF
    tall = u.shape[1] > u.shape[2]
    x = u.transpose(1, 2) if tall else u
    x = (x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)).contiguous()
    for _ in range(steps):
        g = x @ x.transpose(1, 2)
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.transpose(1, 2) if tall else x


def _muon_plain(st):
    g = st["g"].float()
    m = st["momentum"].mul_(MU).add_(g)
    o = _orth_plain(g + MU * m)
    st["master"].mul_(1.0 - st["lr"] * st["decay"]).sub_(o * (st["lr"] * st["scale"]))
    st["w"].copy_(st["master"])
    return {"momentum": m, "master": st["master"], "weight": st["w"]}


# ---- the framework's calls ------------------------------------------------------------------------
def _plan(st):
    """Descriptor and workspace, kept by the program that owns the buffers."""
    import expert_token_dispatch_amd as etd

    if "plan" not in st:
        if st["kind"] == "ffn":
            d = etd.make_desc(st["P"], st["H"], st["I"], st["L"], 1, dtype=st["dtype"])
            size = etd.moe_packed_workspace_size(d, etd.MOE_STAGE_FFN)
            packed = etd.make_packed_experts({k: st[k] for k in ("gate_codes", "gate_scales", "up_codes", "up_scales",
                                                                 "down_codes", "down_scales")})
        elif st["kind"] == "pack":
            d, size, packed = None, 0, None
        else:
            more = {} if st["kind"] == "orth" else dict(momentum=MU, nesterov=True, lr=st["lr"], update_scale=st["scale"],
                                                        weight_decay=st["decay"])
            d = etd.make_muon_desc(st["L"], st["R"], st["C"], dtype=st["dtype"], steps=5, coefs=COEF, eps=EPS, **more)
            size, packed = etd.moe_muon_workspace_size(d), None
        st["plan"] = (d, torch.empty(size, dtype=torch.uint8, device=DEV) if size else None, packed)
    return (etd, *st["plan"])


def _run_own(st):
    etd, d, ws, packed = _plan(st)
    if st["kind"] == "ffn":
        etd.moe_grouped_ffn_packed(d, st["x"], st["offsets"], packed, st["y"], ws=ws)
        return st["y"]
    if st["kind"] == "pack":
        etd.moe_pack_weights(st["w"], st["codes"], st["scales"], weight_layout=st["layout"])
        etd.moe_unpack_weights(st["codes"], st["scales"], st["back"], weight_layout=st["layout"])
        return st["back"]
    if st["kind"] == "orth":
        etd.moe_orthogonalize(d, st["g"], st["o"], ws)
        return st["o"]
    etd.moe_muon_update(d, st["g"], st["momentum"], st["w"], ws, master=st["master"])
    return {"momentum": st["momentum"], "master": st["master"], "weight": st["w"]}


def run(state):
    if own:
        return _run_own(state)
    if state["kind"] == "ffn":
        return _ffn_plain(state)
    if state["kind"] == "pack":
        return _pack_plain(state)
    if state["kind"] == "orth":
        state["o"].copy_(_orth_plain(state["g"].float()))
        return state["o"]
    return _muon_plain(state)


def work(case):
    dt = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "ffn":
        H, I, L, P = case["H"], case["I"], case["L"], case["P"]
        w = _popularity(case)  # experts that have rows, on average
        experts = P if case["spread"] == "one" else sum(1.0 - (1.0 - v / sum(w)) ** P for v in w)
        return {"bytes": 3 * experts * H * I * (0.5 + 1 / GROUP) + 2 * P * H * dt, "flops": 6 * P * H * I}
    if case["kind"] == "pack":
        n = case["L"] * case["N"] * case["K"]
        return {"bytes": 2 * n * dt + 2 * n * (0.5 + 1 / GROUP), "flops": 0}
    L, m, n = case["L"], min(case["R"], case["C"]), max(case["R"], case["C"])
    # symmetric products once; the cheaper of five full steps and three + two steps on the m x m side
    flops = L * min(15 * m * m * n + 5 * m ** 3, 6 * m * m * n + 14 * m ** 3)
    per = 2 * dt if case["kind"] == "orth" else 2 * dt + 16
    return {"bytes": L * m * n * per, "flops": flops}


# ---- the definitions in 64 bits ---------------------------------------------------------------------
def _value64(codes, scales):
    lo, hi = codes & 15, codes >> 4
    c = torch.stack([lo, hi], dim=-1).reshape(*codes.shape[:-1], -1).to(torch.int64)
    e, frac = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(e == 0, frac * 0.5, (1.0 + 0.5 * frac) * torch.pow(2.0, (e - 1).double()))
    s = torch.pow(2.0, scales.double() - 127.0).repeat_interleave(GROUP, dim=-1)
    return torch.where(c >= 8, -mag, mag) * s


def _ffn_exact(st):
    y = torch.zeros((st["P"], st["H"]), dtype=torch.float64, device=DEV)
    at = 0
    for e, n in enumerate(st["counts"]):
        if n:
            x = st["x"][at:at + n].double()
            a = x @ _value64(st["gate_codes"][e], st["gate_scales"][e]).T
            h = a * torch.sigmoid(a) * (x @ _value64(st["up_codes"][e], st["up_scales"][e]).T)
            y[at:at + n] = h @ _value64(st["down_codes"][e], st["down_scales"][e]).T
        at += n
    return y


def _pack_exact(st):
    dim = 2 if st["layout"] == "out_in" else 1
    w = st["w"].double()
    out = torch.empty_like(w)
    grid = torch.tensor(_MAGNITUDES, dtype=torch.float64, device=DEV)
    even = torch.tensor([0.0, 1.0] * 4, dtype=torch.float64, device=DEV)
    for e in range(st["L"]):  # one matrix at a time: nearest of the eight magnitudes, an even code at a tie
        v = w[e].movedim(dim - 1, -1)
        g = v.reshape(v.shape[0], -1, GROUP)
        top = g.abs().amax(-1, keepdim=True)
        s = torch.pow(2.0, torch.floor(torch.log2(top.clamp(min=1e-300))) - 2.0)
        q = (g / s).abs()
        best, far = torch.zeros_like(q), torch.full_like(q, float("inf"))
        for k in range(8):
            d = (q - grid[k]).abs() + even[k] * 1e-12
            best, far = torch.where(d < far, grid[k], best), torch.minimum(d, far)
        out[e] = (torch.copysign(best, g) * s).reshape(v.shape).movedim(-1, dim - 1)
    return out


def _orth_exact(u):
    a, b, c = COEF
    out = torch.empty_like(u)
    for i in range(u.shape[0]):
        x = u[i] / (torch.linalg.vector_norm(u[i]) + EPS)
        for _ in range(5):
            if x.shape[0] <= x.shape[1]:
                g = x @ x.T
                y = g @ x
                x = a * x + b * y + c * (g @ y)
            else:
                g = x.T @ x
                y = x @ g
                x = a * x + b * y + c * (y @ g)
        out[i] = x
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "ffn":
        return _ffn_exact(st)
    if case["kind"] == "pack":
        return _pack_exact(st)
    if case["kind"] == "orth":
        return _orth_exact(st["g"].double())
    m = MU * st["momentum"].double() + st["g"].double()
    w = st["master"].double() * (1.0 - st["lr"] * st["decay"])
    w -= st["lr"] * st["scale"] * _orth_exact(st["g"].double() + MU * m)
    return {"momentum": m, "master": w, "weight": w}
