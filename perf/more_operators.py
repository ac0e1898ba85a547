"""What the operators around one mixture-of-experts layer cost, case by case.

Three kinds of pass:

  join    a block's output normed, gated, scaled and added to the residual stream, and
          the norm before the next block, in one call (moe_block_join)
  back    its gradients: of the stream, the block's output, the gate and both norm
          weights (moe_block_join_backward)
  adapt   the local experts' SwiGLU on rows sorted by expert, with the low-rank adapters
          of many requests beside the three projections (moe_grouped_ffn_adapted)

With `own` false a pass is computed by elementary torch operations in 32 bits.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one token between two blocks: norm after, norm before, nothing else; launch latency
        dict(name="join_one", kind="join", form="full", T=1, H=2880, gate="none", act="linear", offset=0.0, scale=1.0,
             dtype="bf16"),
        # a decode batch, each token's block gated by a logit of its own
        dict(name="join_batch", kind="join", form="full", T=64, H=2048, gate="token", act="sigmoid", offset=0.0, scale=1.0,
             dtype="bf16"),
        # a ragged chunk of a prompt with a gate per element and zero-centred norm weights
        dict(name="join_chunk", kind="join", form="full", T=2047, H=2880, gate="element", act="sigmoid", offset=1.0,
             scale=0.5, dtype="bf16"),
        # prefill of 8192 tokens, a learned scale per channel
        dict(name="join_prefill", kind="join", form="full", T=8192, H=4096, gate="channel", act="linear", offset=0.0,
             scale=0.22, dtype="bf16"),
        # a training step over the same tokens
        dict(name="back_train", kind="back", form="full", T=8192, H=4096, gate="channel", act="linear", offset=0.0,
             scale=0.22, dtype="bf16"),
        # a rank's odd share of a batch, a gate per element
        dict(name="back_share", kind="back", form="full", T=1021, H=2880, gate="element", act="sigmoid", offset=1.0,
             scale=0.5, dtype="bf16"),
        # the small float32 layer's batch, a gate per token, no norm after the block
        dict(name="back_f32", kind="back", form="add", T=4096, H=512, gate="token", act="sigmoid", offset=0.0, scale=1.0,
             dtype="f32"),
        # one token of the decode-sized layer: 8 of its 128 experts get one row each, one adapter
        dict(name="adapt_one", kind="adapt", H=2048, I=768, L=128, P=8, R=16, n=1, plain=0.0, runs=False, spread="one",
             dtype="bf16"),
        # its whole batch: 64 tokens of many customers, 8 experts each, a quarter without an adapter
        dict(name="adapt_batch", kind="adapt", H=2048, I=768, L=128, P=512, R=16, n=24, plain=0.25, runs=False,
             spread="even", dtype="bf16"),
        # a rank that holds 16 of 128 experts, on chunks of a few requests' prompts; experts of very different load
        dict(name="adapt_chunk", kind="adapt", H=2880, I=2880, L=16, P=2047, R=24, n=6, plain=0.2, runs=True,
             spread="skew", dtype="bf16"),
        # prefill of 8192 tokens of eight requests, two experts each, through the widest experts
        dict(name="adapt_prefill", kind="adapt", H=4096, I=14336, L=8, P=16384, R=64, n=8, plain=0.0, runs=True,
             spread="even", dtype="bf16"),
        # a float32 layer's experts on a small batch
        dict(name="adapt_f32", kind="adapt", H=512, I=256, L=8, P=200, R=8, n=5, plain=0.2, runs=False, spread="even",
             dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("join", "join", "back", "back", "adapt", "adapt", "adapt"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if kind != "adapt":
        H, T = 8 * _log(rng, 2, 1024), _log(rng, 1, 16384)
        while H * T * (2 if dtype == "f32" else 1) > 32e6:
            T = max(1, T // 2)
        gate = rng.choice(("none", "channel", "token", "element"))
        form = rng.choice(("full", "full", "full", "add", "post", "enter"))
        return dict(kind=kind, form=form, T=T, H=H, gate="none" if form == "enter" else gate,
                    act=rng.choice(("linear", "sigmoid")), offset=rng.choice((0.0, 1.0)), scale=rng.choice((1.0, 0.5, 0.22)),
                    dtype=dtype)
    step = rng.choice((8, 32, 64))
    H, I = step * _log(rng, 2, 4096 // step), step * _log(rng, 2, 4096 // step)
    L, R, n = _log(rng, 1, 64), rng.choice((8, 16, 16, 24, 32, 64)), _log(rng, 1, 48)
    while 3 * L * H * I > 6e8 or 3 * n * L * R * (H + I) > 6e8:
        L, n = max(1, L // 2), max(1, (n + 1) // 2)
        if L == 1 and n == 1:
            break
    P = _log(rng, 1, 8192 if dtype == "bf16" else 512)
    return dict(kind=kind, H=H, I=I, L=L, P=P, R=R, n=n, plain=rng.choice((0.0, 0.2, 0.5)), runs=rng.choice((True, False)),
                spread=rng.choice(("even", "skew")), dtype=dtype)


# ---- what a program has in hand -----------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _stream(T, H, g):
    """A residual stream: most channels alike, a few large, tokens of different size."""
    v = torch.randn((T, H), generator=g, device=DEV)
    big = torch.rand(H, generator=g, device=DEV) < 0.01
    return v * torch.where(big, 12.0, 1.0) * torch.exp(0.5 * torch.randn((T, 1), generator=g, device=DEV))


def _prepare_join(case, st, g, dt):
    T, H, form = case["T"], case["H"], case["form"]

    def rand(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    w = [((1.0 - case["offset"]) + 0.1 * rand(H)).to(dt) for _ in range(2)]
    st["y"] = None if form == "enter" else (2.0 * rand(T, H)).to(dt)
    st["w_post"] = w[0] if form in ("full", "post") else None
    st["w_pre"] = None if form == "post" else w[1]
    shape = {"none": None, "channel": (H,), "token": (T,), "element": (T, H)}[case["gate"]]
    st["gate"] = None if shape is None else rand(*shape).to(torch.float32 if case["gate"] == "token" else dt)
    st["x"] = _stream(T, H, g).to(dt)
    if case["kind"] == "back":
        st["z"] = st.pop("x")
        st["dz"] = (1e-3 * rand(T, H)).to(dt)
        st["dh"] = None if form == "post" else (1e-3 * rand(T, H)).to(dt)


def _popularity(case):
    """Share of the rows that each expert draws: all alike, or falling off as 1 / rank."""
    return [1.0 if case["spread"] != "skew" else 1.0 / (1 + e) for e in range(case["L"])]


def _prepare_adapt(case, st, g, seed, dt):
    H, I, L, P, R, n = (case[k] for k in "H I L P R n".split())
    rng = torch.Generator().manual_seed(int(seed) + 5)
    # the expert of every row, in token order; then the rows in stable order of their expert
    order = torch.randperm(L, generator=rng)
    if case["spread"] == "one":
        expert = order[:P].sort().values
    else:
        expert = torch.multinomial(torch.tensor(_popularity(case))[order], P, replacement=True, generator=rng)
    pairs = torch.argsort(expert, stable=True)
    counts = torch.bincount(expert, minlength=L)
    # the adapter of every token, -1 for none: requests of many tokens one after another, or one token each
    some = torch.randint(0, n, (P,), generator=rng)
    some[torch.rand(P, generator=rng) < case["plain"]] = -1
    if case["runs"]:
        cuts = torch.sort(torch.randint(0, P, (2 * n,), generator=rng)).values
        some = some[torch.searchsorted(cuts, torch.arange(P), right=True) % P]
    st["counts"], st["ids"] = counts.tolist(), some[pairs].tolist()  # of the sorted rows
    st["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).to(DEV)
    st["pairs"], st["adapter_ids"] = pairs.to(torch.int32).to(DEV), some.to(torch.int32).to(DEV)
    st["x"] = torch.randn((P, H), generator=g, device=DEV).to(dt)
    st["y"] = torch.zeros((P, H), dtype=dt, device=DEV)
    for name, N, K in (("gate", I, H), ("up", I, H), ("down", H, I)):
        st[name] = (torch.randn((L, N, K), generator=g, device=DEV) * K ** -0.5).to(dt)
        st[name + "_a"] = (torch.randn((n, L, R, K), generator=g, device=DEV) * K ** -0.5).to(dt)
        st[name + "_b"] = (torch.randn((n, L, N, R), generator=g, device=DEV) * (0.3 * R ** -0.5)).to(dt)
    st["scale"] = 0.5 + torch.rand(n, generator=g, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    dt = TYPES[case["dtype"]]
    st = {"case": dict(case)}
    if case["kind"] == "adapt":
        _prepare_adapt(case, st, g, seed, dt)
    else:
        _prepare_join(case, st, g, dt)
    return st


# ---- the plain forms ------------------------------------------------------------------------------
def _f(t):
    return None if t is None else t.float()


def _gate_of(case, gate):
    """The gate's value, laid out against [T, H]; 1 where there is none."""
    if gate is None:
        return 1.0
    v = 1.0 / (1.0 + torch.exp(-gate)) if case["act"] == "sigmoid" else gate
    return v[:, None] if case["gate"] == "token" else v


def _factor(case, w):
    return 1.0 if w is None else w + case["offset"]


def _rstd(v):
    return torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _join_plain(st):
    case, dt = st["case"], st["x"].dtype
    z, out = _f(st["x"]), {}
    if st["y"] is not None:
        b = _f(st["y"])
        if st["w_post"] is not None:
            b = b * _rstd(b) * _factor(case, _f(st["w_post"]))
        z = z + case["scale"] * _gate_of(case, _f(st["gate"])) * b
        out["z"] = z.to(dt)
    if st["w_pre"] is not None:
        out["h"] = (z * _rstd(z) * _factor(case, _f(st["w_pre"]))).to(dt)
    return out


def _back_plain(st):
    case, dt = st["case"], st["z"].dtype
    d, out = _f(st["dz"]), {}
    if st["dh"] is not None:
        z, dh = _f(st["z"]), _f(st["dh"])
        r = _rstd(z)
        zh = z * r
        a = dh * _factor(case, _f(st["w_pre"]))
        d = d + r * (a - zh * (a * zh).mean(-1, keepdim=True))
        out["dw_pre"] = (dh * zh).sum(0).to(dt)
    out["dx"] = d.to(dt)
    if st["y"] is None:
        return out
    y, gate = _f(st["y"]), _f(st["gate"])
    g = _gate_of(case, gate)
    post = st["w_post"] is not None
    r = _rstd(y) if post else 1.0
    yh = y * r
    f = _factor(case, _f(st["w_post"]))
    db = case["scale"] * g * d
    if post:
        c = db * f
        out["dw_post"] = (db * yh).sum(0).to(dt)
        out["dy"] = (r * (c - yh * (c * yh).mean(-1, keepdim=True))).to(dt)
    else:
        out["dy"] = db.to(dt)
    if gate is not None:
        dg = case["scale"] * d * (yh * f)
        if case["gate"] == "channel":
            dg = dg.sum(0)
        elif case["gate"] == "token":
            dg = dg.sum(1)
        if case["act"] == "sigmoid":
            s = 1.0 / (1.0 + torch.exp(-gate))
            dg = dg * (s * (1.0 - s))
        out["dgate"] = dg.to(st["gate"].dtype)
    return out


def _adapt_plain(st):
    case = st["case"]
    L, P, n = case["L"], case["P"], case["n"]
    on = [e for e in range(L) if st["counts"][e]]
    active = torch.tensor(on, device=DEV)
    most = max(st["counts"])
    first = st["offsets"][active].long()
    rows = st["offsets"][active + 1].long() - first
    slot = torch.arange(most, device=DEV)
    row = (first[:, None] + slot[None, :]).clamp(max=P - 1)   # [experts with rows, most]
    there = slot[None, :] < rows[:, None]
    ids = torch.where(there, st["adapter_ids"].long()[st["pairs"].long()][row], -1)

    def project(v, name):
        o = v @ st[name][active].float().transpose(1, 2).contiguous()
        for a in range(n):
            mine = (ids == a)[..., None]
            u = v @ st[name + "_a"][a][active].float().transpose(1, 2).contiguous()
            u = torch.where(mine, u * st["scale"][a], torch.zeros((), device=DEV))
            o += u @ st[name + "_b"][a][active].float().transpose(1, 2).contiguous()
        return o

    xe = st["x"].float()[row] * there[..., None]
    a = project(xe, "gate")
    h = a / (1.0 + torch.exp(-a)) * project(xe, "up")
    del a, xe
    y = project(h, "down")
    st["y"][row[there]] = y[there].to(st["y"].dtype)
    return st["y"]


# ---- the framework's calls ------------------------------------------------------------------------
def _plan(st):
    """Descriptor, buffers and workspace, kept by the program that owns the tensors."""
    import expert_token_dispatch_amd as etd

    if "plan" not in st:
        case = st["case"]
        if case["kind"] == "adapt":
            d = etd.make_desc(case["P"], case["H"], case["I"], case["L"], 1, dtype=case["dtype"])
            ad = etd.make_adapters({k: st[k] for k in ("gate_a", "gate_b", "up_a", "up_b", "down_a", "down_b", "scale")})
            size, bufs = etd.moe_adapted_workspace_size(d, ad, etd.MOE_STAGE_FFN), ad
        else:
            v = st["z"] if case["kind"] == "back" else st["x"]
            d = etd.make_join_desc(case["T"], case["H"], dtype=case["dtype"], post_norm=st["w_post"] is not None,
                                   gate=case["gate"], gate_act=case["act"], eps=EPS, weight_offset=case["offset"],
                                   residual_scale=case["scale"])
            size = etd.moe_join_workspace_size(d) if case["kind"] == "back" else 0

            def like(t):
                return None if t is None else torch.empty_like(t)

            if case["kind"] == "join":
                bufs = {"z": like(st["y"]), "h": None if st["w_pre"] is None else like(v)}
            else:
                bufs = {"dx": like(v), "dy": like(st["y"]), "dgate": like(st["gate"]), "dw_post": like(st["w_post"]),
                        "dw_pre": like(st["w_pre"])}
        st["plan"] = (d, torch.empty(size, dtype=torch.uint8, device=DEV) if size else None, bufs)
    return (etd, *st["plan"])


def _run_own(st):
    etd, d, ws, bufs = _plan(st)
    kind = st["case"]["kind"]
    if kind == "adapt":
        etd.moe_grouped_ffn_adapted(d, st["x"], st["offsets"], st["pairs"], st["adapter_ids"], st["gate"], st["up"],
                                    st["down"], bufs, st["y"], ws)
        return st["y"]
    if kind == "join":
        etd.moe_block_join(d, st["x"], st["y"], st["gate"], st["w_post"], st["w_pre"], bufs["z"], bufs["h"])
    else:
        etd.moe_block_join_backward(d, st["z"], st["y"], st["gate"], st["w_post"], st["w_pre"], st["dz"], st["dh"],
                                    bufs["dx"], bufs["dy"], bufs["dgate"], bufs["dw_post"], bufs["dw_pre"], ws)
    return {k: v for k, v in bufs.items() if v is not None}


def run(state):
    if own:
        return _run_own(state)
    return {"join": _join_plain, "back": _back_plain, "adapt": _adapt_plain}[state["case"]["kind"]](state)


def work(case):
    dt = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "adapt":
        H, I, L, P, R, n = (case[k] for k in "H I L P R n".split())
        w = _popularity(case)  # experts, and their adapters, that have rows, on average
        if case["spread"] == "one":
            experts, mine = P, P * (1.0 - case["plain"])
        else:
            experts = sum(1.0 - (1.0 - v / sum(w)) ** P for v in w)
            mine = n * sum(1.0 - (1.0 - v / sum(w) * (1.0 - case["plain"]) / n) ** P for v in w)
        return {"bytes": (3 * experts * H * I + 3 * mine * R * (H + I) + 2 * P * H) * dt,
                "flops": 6 * P * H * I + 6 * P * (1.0 - case["plain"]) * R * (H + I)}
    form = case["form"]
    whole = 1 if case["gate"] == "element" else 0
    if case["kind"] == "join":
        tensors = {"full": 4, "add": 4, "post": 3, "enter": 2}[form] + whole
        per = {"full": 13, "add": 7, "post": 8, "enter": 5}[form]
    else:
        tensors = {"full": 6, "add": 6, "post": 4, "enter": 4}[form] + 2 * whole
        per = {"full": 28, "add": 18, "post": 14, "enter": 13}[form]
    return {"bytes": tensors * case["T"] * case["H"] * dt, "flops": per * case["T"] * case["H"]}


# ---- the definitions in 64 bits ---------------------------------------------------------------------
def _norm64(v, w, offset):
    ms = torch.linalg.vector_norm(v, dim=-1, keepdim=True) ** 2 / v.shape[-1]
    return v / torch.sqrt(ms + EPS) * (offset + w)


def _join64(case, x, y, gate, w_post, w_pre):
    """z (or None) and h (or None) of float64 tensors."""
    z = x
    if y is not None:
        b = y if w_post is None else _norm64(y, w_post, case["offset"])
        if gate is not None:
            v = torch.sigmoid(gate) if case["act"] == "sigmoid" else gate
            b = b * (v.unsqueeze(1) if case["gate"] == "token" else v)
        z = torch.add(x, b, alpha=case["scale"])
    return (z if y is not None else None), (None if w_pre is None else _norm64(z, w_pre, case["offset"]))


def _d(t):
    return None if t is None else t.double()


def _join_exact(st):
    z, h = _join64(st["case"], _d(st["x"]), _d(st["y"]), _d(st["gate"]), _d(st["w_post"]), _d(st["w_pre"]))
    return {k: v for k, v in (("z", z), ("h", h)) if v is not None}


def _back_exact(st):
    """By differentiating the definition: x is the z given less what the block adds."""
    case = st["case"]
    names = [k for k in ("y", "gate", "w_post", "w_pre") if st[k] is not None]
    p = {k: st[k].double().requires_grad_() for k in names}
    add = None
    if "y" in p:
        add, _ = _join64(case, torch.zeros_like(p["y"]), p["y"], p.get("gate"), p.get("w_post"), None)
    x = st["z"].double() if add is None else st["z"].double() - add.detach()
    x.requires_grad_()
    z = x if add is None else x + add
    total = (z * st["dz"].double()).sum()
    if "w_pre" in p:
        total = total + (_norm64(z, p["w_pre"], case["offset"]) * st["dh"].double()).sum()
    grads = torch.autograd.grad(total, [x] + [p[k] for k in names])
    known = dict(zip(["x"] + names, grads))
    out = {"dx": known["x"]}
    for k, v in (("dy", "y"), ("dgate", "gate"), ("dw_post", "w_post"), ("dw_pre", "w_pre")):
        if v in known:
            out[k] = known[v]
    return out


def _adapt_exact(st):
    y = torch.zeros((st["case"]["P"], st["case"]["H"]), dtype=torch.float64, device=DEV)
    at = 0
    for e, n in enumerate(st["counts"]):
        if n:
            ids = st["ids"][at:at + n]
            mine = {a: torch.tensor([i for i, b in enumerate(ids) if b == a], device=DEV) for a in set(ids) if a >= 0}

            def through(v, name):
                o = v @ st[name][e].double().T
                for a, rows in mine.items():
                    low = v[rows] @ st[name + "_a"][a, e].double().T
                    o[rows] += st["scale"][a].double() * (low @ st[name + "_b"][a, e].double().T)
                return o

            x = st["x"][at:at + n].double()
            g = through(x, "gate")
            y[at:at + n] = through(g * torch.sigmoid(g) * through(x, "up"), "down")
        at += n
    return y


def exact(case, seed):
    st = prepare(case, seed)
    return {"join": _join_exact, "back": _back_exact, "adapt": _adapt_exact}[case["kind"]](st)
