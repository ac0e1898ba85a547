"""Orthogonalisation on the GPU of gradients with few directions, such as those of an expert that saw
few tokens: nothing of a broad floor hides what a rounding leaves in the directions that should stay
empty, and what every step multiplies.  And of matrices whose entries take few values: their roundings
are alike and add up."""

import numpy as np
import pytest

from tests._harness import say
from tests.test_gpu_muon import TOL, USUAL, gradient, newton_schulz, newton_schulz_f64, orthogonalize

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import expert_token_dispatch_amd as etd  # noqa: E402


def outer(shape, rank, seed):
    """Sums of `rank` outer products of normal vectors, rounded to bfloat16."""
    rng = np.random.default_rng(seed)
    L, R, C = shape
    g = rng.standard_normal((L, R, rank)) @ rng.standard_normal((L, rank, C))
    return torch.from_numpy(g.astype(np.float32)).bfloat16()


def off_by(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


# One phase, from the split X_0 straight to the result.  Without its low half, 2^-12 of the high one
# and in every direction, three steps leave a^3 = 41 times that beside singular values of 0.7: 1.2%.
@pytest.mark.parametrize("steps", [1, 2, 3])
@pytest.mark.parametrize("shape", [(14, 990, 1010), (14, 1010, 990)])
def test_few_steps_on_a_stack_that_fills_the_card(shape, steps):
    say(f"[muon] stack {shape}, {steps} steps")
    g = outer(shape, 1, steps).cuda()
    o = orthogonalize(g, "bf16", steps=steps)
    m = etd.make_muon_desc(*shape, steps=steps, momentum=0.0, nesterov=False, lr=1.0, update_scale=-1.0)
    ws = torch.full((etd.moe_muon_workspace_size(m),), 255, dtype=torch.uint8, device="cuda")
    mast, weight, mom = torch.zeros(shape, device="cuda"), torch.zeros_like(g), torch.zeros(shape, device="cuda")
    etd.moe_muon_update(m, g, mom, weight, ws, master=mast)   # from zero: W is the orthogonalised gradient
    torch.cuda.synchronize()
    for z in (0, 7, 13):
        ref = newton_schulz_f64(g[z].double(), steps)
        say(f"[muon]   matrix {z} error {off_by(o[z], ref):.2e}, update {off_by(mast[z], ref):.2e}")
        assert off_by(o[z], ref) <= TOL["bf16"]
        assert off_by(mast[z], ref) <= TOL["bf16"]


def integers(shape, seed):
    """Sums of four outer products of small integers: the rank is four in bfloat16 too."""
    rng = np.random.default_rng(seed)
    L, R, C = shape
    g = rng.integers(-3, 4, (L, R, 4)) @ rng.integers(-3, 4, (L, 4, C))
    return torch.from_numpy(g.astype(np.float32)).bfloat16()


def newton_schulz_f32(u, steps, eps=1e-7):
    """The formula on float32 matrices, with float32 products."""
    a, b, c = USUAL
    x = (u.double() / (u.double().norm() + eps)).float()
    for _ in range(steps):
        wide = x.shape[0] <= x.shape[1]
        g = torch.mm(x, x.t().contiguous()) if wide else torch.mm(x.t().contiguous(), x)
        p = b * g + c * torch.mm(g, g)
        x = a * x + (torch.mm(p, x) if wide else torch.mm(x, p))
    return x


# From the first X on a rounding that leaves the matrix's few directions grows a = 3.44-fold a step,
# whatever the type: float32's own error shows by how much.  The sum of two float16 is 22 bits, two
# fewer than float32: four times that error, beside what every case is allowed.
@pytest.mark.parametrize("steps", [4, 5, 6, 7, 8, 9, 10])
@pytest.mark.parametrize("shape", [(2, 96, 160), (2, 160, 96), (1, 200, 256), (1, 300, 400), (1, 400, 300), (1, 257, 700),
                                   (14, 990, 1010), (14, 1010, 990)])
def test_matrices_of_rank_four_over_the_steps(shape, steps):
    say(f"[muon] rank 4 {shape}, {steps} steps")
    g = integers(shape, shape[1]).cuda()
    o = orthogonalize(g, "bf16", steps=steps)
    for z in sorted({0, shape[0] - 1}):
        ref = newton_schulz_f64(g[z].double(), steps)
        single = off_by(newton_schulz_f32(g[z], steps), ref)
        say(f"[muon]   matrix {z} error {off_by(o[z], ref):.2e}, float32 {single:.2e}")
        assert off_by(o[z], ref) <= TOL["bf16"] + 4 * single


@pytest.mark.parametrize("shape", [(1, 4100, 4170), (1, 4170, 4100)])
def test_large_matrices_of_rank_four(shape):
    g = integers(shape, 6).cuda()
    o = orthogonalize(g, "bf16", steps=8)
    ref = newton_schulz_f64(g[0].double(), 8)
    single = off_by(newton_schulz_f32(g[0], 8), ref)
    say(f"[muon] rank 4 {shape}, 8 steps: error {off_by(o[0], ref):.2e}, float32 {single:.2e}")
    assert off_by(o[0], ref) <= TOL["bf16"] + 4 * single


@pytest.mark.parametrize("shape", [(2, 96, 160), (14, 990, 1010)])
def test_update_of_matrices_of_rank_four(shape):
    steps = 8
    g = integers(shape, 5).cuda()
    m = etd.make_muon_desc(*shape, steps=steps, momentum=0.0, nesterov=False, lr=1.0, update_scale=-1.0)
    ws = torch.full((etd.moe_muon_workspace_size(m),), 255, dtype=torch.uint8, device="cuda")
    mast, weight, mom = torch.zeros(shape, device="cuda"), torch.zeros_like(g), torch.zeros(shape, device="cuda")
    etd.moe_muon_update(m, g, mom, weight, ws, master=mast)
    torch.cuda.synchronize()
    assert torch.equal(weight, mast.bfloat16())
    for z in (0, shape[0] - 1):
        ref = newton_schulz_f64(g[z].double(), steps)
        assert off_by(mast[z], ref) <= TOL["bf16"] + 4 * off_by(newton_schulz_f32(g[z], steps), ref)


# the rounding of matrices with few directions to bfloat16 leaves 2^-9 of them everywhere, as a gradient has it
@pytest.mark.parametrize("rank", [1, 4])
@pytest.mark.parametrize("shape", [(1, 128, 512), (1, 200, 256), (1, 500, 300), (14, 990, 1010)])
def test_gradients_of_few_tokens(shape, rank):
    g = outer(shape, rank, shape[1] + rank).cuda()
    for steps in (5, 10):
        o = orthogonalize(g, "bf16", steps=steps)
        ref = newton_schulz_f64(g[0].double(), steps)
        single = off_by(newton_schulz_f32(g[0], steps), ref)
        say(f"[muon] {shape} rank {rank}, {steps} steps: error {off_by(o[0], ref):.2e}, float32 {single:.2e}")
        assert off_by(o[0], ref) <= TOL["bf16"] + 4 * single


def float16_of(x, scale):
    return np.ldexp(np.ldexp(x, scale).astype(np.float16).astype(np.float32), -scale)


def mirrored(m):
    return np.triu(m) + np.triu(m, 1).T


def stored_in_float16(u, steps, eps=1e-7):
    """The formula with what a bfloat16 stack's products round: X, A and T = P A scaled by 2^14 and 2^12,
    P and Q by 2^9 beside float32 diagonals, in single steps or in phases of three, two, two, .. steps;
    sums in float32, the result not rounded."""
    a, b, c = (np.float32(v) for v in USUAL)
    x = (u / (np.linalg.norm(u) + eps)).astype(np.float32)
    tall = x.shape[0] > x.shape[1]
    x = np.ascontiguousarray(x.T) if tall else x
    short, long = x.shape
    single = short <= 128 or (short <= 256 and long < 2 * short)
    done, split = 0, True
    while done < steps:
        hi = float16_of(x, 14)
        lo = float16_of(x - hi, 14) if split else np.zeros_like(x)
        n = min(steps - done, 1 if single else 3 if done == 0 else 2)
        g, q = float16_of(mirrored(hi @ hi.T), 12), None
        for j in range(n):
            p = mirrored(b * g + c * (g @ g))
            dp, p = np.diag(p) + a, float16_of(p - np.diag(np.diag(p)), 9)
            if q is None:
                q, dq = p, dp
            else:
                r = mirrored(p @ q + dp[:, None] * q + p * dq[None])
                dq, q = np.diag(r) + dp * dq, float16_of(r - np.diag(np.diag(r)), 9)
            if j + 1 < n:
                t = float16_of(mirrored(p @ g + dp[:, None] * g), 12)
                g = float16_of(mirrored(p @ t + dp[:, None] * t), 12)
        x = q @ lo + q @ hi + dq[:, None] * (hi + lo)
        done += n
        split = steps - done > 2 or (single and done == 1)
    return (x.T if tall else x).astype(np.float64)


def few_values(kind, R, C):
    rng = np.random.default_rng(3)
    g = np.zeros((R, C))
    if kind == "one entry":
        g[R // 3, C // 2] = -3.0
    elif kind == "powers of two":
        g = 2.0 ** rng.integers(-3, 4, (R, 1)) * 2.0 ** rng.integers(-3, 4, (1, C))
    elif kind == "ones":
        g[:] = 1.0
    elif kind == "equal rows":
        g[:R // 4] = rng.integers(-3, 4, (1, C))
    else:
        g[:, :C // 4] = rng.integers(-3, 4, (R, 1))
    return g


# The error that those roundings leave, once and a half (a float32 sum in another order may turn a
# rounding), and half a step of the result.  In single steps it is 0.1 to 0.6%; in phases, whose errors
# of A and P grow by up to a^2 = 12 until X is multiplied, 0.1 to 4% (equal columns, 256 x 1024).
@pytest.mark.parametrize("steps", [5, 7])
@pytest.mark.parametrize("kind", ["one entry", "powers of two", "ones", "equal rows", "equal columns"])
@pytest.mark.parametrize("shape", [(1, 100, 120), (1, 60, 300), (1, 300, 320), (1, 256, 1024), (1, 700, 520),
                                   (14, 990, 1010)])
def test_matrices_of_few_values(shape, kind, steps):
    L, R, C = shape
    u = few_values(kind, R, C)
    g = torch.from_numpy(u).bfloat16().cuda().expand(shape).contiguous()
    o = orthogonalize(g, "bf16", steps=steps)
    ref = newton_schulz(u, steps)
    norm = np.linalg.norm(ref)
    model = np.linalg.norm(stored_in_float16(u, steps) - ref) / norm
    err = np.linalg.norm(o[L - 1].double().cpu().numpy() - ref) / norm
    say(f"[muon] {kind} {shape}, {steps} steps: error {err:.2e}, of the stored values {model:.2e}")
    assert err <= 1.5 * model + 2.0 ** -8
    if kind == "one entry" or min(R, C) <= 128:
        assert err <= TOL["bf16"]


# Gradients in a few rows or columns: where that leaves one or two along K of A = X X^T, nothing averages
# out either (1.4% for one row of 700 x 520); from five on it is 0.2 to 0.6%.
@pytest.mark.parametrize("count", [1, 2, 5])
@pytest.mark.parametrize("side", ["rows", "columns"])
@pytest.mark.parametrize("shape", [(1, 128, 512), (1, 200, 256), (1, 300, 500), (1, 700, 520), (14, 1010, 990)])
def test_gradients_in_few_rows(shape, side, count):
    L, R, C = shape
    rng = np.random.default_rng(count)
    u = np.zeros((R, C))
    if side == "rows":
        u[3:3 + count] = rng.standard_normal((count, C))
    else:
        u[:, 3:3 + count] = rng.standard_normal((R, count))
    g = torch.from_numpy(u).bfloat16()
    o = orthogonalize(g.cuda().expand(shape).contiguous(), "bf16")
    u = g.double().numpy()
    ref = newton_schulz(u)
    norm = np.linalg.norm(ref)
    model = np.linalg.norm(stored_in_float16(u, 5) - ref) / norm
    err = np.linalg.norm(o[L - 1].double().cpu().numpy() - ref) / norm
    say(f"[muon] {count} {side} of {shape}: error {err:.2e}, of the stored values {model:.2e}")
    assert err <= 1.5 * model + 2.0 ** -8
    if count == 5:
        assert err <= TOL["bf16"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(4, 80, 300), (4, 300, 290), (14, 990, 1010)])
def test_the_same_call_gives_the_same_bits(shape, dtype):
    g = torch.from_numpy(gradient(shape, 7)).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
    g[1] = 0
    g[2, 3, 5] = float("nan")
    a, b = orthogonalize(g, dtype), orthogonalize(g.clone(), dtype)
    assert torch.isnan(a[2]).all() and torch.isnan(b[2]).all()
    assert torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))
    assert not torch.isnan(a[[z for z in range(shape[0]) if z != 2]]).any()
