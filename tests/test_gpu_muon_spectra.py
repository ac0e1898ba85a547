"""Orthogonalisation on the GPU of gradients with few directions, such as those of an expert that saw
few tokens: nothing of a broad floor hides what a rounding leaves in the directions that should stay
empty, and what every step multiplies."""

import numpy as np
import pytest

from tests._harness import say
from tests.test_gpu_muon import TOL, USUAL, newton_schulz_f64, orthogonalize

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
