"""Orthogonalisation on the GPU of gradients with few directions, such as those of an expert that saw
few tokens: nothing of a broad floor hides what a rounding leaves in the directions that should stay
empty, and what every step multiplies."""

import numpy as np
import pytest

from tests._harness import say
from tests.test_gpu_muon import TOL, newton_schulz_f64, orthogonalize

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
