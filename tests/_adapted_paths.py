"""Shapes of the experts with adapters, under the product kernel that each is there for."""

import expert_token_dispatch_amd as etd
from expert_token_dispatch_amd import _lib as L

# kernel -> (H, I, L, P, layout, spread).  "decode" twice: with waves that split K, and with whole ones in the
# first product (64 or more column blocks an expert), or in the second; "large" ends segments in its wide tiles
# (600 rows on each of 4: 88 behind two whole tiles), in regular ones (1200 on each of 2), and cuts tiles along K
# where an expert has 4096 k.
SHAPES = {
    "decode": [(128, 200, 8, 60, "out_in", "even"), (128, 200, 8, 60, "in_out", "even"),
               (64, 2048, 32, 300, "out_in", "even"), (2048, 64, 64, 300, "out_in", "even")],
    "tiles": [(136, 200, 3, 300, "out_in", "even"), (520, 136, 3, 900, "out_in", "even"),
              (2048, 256, 2, 1500, "out_in", "even")],
    "large": [(256, 4096, 4, 2400, "out_in", "even"), (4096, 4096, 2, 2400, "out_in", "even"),
              (4096, 4096, 2, 2200, "out_in", "even"), (256, 512, 4, 1100, "in_out", "even")],
    "general": [(136, 264, 3, 500, "in_out", "even")],
}
CASES = [(kernel, *s) for kernel, shapes in SHAPES.items() for s in shapes]


def align(n):
    return (n + 255) // 256 * 256


def kernel_of(H, I, Lc, P, layout, R=16, dtype="bf16"):
    """Which product kernel a call takes, by what its workspace holds behind the rows of h, ids and both u."""
    d = etd.make_desc(P, H, I, Lc, 1, dtype=dtype, weight_layout=layout)
    a = L.Adapters(2, R, *[256] * 7)
    size = 2 if dtype == "bf16" else 4
    own = etd.moe_adapted_workspace_size(d, a, L.MOE_STAGE_FFN) - align(P * I * size) - align(P * 4) - align(P * 2 * R * 4) - align(P * R * 4)
    if own == 0:
        return "decode" if P <= 32 * Lc and (dtype == "bf16" or layout == "out_in") else "general"
    return "tiles" if own == 8 * 32 * 128 * 256 * 4 else "large"
