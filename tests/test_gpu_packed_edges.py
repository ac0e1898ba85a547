"""Expert weights in 4 bits at the ends of the format and of the sizes."""

import numpy as np
import pytest

from tests._harness import np_of, say
from tests.test_gpu_packed_experts import TYPES, ffn_packed, packed_by_definition, values_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import expert_token_dispatch_amd as etd  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["out_in", "in_out"])
def test_every_scale_byte(layout, dtype):
    """From 2^-127, where values are subnormal, past the type's largest value, where they are infinite."""
    codes = torch.arange(256, dtype=torch.uint8).reshape(1, 16, 16).repeat(1, 16, 1)
    scales = torch.arange(256, dtype=torch.uint8).reshape(1, 256, 1)
    w = torch.empty((1, 256, 32) if layout == "out_in" else (1, 32, 256), dtype=TYPES[dtype], device="cuda")
    etd.moe_unpack_weights(codes.cuda(), scales.cuda(), w, weight_layout=layout)
    want = values_of(codes.numpy(), scales.numpy())
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    got = w.cpu().double().numpy()
    np.testing.assert_array_equal(got if layout == "out_in" else got.transpose(0, 2, 1), want)


@pytest.mark.parametrize("layout", ["out_in", "in_out"])
@pytest.mark.parametrize("e", [-118, -123, -124, -125, -126, -127, -130, -149])
def test_packing_of_tiny_groups(e, layout):
    rng = np.random.default_rng(-e)
    w = np.ldexp(rng.integers(-16, 17, (2, 16, 64)) / 8.0, e).astype(np.float32)    # down to subnormal weights
    stored = torch.from_numpy(w if layout == "out_in" else np.ascontiguousarray(w.transpose(0, 2, 1))).cuda()
    codes = torch.empty((2, 16, 32), dtype=torch.uint8, device="cuda")
    scales = torch.empty((2, 16, 2), dtype=torch.uint8, device="cuda")
    etd.moe_pack_weights(stored, codes, scales, weight_layout=layout)
    got = values_of(codes.cpu().numpy(), scales.cpu().numpy())
    np.testing.assert_array_equal(got, packed_by_definition(w.astype(np.float64)))


@pytest.mark.parametrize("rows", [3, 40])
def test_bf16_experts_too_large_for_the_kernels_on_codes(rows):
    """Codes of 4 GiB and more: the stacks are unpacked.  3 rows, and more than 32, take different products."""
    side = 92736                                  # side^2 / 2 is just past 2^32
    # rows on both sides of 4 GiB of weights, of 2^32 weights and of 4 GiB of codes, and the last
    at = [0, 5, 23157, 23158, 46314, 46315, 92627, 92628, side - 1]
    say(f"[packed ffn] H = I = {side}, rows={rows}")
    rng = np.random.default_rng(rows)
    codes = torch.zeros((1, side, side // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((1, side, side // 32), 127, dtype=torch.uint8, device="cuda")
    c = rng.integers(0, 256, (len(at), side // 2), dtype=np.uint8)
    s = rng.integers(117, 120, (len(at), side // 32)).astype(np.uint8)
    codes[0, at], scales[0, at] = torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()
    x = torch.from_numpy(rng.standard_normal((rows, side), dtype=np.float32)).bfloat16()
    y = ffn_packed(x.cuda(), [rows], {n: (codes, scales) for n in ("gate", "up", "down")})
    got = np_of(y).astype(np.float64)
    del codes, scales, y
    torch.cuda.empty_cache()
    w = values_of(c, s)                           # the other weights are zero: so is the rest of h, and of y
    x64 = x.double().numpy()
    a = x64 @ w.T
    ref = (a / (1.0 + np.exp(-a)) * a) @ w[:, at].T
    # h and y rounded once, half a step each; a sum of 92736 products in float32 is 2^-15 off
    err = np.linalg.norm(got[:, at] - ref) / np.linalg.norm(ref)
    say(f"[packed ffn]   error {err:.2e}")
    assert err <= 2.0 ** -7
    got[:, at] = 0.0
    assert not got.any()
