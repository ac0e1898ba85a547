"""Which product kernel the experts with adapters take: the shapes that stand for each keep it."""

import pytest

from tests._adapted_paths import CASES, SHAPES, kernel_of


@pytest.mark.parametrize("kernel,H,I,Lc,P,layout,spread", CASES)
@pytest.mark.parametrize("R", (8, 16, 72))
def test_each_shape_takes_its_kernel(kernel, H, I, Lc, P, layout, spread, R):
    assert kernel_of(H, I, Lc, P, layout, R) == kernel


def test_every_kernel_has_a_shape():
    assert set(SHAPES) == {"decode", "tiles", "large", "general"} and all(SHAPES.values())


@pytest.mark.parametrize("P", (65, 250))
@pytest.mark.parametrize("layout,dtype", [("out_in", "bf16"), ("in_out", "bf16"), ("out_in", "f32")])
def test_many_rows_on_one_of_few_small_experts_stay_in_the_decode_kernel(layout, dtype, P):
    assert kernel_of(128, 200, 8, P, layout, dtype=dtype) == "decode"
    assert kernel_of(64, 2048, 32, P, layout, dtype=dtype) == "decode"
    assert kernel_of(2048, 64, 64, P, layout, dtype=dtype) == "decode"
