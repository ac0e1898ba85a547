"""Workspaces hold what the calls use, no more.  No GPU."""

import pytest

import expert_token_dispatch_amd as etd


# bf16: X, the X after it and the low halves are each held as they are and transposed, but a tall
# matrix's low halves only as they are
@pytest.mark.parametrize("steps,halves", [(1, 1), (5, 1), (6, 2), (10, 2)])
@pytest.mark.parametrize("sides", [(600, 2000), (256, 512)])
def test_a_tall_stack_holds_its_low_halves_once(sides, steps, halves):
    count, (m, n) = 8, sides
    copy = 2 * count * (-(-m // 64) * 64) * (-(-n // 64) * 64)
    wide = etd.moe_muon_workspace_size(etd.make_muon_desc(count, m, n, steps=steps))
    tall = etd.moe_muon_workspace_size(etd.make_muon_desc(count, n, m, steps=steps))
    assert wide - tall == halves * copy
    f32 = [etd.moe_muon_workspace_size(etd.make_muon_desc(count, *s, dtype="f32", steps=steps)) for s in (sides, sides[::-1])]
    assert f32[0] == f32[1]                       # float32: no low halves
