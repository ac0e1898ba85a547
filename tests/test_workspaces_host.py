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


def test_the_packed_layer_reserves_nothing_for_the_other_feed_forward():
    d = etd.make_desc(8192, 2048, 2816, 8, 2)      # its products may be cut along K, in pieces of 256 KB
    plain = etd.moe_workspace_size(d, etd.MOE_STAGE_FFN)
    h = etd.moe_packed_workspace_size(d, etd.MOE_STAGE_FFN)     # bf16: no scratch of its own
    assert h == 8192 * 2 * 2816 * 2 and plain > h + (100 << 20)
    layer, packed = etd.moe_workspace_size(d, etd.MOE_STAGE_LAYER), etd.moe_packed_workspace_size(d, etd.MOE_STAGE_LAYER)
    assert layer - packed == plain - h
    # float32 with many rows: the unpacked stacks, and what the products on them need
    f = etd.make_desc(8192, 512, 256, 8, 2, dtype="f32")
    scratch = etd.moe_packed_workspace_size(f, etd.MOE_STAGE_FFN) - 8192 * 2 * 256 * 4
    assert scratch >= 3 * 8 * 512 * 256 * 4
    assert etd.moe_packed_workspace_size(f, etd.MOE_STAGE_LAYER) == etd.moe_workspace_size(f, etd.MOE_STAGE_LAYER) + scratch
