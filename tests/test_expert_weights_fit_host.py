"""Packed experts that are not the descriptor's: refused by the bindings, without a GPU."""

import pytest
import torch

import expert_token_dispatch_amd as etd
from expert_token_dispatch_amd import _lib as L


def packed_of(count, hidden, intermediate):
    """A struct over host tensors of a layer's sizes, as make_packed_experts leaves it on the GPU."""
    t = {}
    for name, out, in_ in (("gate", intermediate, hidden), ("up", intermediate, hidden), ("down", hidden, intermediate)):
        t[name + "_codes"] = torch.zeros((count, out, in_ // 2), dtype=torch.uint8)
        t[name + "_scales"] = torch.zeros((count, out, in_ // 32), dtype=torch.uint8)
    v = L.PackedExperts(*[t[n].data_ptr() for n, _ in L.PackedExperts._fields_])
    v._tensors = t
    return v


def calls(d, packed):
    yield lambda: etd.moe_grouped_ffn_packed(d, None, None, packed, None)
    yield lambda: etd.moe_layer_forward_packed(d, None, None, None, None, packed, None, None)


# hidden, intermediate or local experts of another layer
@pytest.mark.parametrize("other", [(4, 128, 96), (4, 64, 128), (3, 64, 96), (5, 64, 96)])
def test_packed_experts_of_another_layer_are_refused(other):
    d = etd.make_desc(16, 64, 96, 8, 2, local_begin=2, local_count=4)
    for call in calls(d, packed_of(*other)):
        with pytest.raises(ValueError, match="of this layer"):
            call()


@pytest.mark.parametrize("field", [n for n, _ in L.PackedExperts._fields_])
def test_every_tensor_is_looked_at(field):
    d = etd.make_desc(16, 64, 96, 4, 2)
    for bad in (lambda t: t[:-1], lambda t: t[:, :-8], lambda t: t[..., :-1], lambda t: t.to(torch.int8),
                lambda t: t.transpose(1, 2).contiguous()):
        packed = packed_of(4, 64, 96)
        packed._tensors[field] = bad(packed._tensors[field])
        for call in calls(d, packed):
            with pytest.raises(ValueError, match=field):
                call()
    assert L._packed(d, packed_of(4, 64, 96)) and L._packed(d, None) is None
