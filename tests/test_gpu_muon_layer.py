"""The layer's weight update: the workspace that its calls share, eager and captured."""

import pytest

import synth
from tests._harness import layer_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# out_in: gate and up are taller than wide or the other way round, down the opposite
@pytest.mark.parametrize("H,I", [(320, 288), (160, 384)])
def test_a_captured_update_keeps_its_workspace_when_another_call_takes_more_steps(H, I):
    s = synth.spec("gptoss_ep8_share", T=64, H=H, I=I, E=4, k=2, L=4)
    inp = synth.make_layer(s)

    def fresh():
        layer, x = layer_of(inp)
        state = layer.muon_state()
        y, saved = layer.forward_train(x)
        gen = torch.Generator(device="cuda").manual_seed(5)
        dy = torch.randn(y.shape, device="cuda", generator=gen).to(y.dtype)
        return layer, state, layer.backward(x, saved, dy)

    layer, state, grads = fresh()
    eager, eager_state, _ = fresh()
    layer.muon_update(grads, state, lr=1e-2)                   # warm-up, and the workspace
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.muon_update(grads, state, lr=1e-2)
    size = max(w.numel() for w in layer._ws.values() if w is not None)
    layer.muon_update(grads, state, lr=1e-2, steps=10)
    fill = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]  # where freed memory would go
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
    assert all(bool((f == 7).all()) for f in fill)
    eager.muon_update(grads, eager_state, lr=1e-2)
    eager.muon_update(grads, eager_state, lr=1e-2, steps=10)
    for _ in range(3):
        eager.muon_update(grads, eager_state, lr=1e-2)
    torch.cuda.synchronize()
    for n in layer.MUON_WEIGHTS:
        assert torch.equal(state["master"][n], eager_state["master"][n])
        assert torch.equal(getattr(layer, n), getattr(eager, n))
