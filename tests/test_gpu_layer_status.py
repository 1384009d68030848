"""A layer's status covers the products that make its logits and its gradients."""
import pytest
import torch

from combine_overlap_b200 import synth

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")


def _layer(T=300, d=512, f=256, E=16, k=3):
    wl = synth.small("status", T, d, f, E, k, "uniform", 5)
    inp = synth.make_inputs(wl, "cuda")
    g = torch.Generator().manual_seed(1)
    router = moe.Router((torch.randn(d, E, generator=g) * d ** -0.5).bfloat16().cuda())
    make = lambda: moe.MoELayer(inp["W1"], inp["W3"], inp["W2"], k, T, router=router)  # noqa: E731
    return inp["x"], make(), make()


def test_a_timeout_of_the_gate_projection_is_the_layers():
    x, layer, other = _layer()
    want = layer.forward(x)
    assert layer.get_status()[0] == moe.MOE_OK
    other.forward(x)
    for call in (lambda: layer.forward(x), lambda: layer.forward_train(x)):
        with moe.linear_debug(timeout_us=20000, withhold=True):
            call()
        # the FFN's own status knows nothing of it, and asking for another one takes nothing away
        assert moe.get_status(layer.ws)[0] == moe.MOE_OK
        assert moe.linear_get_status() == moe.MOE_ERR_TIMEOUT
        assert layer.get_status()[0] == moe.MOE_ERR_TIMEOUT
        assert layer.get_status()[0] == moe.MOE_OK
    assert other.get_status()[0] == moe.MOE_ERR_TIMEOUT      # any product's on the device since its own last one
    assert torch.equal(layer.forward(x), want) and layer.get_status()[0] == moe.MOE_OK


def test_a_timeout_of_the_gradients_is_the_layers():
    x, layer, _ = _layer()
    out, saved = layer.forward_train(x)
    dout = torch.randn(out.shape, device="cuda").bfloat16()
    want = layer.backward(dout, saved)["dWg"]
    assert layer.get_status()[0] == moe.MOE_OK
    with moe.linear_debug(timeout_us=20000, withhold=True):
        layer.backward(dout, saved)
    assert layer.get_status()[0] == moe.MOE_ERR_TIMEOUT
    assert torch.equal(layer.backward(dout, saved)["dWg"], want)
    assert layer.get_status()[0] == moe.MOE_OK and moe.linear_get_status() == moe.MOE_ERR_TIMEOUT
    assert moe.linear_get_status() == moe.MOE_OK


def test_a_layer_without_a_router_has_the_workspaces_status():
    x, layer, _ = _layer()
    plain = moe.MoELayer(layer.W1, layer.W3, layer.W2, layer.k, x.shape[0])
    plain.forward(x, torch.randn(x.shape[0], layer.E, device="cuda"))
    assert plain.get_status() == moe.get_status(plain.ws) and plain.get_status()[0] == moe.MOE_OK
