"""The router's operators together, as they are used: a layer whose gate projection and
scored routing the library runs (one call, and step by step), the gradients back to the
gate's weights, and the layer with the scored router inside a CUDA graph."""
import numpy as np
import pytest
import torch

import router_ref as ref
from combine_overlap_b200 import synth

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")

ROUTERS = [dict(score=moe.SCORE_SIGMOID, n_groups=4, topk_groups=2, group_score=moe.GROUP_TOP2, scale=2.5, biased=True),
           dict(score=moe.SCORE_SOFTMAX, renorm=False, biased=False),
           dict(score=moe.SCORE_SOFTMAX, n_groups=4, topk_groups=3, biased=True)]


def _layer(opts, T=300, d=512, f=256, E=16, k=3, seed=5):
    wl = synth.small("router", T, d, f, E, k, "uniform", seed)
    inp = synth.make_inputs(wl, "cuda")
    g = torch.Generator().manual_seed(seed)
    opts = dict(opts)
    bias = (0.05 * torch.randn(E, generator=g)).cuda() if opts.pop("biased") else None
    Wg = (torch.randn(d, E, generator=g) * d ** -0.5).bfloat16().cuda()
    bg = (0.1 * torch.randn(E, generator=g)).cuda()
    router = moe.Router(Wg, bg, bias=bias, **opts)
    return inp["x"], moe.MoELayer(inp["W1"], inp["W3"], inp["W2"], k, T, router=router), router


@pytest.mark.parametrize("opts", ROUTERS)
@pytest.mark.parametrize("mode", [0, 1])
def test_layer_with_router(opts, mode):
    x, layer, router = _layer(opts)
    out, routing = layer.forward(x, mode=mode, outputs=True)
    steps, saved = layer.forward_train(x)
    torch.cuda.synchronize()
    assert moe.get_status(layer.ws)[0] == moe.MOE_OK
    assert torch.equal(routing["topk_idx"], saved["idx"]) and torch.equal(routing["topk_gate"], saved["gate"])
    assert torch.equal(out, steps)                       # the same kernels' arithmetic
    z = saved["logits"].cpu().numpy()
    b = None if router.bias is None else router.bias.cpu().numpy()
    idx, gate = ref.route(z, layer.k, router.score, b, router.n_groups, router.topk_groups,
                          router.group_score == moe.GROUP_TOP2, router.renorm, router.scale)
    assert np.array_equal(idx, saved["idx"].cpu().numpy())


def test_layer_without_router_is_what_it_was():
    x, layer, router = _layer(ROUTERS[1])
    logits = router.logits(x)
    plain = moe.MoELayer(layer.W1, layer.W3, layer.W2, layer.k, x.shape[0])
    want = moe.layer_forward(x, logits, layer.W1, layer.W3, layer.W2, layer.k, plain.ws)
    assert torch.equal(plain.forward(x, logits), want)
    with pytest.raises(ValueError):
        plain.forward(x)
    with pytest.raises(ValueError):
        plain.forward_train(x)


@pytest.mark.parametrize("opts", ROUTERS)
def test_router_gradients_end_to_end(opts):
    x, layer, router = _layer(opts)
    out, s = layer.forward_train(x)
    dout = torch.randn(out.shape, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    g = layer.backward(dout, s, want_dy=True)
    n = lambda t: t.detach().cpu().double().numpy()  # noqa: E731
    T, k = s["gate"].shape
    _, dgate, bg = ref.combine_backward(n(dout), n(s["y"]), s["row_of"].cpu().numpy(), n(s["gate"]), n(g["dy"]))
    z = s["logits"].cpu().numpy()
    idx = s["idx"].cpu().numpy()
    dz, bz = ref.route_backward(dgate, z, idx, router.score, router.renorm, router.scale)
    # dgate's own error goes through the same linear map
    big, _ = ref.route_backward(bg, z, idx, router.score, False, router.scale)
    S = np.array([1.0 if not router.renorm else ref.scores(z[t], router.score)[0][idx[t]].sum() for t in range(T)])
    through = 2 * router.scale * bg.sum(1, keepdims=True) / S[:, None]
    got = n(g["dlogits"])
    assert np.all(np.abs(got - dz) <= bz + through + 1e-37)
    r = ref.linear_backward(got, n(x), n(router.Wg), None, 0, ref.F32)
    assert np.all(np.abs(n(g["dWg"]) - r["dW"]) <= (1 + ref.F32) * r["bW"] + ref.F32 * np.abs(r["dW"]))
    assert np.all(np.abs(n(g["dbg"]) - r["dbias"]) <= 1.01 * r["bb"] + ref.F32 * np.abs(r["dbias"]))
    assert g["dx"].shape == x.shape and torch.isfinite(g["dx"].float()).all()
    # a second pass over the same saved state gives the same bits
    again = layer.backward(dout, s)
    assert torch.equal(again["dWg"], g["dWg"]) and torch.equal(again["dlogits"], g["dlogits"])
    assert again["dy"] is None


def test_layer_with_router_and_gradients_in_a_graph():
    x, layer, router = _layer(ROUTERS[0])
    dout = torch.randn(x.shape, device="cuda").bfloat16()

    def step():
        out = layer.forward(x)
        _, s = layer.forward_train(x)
        return out, layer.backward(dout, s)["dWg"]

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, dW = step()
    for seed in (1, 2):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)).bfloat16())
        g.replay()
        torch.cuda.synchronize()
        a, b = out.clone(), dW.clone()
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_shared_expert_onto_the_routed_output():
    """A shared SwiGLU expert beside the routed ones: its down projection adds the routed
    output in the epilogue."""
    x, layer, _ = _layer(ROUTERS[1])
    d, f = layer.d, layer.f
    g = torch.Generator().manual_seed(2)
    Ws1, Ws2 = ((torch.randn(*s, generator=g) * s[0] ** -0.5).bfloat16().cuda() for s in ((d, f), (f, d)))
    routed = layer.forward(x)
    h = moe.linear(x, Ws1, act=moe.ACT_SILU)
    out = moe.linear(h, Ws2, residual=routed)
    n = lambda t: t.cpu().double().numpy()  # noqa: E731
    want, _, bound, _ = ref.linear(n(h), n(Ws2), None, n(routed), 0, ref.BF16)
    assert np.all(np.abs(n(out) - want) <= bound)
