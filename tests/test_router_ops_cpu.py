"""The router's operators without a GPU: the references' gradients against differences,
and the refusals of the C ABI and of the binding (all of them before any CUDA call)."""
import ctypes

import numpy as np
import pytest
import torch

import router_ref as ref

moe = pytest.importorskip("combine_overlap_b200.moe")
P = ctypes.c_void_p
INVALID, UNSUPPORTED, WORKSPACE = moe.MOE_ERR_INVALID, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE


# ---- the references against central differences (64 bits, step 1e-5: error ~1e-9) ----
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_is_the_difference_quotient(kind, renorm):
    rng = np.random.default_rng(7)
    z, dg = rng.normal(size=(5, 9)), rng.normal(size=(5, 3))
    z[1, 4] = -np.inf
    idx, _ = ref.route(z, 3, kind, renorm=renorm, scale=1.5)
    dz, _ = ref.route_backward(dg, z, idx, kind, renorm, 1.5)

    def loss(zz):
        tot = 0.0
        for t in range(5):
            p, _ = ref.scores(zz[t], kind)
            w = p[idx[t]]
            tot += (dg[t] * 1.5 * (w / w.sum() if renorm else w)).sum()
        return tot

    for t in range(5):
        for e in range(9):
            if np.isinf(z[t, e]):
                assert dz[t, e] == 0
                continue
            a, b = z.copy(), z.copy()
            a[t, e] += 1e-5
            b[t, e] -= 1e-5
            assert abs((loss(a) - loss(b)) / 2e-5 - dz[t, e]) < 1e-8


@pytest.mark.parametrize("kind", [0, 1, 2, 3])
def test_linear_gradient_is_the_difference_quotient(kind):
    rng = np.random.default_rng(3)
    x, W, b = rng.normal(size=(4, 5)), rng.normal(size=(5, 3)), rng.normal(size=3)
    dout = rng.normal(size=(4, 3))
    r = ref.linear_backward(dout, x, W, x @ W + b, kind, 0.0)
    f = lambda x_, W_, b_: (dout * ref.act(kind, x_ @ W_ + b_)).sum()  # noqa: E731
    for name, a, g in (("x", x, r["dx"]), ("W", W, r["dW"]), ("b", b, r["dbias"])):
        for at in np.ndindex(a.shape):
            keep, h = a[at], 1e-5
            a[at] = keep + h
            up = f(x, W, b)
            a[at] = keep - h
            down = f(x, W, b)
            a[at] = keep
            assert abs((up - down) / (2 * h) - g[at]) < 1e-7, (name, at)


def test_route_reference_masks_ties_and_groups():
    inf = np.inf
    z = np.array([[0.0, 0.0, 1.0, 1.0], [-inf, -inf, -inf, -inf], [2.0, -inf, np.nan, 1.0]])
    idx, gate = ref.route(z, 3)
    assert idx.tolist() == [[2, 3, 0], [0, 1, 2], [0, 3, 1]]
    assert gate[1].tolist() == [0, 0, 0] and gate[2, 2] == 0 and abs(gate[2].sum() - 1) < 1e-15
    # two groups of two: the best pair wins by its sum, the best single by its maximum
    z = np.array([[3.0, -9.0, 2.5, 2.4]])
    assert ref.route(z, 2, kind=1, n_groups=2, topk_groups=1, top2=True)[0].tolist() == [[2, 3]]
    assert ref.route(z, 2, kind=1, n_groups=2, topk_groups=1, top2=False)[0].tolist() == [[0, 1]]


# ---- refusals ----
def _router(**kw):
    r = moe.RouterArgs(0, None, 1, 0, 0, 1, 1.0)
    for k_, v in kw.items():
        setattr(r, k_, v)
    return r


def _route(T=16, E=8, k=2, r=None, logits=0x1000, idx=0x2000, gate=0x3000, counts=None, ws=None, n=0):
    r = r if r is not None else _router()
    return moe._lib.moe_route_scored(P(logits), T, E, k, ctypes.byref(r), P(idx), P(gate), P(counts), P(ws), n, None)


def test_route_scored_refusals():
    assert _route(T=0) == INVALID
    assert _route(k=9) == INVALID                       # k > E
    assert _route(E=16, k=9) == UNSUPPORTED
    assert _route(E=300) == UNSUPPORTED
    assert _route(T=1 << 29, E=8, k=4) == UNSUPPORTED   # 2^31 slots
    assert _route(r=_router(score=2)) == INVALID
    assert _route(r=_router(group_score=2)) == INVALID
    assert _route(r=_router(n_groups=3)) == INVALID      # does not divide 8
    assert _route(r=_router(n_groups=-1)) == INVALID
    assert _route(r=_router(n_groups=4, topk_groups=5)) == INVALID
    assert _route(k=3, r=_router(n_groups=8, topk_groups=2)) == INVALID   # 2 experts for k = 3
    assert _route(E=128, r=_router(n_groups=64, topk_groups=4)) == UNSUPPORTED
    assert _route(r=_router(scale=float("nan"))) == INVALID
    assert _route(r=_router(scale=float("inf"))) == INVALID
    assert _route(r=_router(bias=0x1004)) == INVALID
    assert _route(logits=0) == INVALID
    assert _route(gate=0x3008) == INVALID
    assert _route(counts=0x4000) == WORKSPACE
    assert _route(counts=0x4000, ws=0x5000, n=64) == WORKSPACE
    assert moe._lib.moe_route_scored(P(0x1000), 16, 8, 2, None, P(0x2000), P(0x3000), None, None, 0, None) == INVALID


def test_route_scored_backward_refusals():
    f = lambda T=16, E=8, k=2, r=None, dg=0x1000, out=0x4000: moe._lib.moe_route_scored_backward(  # noqa: E731
        P(dg), P(0x2000), P(0x3000), T, E, k, ctypes.byref(r if r is not None else _router()), P(out), None)
    assert f(T=0) == INVALID
    assert f(E=300) == UNSUPPORTED
    assert f(r=_router(score=-1)) == INVALID
    assert f(dg=0) == INVALID
    assert f(out=0x4004) == INVALID


def test_layer_forward_scored_refusals():
    a = moe.LayerArgs(256, 512, 1024, 8, 2, 0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000,
                      0, 0, 0, 0, 0, 0, 1, 0, 0, None, None)
    f = lambda a_, r, n=1 << 40: moe._lib.moe_layer_forward_scored(  # noqa: E731
        ctypes.byref(a_), ctypes.byref(r) if r else None, 1, P(0x100000), n, None)
    assert f(a, None) == INVALID
    assert f(a, _router(n_groups=3)) == INVALID
    assert f(a, _router(), 1024) == WORKSPACE
    a.d = 320
    assert f(a, _router()) == UNSUPPORTED
    a.T = 0
    assert f(a, _router()) == INVALID
    assert moe._lib.moe_layer_forward_scored(None, ctypes.byref(_router()), 1, P(0x100000), 1 << 40, None) == INVALID


def test_combine_backward_refusals():
    f = lambda T=16, d=512, k=2, dout=0x1000, dy=None, dg=0x5000: moe._lib.moe_combine_backward(  # noqa: E731
        P(dout), P(0x2000), P(0x3000), P(0x4000), T, d, k, P(dy), P(dg), None)
    assert f(T=0) == INVALID
    assert f(d=500) == UNSUPPORTED
    assert f(k=9) == UNSUPPORTED
    assert f(T=1 << 29, k=4) == UNSUPPORTED
    assert f(dout=0) == INVALID
    assert f(dy=0x6008) == INVALID
    assert f(dg=0) == INVALID


def _linear(**kw):
    a = moe.LinearArgs(16, 64, 32, 0x1000, 0x2000, None, None, 0, 0, 0x3000, None)
    for k_, v in kw.items():
        setattr(a, k_, v)
    return moe._lib.moe_linear(ctypes.byref(a), None, 0, None)


def test_linear_refusals():
    for field in ("M", "K", "N"):
        assert _linear(**{field: 0}) == INVALID
    assert _linear(M=1 << 30, K=1 << 20) == UNSUPPORTED
    assert _linear(act=4) == INVALID
    assert _linear(out_dtype=2) == INVALID
    assert _linear(x=0) == INVALID
    assert _linear(W=0x2002) == INVALID
    assert _linear(bias=0x2004) == INVALID
    assert _linear(residual=0x2008) == INVALID
    assert _linear(out=0) == INVALID
    assert _linear(pre=0x2004) == INVALID
    assert moe._lib.moe_linear(None, None, 0, None) == INVALID
    assert moe.linear_workspace_size(0, 8, 8) > 1 << 62


def _linear_bwd(ws=0x100000, n=1 << 40, **kw):
    a = moe.LinearBwdArgs(16, 64, 32, 0x1000, 0x2000, 0x3000, None, 0, 0, 1, 0x4000, 0x5000, 0x6000)
    for k_, v in kw.items():
        setattr(a, k_, v)
    return moe._lib.moe_linear_backward(ctypes.byref(a), P(ws), n, None)


def test_linear_backward_refusals():
    assert _linear_bwd(N=0) == INVALID
    assert _linear_bwd(act=-1) == INVALID
    assert _linear_bwd(act=2) == INVALID                       # an activation without pre
    assert _linear_bwd(dout_dtype=5) == INVALID
    assert _linear_bwd(dW_dtype=5) == INVALID
    assert _linear_bwd(dout=0) == INVALID
    assert _linear_bwd(W=None) == INVALID                      # dx without W
    assert _linear_bwd(x=None) == INVALID                      # dW without x
    assert _linear_bwd(dx=None, dW=None, dbias=None) == INVALID
    assert _linear_bwd(dW=0x5004) == INVALID
    assert _linear_bwd(ws=None) == WORKSPACE
    assert _linear_bwd(n=moe.linear_backward_workspace_size(16, 64, 32) - 1) == WORKSPACE


def test_binding_refuses_host_tensors_and_missing_pieces():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    W = torch.zeros(64, 8, dtype=torch.bfloat16)
    z = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        moe.linear(x, W)
    with pytest.raises(TypeError):
        moe.linear_backward(z, x, W)
    with pytest.raises(TypeError):
        moe.route_scored(z, 2)
    with pytest.raises(TypeError):
        moe.route_scored_backward(z, z, z)
    with pytest.raises(TypeError):
        moe.combine_backward(x, x, z, z)
    with pytest.raises(ValueError):
        moe.Router().logits(x)
