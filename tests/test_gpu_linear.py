"""moe_linear and moe_linear_backward against plain 64-bit products, element by element
within bounds that count the roundings (router_ref): odd, ragged and small sizes, every
activation, type and optional tensor, repeatability, other streams, graphs."""
import numpy as np
import pytest
import torch

import router_ref as ref

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")

BF, F32 = torch.bfloat16, torch.float32


def _rand(seed, *shape, scale=1.0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def _np(t):
    return t.detach().cpu().double().numpy()


def _case(M, K, N, seed=0):
    return _rand(seed, M, K), _rand(seed + 1, K, N, scale=K ** -0.5)


def _check(got, want, bound, what):
    got = _np(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= bound + 1e-30)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} beyond the bound, worst " \
        f"{np.nanmax(np.abs(got - want) / (bound + 1e-30)):.2f} times it, first at {np.argwhere(bad)[0]}"


SIZES = [(1, 1, 1), (1, 64, 8), (1, 2048, 60), (2, 65, 7), (3, 256, 128), (7, 63, 200), (16, 1000, 256),
         (17, 512, 129), (33, 128, 64), (64, 64, 64), (65, 72, 24), (127, 200, 33), (128, 128, 256),
         (129, 320, 130), (200, 1408, 512), (257, 96, 264), (300, 777, 60), (513, 2048, 60)]


def _forward(M, K, N, act, out_dtype, bias, residual, pre, seed=0):
    x, W = _case(M, K, N, seed)
    b = _rand(seed + 2, N, dtype=F32) if bias else None
    r = _rand(seed + 3, M, N, dtype=out_dtype) if residual else None
    dev = [None if t is None else t.cuda() for t in (x, W, b, r)]
    got = moe.linear(dev[0], dev[1], bias=dev[2], residual=dev[3], act=act, out_dtype=out_dtype, pre=pre)
    step = ref.F32 if out_dtype is F32 else ref.BF16
    n = [None if t is None else _np(t) for t in (x, W, b, r)]
    out, u, bound, err = ref.linear(*n, act, step)
    what = f"{M}x{K}x{N} act {act} {out_dtype}"
    _check(got[0] if pre else got, out, bound, what)
    if pre:
        _check(got[1], u, err * (1 + ref.BF16) + ref.BF16 * np.abs(u), what + " pre")


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_linear_sizes(M, K, N, out_dtype):
    _forward(M, K, N, moe.ACT_NONE, out_dtype, bias=out_dtype is F32, residual=False, pre=False)


@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("M,K,N", [(1, 128, 96), (5, 72, 40), (130, 192, 136), (130, 65, 67), (260, 256, 512)])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_linear_epilogue(act, M, K, N, out_dtype):
    _forward(M, K, N, act, out_dtype, bias=True, residual=True, pre=True, seed=act)


@pytest.mark.parametrize("M", [2, 4, 8, 12, 24, 32, 48, 96, 160, 384])
def test_linear_small_batches(M):
    _forward(M, 4096, 264, moe.ACT_SILU, BF, bias=True, residual=False, pre=False, seed=M)


def test_linear_large_k_and_n():
    _forward(40, 14336, 96, moe.ACT_NONE, F32, True, False, False)
    _forward(300, 200, 2056, moe.ACT_GELU, BF, True, True, True)


def test_linear_in_place_residual_and_out():
    x, W = (t.cuda() for t in _case(70, 96, 72))
    r = _rand(9, 70, 72).cuda()
    want = moe.linear(x, W, residual=r)
    out = r.clone()
    got = moe.linear(x, W, residual=out, out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(got, want)


def test_linear_special_values_stay_in_their_rows():
    x, W = (t.cuda() for t in _case(140, 128, 80))
    want = moe.linear(x, W)
    x[3, 5], x[131, 0] = float("nan"), float("inf")
    got = moe.linear(x, W)
    rows = torch.ones(140, dtype=torch.bool, device="cuda")
    rows[[3, 131]] = False
    assert torch.equal(got[rows], want[rows])
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[131]).any()


@pytest.mark.parametrize("M,K,N", [(1, 2048, 60), (512, 4096, 128), (300, 777, 60), (130, 65, 67)])
def test_linear_writes_its_rows_only_and_repeats(M, K, N):
    x, W = (t.cuda() for t in _case(M, K, N))
    big = torch.full((M * N + 4096,), 7.0, device="cuda")
    out = big[2048:2048 + M * N].view(M, N)
    moe.linear(x, W, out=out, out_dtype=F32)
    first = out.clone()
    assert (big[:2048] == 7).all() and (big[2048 + M * N:] == 7).all()
    for _ in range(3):
        out.zero_()
        moe.linear(x, W, out=out, out_dtype=F32)
        assert torch.equal(out, first)


BWD = [(1, 1, 1), (1, 64, 8), (5, 72, 40), (64, 64, 64), (130, 65, 67), (129, 200, 60), (257, 96, 264),
       (300, 512, 128), (1001, 136, 72), (40, 1408, 520)]


def _backward(M, K, N, act, dout_dtype, dW_dtype, seed=0):
    x, W = _case(M, K, N, seed)
    dout = _rand(seed + 5, M, N, dtype=dout_dtype)
    pre = _rand(seed + 6, M, N, scale=2.0) if act else None
    dx, dW, db = moe.linear_backward(dout.cuda(), x.cuda(), W.cuda(), pre=None if pre is None else pre.cuda(),
                                     act=act, dW_dtype=dW_dtype, want_dbias=True)
    exact = dout_dtype is BF and not act
    # the bf16 terms of du: all of it, 24 bits of it, or at the least one rounding to bf16
    step = 0.0 if exact else ref.F32 if dW_dtype is F32 else ref.BF16
    r = ref.linear_backward(_np(dout), _np(x), _np(W), None if pre is None else _np(pre), act, step)
    what = f"{M}x{K}x{N} act {act} {dout_dtype} {dW_dtype}"
    _check(dW, r["dW"], r["bW"] + (ref.F32 if dW_dtype is F32 else ref.BF16) * (np.abs(r["dW"]) + r["bW"]), what + " dW")
    _check(db, r["dbias"], r["bb"] * 1.01 + ref.F32 * np.abs(r["dbias"]), what + " dbias")
    step = 0.0 if exact else ref.BF16
    r = ref.linear_backward(_np(dout), _np(x), _np(W), None if pre is None else _np(pre), act, step)
    _check(dx, r["dx"], r["bx"] + ref.BF16 * (np.abs(r["dx"]) + r["bx"]), what + " dx")


@pytest.mark.parametrize("M,K,N", BWD)
@pytest.mark.parametrize("dout_dtype,dW_dtype", [(F32, F32), (BF, BF), (BF, F32), (F32, BF)])
def test_linear_backward_sizes(M, K, N, dout_dtype, dW_dtype):
    _backward(M, K, N, moe.ACT_NONE, dout_dtype, dW_dtype)


@pytest.mark.parametrize("act", [1, 2, 3])
@pytest.mark.parametrize("M,K,N", [(3, 64, 40), (130, 65, 67), (300, 264, 280)])
@pytest.mark.parametrize("dW_dtype", [BF, F32])
def test_linear_backward_activations(act, M, K, N, dW_dtype):
    _backward(M, K, N, act, BF, dW_dtype, seed=act)


def test_linear_backward_optional_outputs_and_repeats():
    M, K, N = 200, 136, 72
    x, W = (t.cuda() for t in _case(M, K, N))
    dout = _rand(5, M, N, dtype=F32).cuda()
    dx, dW, db = moe.linear_backward(dout, x, W, want_dbias=True)
    for want in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0)):
        got = moe.linear_backward(dout, x, W, want_dx=bool(want[0]), want_dW=bool(want[1]), want_dbias=bool(want[2]))
        for w, g, full in zip(want, got, (dx, dW, db)):
            assert (g is None) == (not w)
            assert not w or torch.equal(g, full)


def test_linear_gradients_against_differences():
    """The directional derivative of sum(dout * linear(x, W + t V)) along V by a central
    difference in 64 bits on the reference, against the kernels' dW: |<dW, V>| up to the
    kernels' own bound."""
    M, K, N = 37, 72, 40
    x, W = _case(M, K, N)
    dout, V = _rand(5, M, N, dtype=F32), _rand(6, K, N, dtype=F32)
    u = moe.linear(x.cuda(), W.cuda(), act=moe.ACT_SILU, out_dtype=F32, pre=True)[1]
    _, dW, _ = moe.linear_backward(dout.cuda(), x.cuda(), W.cuda(), pre=u, act=moe.ACT_SILU)
    f = lambda t: (_np(dout) * ref.act(2, _np(x) @ (_np(W) + t * _np(V)))).sum()  # noqa: E731
    diff = (f(1e-5) - f(-1e-5)) / 2e-5
    # pre is rounded to bf16: |silu''| <= 0.5, so du moves by at most 2^-8 |u| |dout| / 2
    moved = ref.BF16 * 0.5 * np.abs(_np(dout)) * np.abs(_np(x) @ _np(W))
    bound = (np.abs(_np(x) @ _np(V)) * moved).sum() + 1e-4 * (np.abs(_np(dW) * _np(V))).sum()
    assert abs((_np(dW) * _np(V)).sum() - diff) <= bound


def test_linear_on_another_stream_and_two_at_once():
    x, W = (t.cuda() for t in _case(300, 777, 60))
    dout = _rand(5, 300, 60, dtype=F32).cuda()
    want = moe.linear(x, W, out_dtype=F32)
    wx, wW, _ = moe.linear_backward(dout, x, W)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        got.append((moe.linear(x, W, out_dtype=F32, stream=s), *moe.linear_backward(dout, x, W, stream=s)[:2]))
    for s in streams:
        s.synchronize()
    for a, b, c in got:
        assert torch.equal(a, want) and torch.equal(b, wx) and torch.equal(c, wW)


def test_linear_in_a_graph():
    M, K, N = 130, 65, 67
    x, W = (t.cuda() for t in _case(M, K, N))
    pre = _rand(4, M, N).cuda()
    dout = _rand(5, M, N).cuda()
    out = torch.empty(M, N, dtype=BF, device="cuda")
    ws = torch.empty(moe.linear_workspace_size(M, K, N) + 16, dtype=torch.uint8, device="cuda")
    step = lambda: (moe.linear(x, W, act=2, out=out, ws=ws),) + moe.linear_backward(dout, x, W, pre=pre, act=2)[:2]  # noqa: E731
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in (11, 12):
        x.copy_(_rand(seed, M, K))
        dout.copy_(_rand(seed + 1, M, N))
        g.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(kept, step()))


def test_linear_refuses_wrong_tensors():
    x, W = (t.cuda() for t in _case(8, 64, 16))
    with pytest.raises(ValueError):
        moe.linear(x, W.t())                           # not contiguous
    with pytest.raises(ValueError):
        moe.linear(x, W[:32])
    with pytest.raises(ValueError):
        moe.linear(x[0], W)
    with pytest.raises(TypeError):
        moe.linear(x, W, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        moe.linear(x.float(), W)
    with pytest.raises(ValueError):
        moe.linear(x, W, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(TypeError):
        moe.linear(x, W, residual=torch.zeros(8, 16, device="cuda"))     # not out_dtype
    with pytest.raises(ValueError):
        moe.linear_backward(torch.zeros(8, 16, device="cuda"), x, W, act=moe.ACT_SILU)
    with pytest.raises(ValueError):
        moe.linear_backward(torch.zeros(8, 15, device="cuda"), x, W)
    with pytest.raises(moe.MoEError) as e:
        moe.linear(x[:0], W)
    assert e.value.code == moe.MOE_ERR_INVALID
