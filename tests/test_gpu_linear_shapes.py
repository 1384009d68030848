"""The linear layer's product in every tile and split that it may choose: single blocks and
pairs, each tile width, reductions over clusters of 2, 4 and 8 and in slices, with all of the
epilogue, in both output types, at ragged sizes; against 64-bit products on the device."""
import pytest
import torch

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")

BF, F32 = torch.bfloat16, torch.float32
STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}
WIDTHS = [16] + list(range(32, 257, 32))
TILES = [(cg, s) for cg in (1, 2) for s in (1, 2, 4, 8) if cg * s <= 8]


def _rand(g, *shape, scale=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _within(got, want, bound, what):
    off = (got.double() - want).abs() - bound
    assert not (off > 1e-30).any() and torch.isfinite(got.float()).all(), f"{what}: {int((off > 1e-30).sum())} of {off.numel()}"


def _sum_error(K, dtype, size):
    """fp32: chains of 32 truncated additions (2^-23 each) and K / 512 + 8 rounded ones (the
    chains', the splits'); bf16: one chain of K / 16."""
    chains = 32 * 2.0 ** -23 + (K // 512 + 10) * 2.0 ** -24
    return (chains if dtype is F32 else (K // 16 + 8) * 2.0 ** -23) * size


def _tried(f):
    """f's result, or None where the size is never cut that way."""
    try:
        return f()
    except moe.MoEError as e:
        assert e.code == moe.MOE_ERR_UNSUPPORTED
        return None


# rows of 16-byte multiples and not; 33 blocks of 64 in K, the last one partly there; N for each width's edges;
# bf16 sums of more than one chain
@pytest.mark.parametrize("M,K,N", [(333, 2088, 520), (141, 2053, 267), (300, 2048, 12), (141, 16523, 267)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", [0, 2])
def test_forward(M, K, N, dtype, act):
    g = torch.Generator(device="cuda").manual_seed(M)
    x, W = _rand(g, M, K), _rand(g, K, N, scale=K ** -0.5)
    b, r = _rand(g, N, dtype=F32), _rand(g, M, N, dtype=dtype)
    u = x.double() @ W.double() + b.double()
    e = _sum_error(K, dtype, x.double().abs() @ W.double().abs()) + STEP[F32] * u.abs()
    h = u * torch.sigmoid(u) if act else u
    want = h + r.double()
    # the activation's own roundings: 8 of values up to |u|; |act'| <= 1.1
    eo = (1.1 * e + 8 * STEP[F32] * u.abs() if act else e) + STEP[F32] * want.abs()
    ran = set()
    for cg, s in TILES:
        for bn in WIDTHS:
            with moe.linear_debug(cg, bn, s):
                got = _tried(lambda: moe.linear(x, W, bias=b, residual=r, act=act, out_dtype=dtype, pre=True))
            if got is None:
                continue
            ran.add((cg, s, bn))
            what = f"pair {cg} width {bn} split {s}"
            _within(got[0], want, eo * (1 + STEP[dtype]) + STEP[dtype] * want.abs(), what)
            _within(got[1], u, e * (1 + STEP[BF]) + STEP[BF] * u.abs(), what + " pre")
            with moe.linear_debug(cg, bn, s):     # without the epilogue's reads, and equal bits again
                plain = moe.linear(x, W, out_dtype=dtype)
                assert torch.equal(moe.linear(x, W, out_dtype=dtype), plain)
            v = u - b.double()
            _within(plain, v, e * (1 + STEP[dtype]) + STEP[dtype] * v.abs(), what + " plain")
    assert moe.linear_get_status() == moe.MOE_OK
    if N > 256:                                   # every one of them, where the tiles fit
        assert {(cg, s) for cg, s, _ in ran} == set(TILES)
        assert {(1, 1, b) for b in WIDTHS[1:]} | {(2, 1, b) for b in WIDTHS[1:]} | {(2, 2, 160), (2, 2, 192), (2, 2, 224)} <= ran
    else:
        assert {(1, s, 16) for s in (1, 2, 4, 8)} <= ran


# (tokens, K, N): dx reduces N, dW the tokens
@pytest.mark.parametrize("M,K,N", [(2088, 264, 333), (2051, 133, 520), (333, 264, 2088), (141, 267, 2053),
                                   (16523, 133, 267), (141, 267, 16523)])
@pytest.mark.parametrize("dout_dtype,dW_dtype", [(BF, BF), (F32, F32), (F32, BF)])
def test_gradients(M, K, N, dout_dtype, dW_dtype):
    g = torch.Generator(device="cuda").manual_seed(N)
    x, W, dout = _rand(g, M, K), _rand(g, K, N), _rand(g, M, N, dtype=dout_dtype)
    du = dout.double()
    exact = dout_dtype is BF
    want_x, size = du @ W.double().t(), du.abs() @ W.double().abs().t()
    bx = (0 if exact else STEP[BF]) * size + _sum_error(N, BF, size)
    want_W, size = x.double().t() @ du, x.double().abs().t() @ du.abs()
    bW = (0 if exact else STEP[dW_dtype]) * size + _sum_error(M, dW_dtype, size)
    db = du.sum(0)
    ran = set()
    for cg, s in TILES:
        for bn in WIDTHS[1:]:
            with moe.linear_debug(cg, bn, s):
                a = _tried(lambda: moe.linear_backward(dout, x, W, want_dW=False)[0])
            if a is not None:
                ran.add(("dx", cg, s, bn))
                _within(a, want_x, bx + STEP[BF] * (want_x.abs() + bx), f"dx pair {cg} width {bn} split {s}")
            for sw in (1, 2, 5, 8) if s == 1 else (1,):
                with moe.linear_debug(cg, bn, s, sw):
                    a = _tried(lambda: moe.linear_backward(dout, x, W, dW_dtype=dW_dtype, want_dx=False, want_dbias=True)[1:])
                if a is not None:
                    ran.add(("dW", cg, s * 100 + sw, bn))
                    what = f"dW pair {cg} width {bn} split {s} slices {sw}"
                    _within(a[0], want_W, bW + STEP[dW_dtype] * (want_W.abs() + bW), what)
                    # at most M / 16 additions in a thread, then a few dozen
                    _within(a[1], db, (M // 16 + 64) * STEP[F32] * du.abs().sum(0), what + " dbias")
    assert moe.linear_get_status() == moe.MOE_OK
    if M > 2000:
        assert {(cg, sw) for k, cg, sw, _ in ran if k == "dW"} >= {(1, 101), (1, 108), (2, 105), (1, 801), (2, 201), (2, 401)}
    else:
        assert {(cg, s) for k, cg, s, _ in ran if k == "dx"} == set(TILES)


def test_shapes_that_no_product_has_are_refused():
    x, W = torch.zeros(100, 512, dtype=BF, device="cuda"), torch.zeros(512, 64, dtype=BF, device="cuda")
    for kw in (dict(cg=2, bn=64), dict(cg=1, bn=96), dict(cg=1, bn=48), dict(cg=1, bn=16), dict(cg=1, bn=64, s=3),
               dict(cg=1, bn=64, s=4), dict(cg=1, bn=64, sw=2), dict(cg=3, bn=64), dict(cg=1, bn=512)):
        with moe.linear_debug(**kw):
            assert _tried(lambda: moe.linear(x, W)) is None, kw
    with pytest.raises(moe.MoEError):
        with moe.linear_debug(cg=1, bn=0):
            pass
    assert moe.linear(x, W).shape == (100, 64)    # and the library's own choice is back
