"""dx of an fp32 gradient beside an fp32 dW: 16 bits of du, so that dx has the one rounding of its
own type.

Element by element: du is off by 2^-17 of itself (two bf16 terms), and by its own 12 fp32 roundings of
values up to |dout| (1 + |pre|) with an activation; the sum by 2^-23 of sum |du W| for each of its
2 N / 16 products' additions.  With one bf16 term it would be off by 2^-8 of sum |du W|."""
import pytest
import torch

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")

BF, F32 = torch.bfloat16, torch.float32


def _dsilu(u):
    s = torch.sigmoid(u)
    return s * (1 + u * (1 - s))


@pytest.mark.parametrize("M,K,N", [(1, 64, 8), (37, 264, 60), (300, 512, 64), (130, 65, 67), (1000, 4096, 128), (257, 1408, 200),
                                   (2048, 256, 1001), (129, 2048, 2056)])
@pytest.mark.parametrize("act,dtype", [(moe.ACT_NONE, F32), (moe.ACT_SILU, F32), (moe.ACT_SILU, BF)])
def test_dx_is_rounded_once(M, K, N, act, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF)
    W = torch.randn(K, N, generator=g, device="cuda").to(BF)
    dout = torch.randn(M, N, generator=g, device="cuda").to(dtype)
    pre = torch.randn(M, N, generator=g, device="cuda").mul(2).to(BF) if act else None
    dx, dW, _ = moe.linear_backward(dout, x, W, pre=pre, act=act)
    du = dout.double() * (_dsilu(pre.double()) if act else 1)
    e = 2.0 ** -17 * du.abs() + (12 * 2.0 ** -24 * dout.double().abs() * (1 + pre.double().abs()) if act else 0)
    want, size = du @ W.double().t(), du.abs() @ W.double().abs().t()
    bound = e @ W.double().abs().t() + (2 * N // 16 + 8) * 2.0 ** -23 * size
    assert ((dx.double() - want).abs() <= 2.0 ** -8 * (want.abs() + bound) + bound).all()
    # what else is wanted changes no bit
    full = moe.linear_backward(dout, x, W, pre=pre, act=act, want_dbias=True)
    assert torch.equal(full[0], dx) and torch.equal(full[1], dW)
    for i in range(3):
        some = moe.linear_backward(dout, x, W, pre=pre, act=act, want_dx=i == 0, want_dW=i == 1, want_dbias=i == 2)
        assert torch.equal(some[i], full[i])


def test_infinities_of_dout_stay_in_their_rows():
    g = torch.Generator(device="cuda").manual_seed(0)
    x, W = (torch.randn(*s, generator=g, device="cuda").to(BF) for s in ((200, 128), (128, 72)))
    dout = torch.randn(200, 72, generator=g, device="cuda")
    want = moe.linear_backward(dout, x, W)[0]
    dout[7, 3], dout[9, 0] = float("inf"), float("nan")
    got = moe.linear_backward(dout, x, W)[0]
    rows = torch.ones(200, dtype=torch.bool, device="cuda")
    rows[[7, 9]] = False
    assert torch.equal(got[rows], want[rows]) and (got[7].abs() == float("inf")).all() and got[9].isnan().all()
