"""NaN and infinities in the linear layer: they show in the rows that hold them, through every
activation, and change no other row."""
import pytest
import torch

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")

BF, F32 = torch.bfloat16, torch.float32


# few rows (without the tensor cores), one tile, long sums, several tiles, rows that are no 16-byte multiples
@pytest.mark.parametrize("M,K,N", [(3, 128, 80), (3, 65, 77), (140, 128, 80), (140, 4096, 64), (300, 1000, 520), (200, 65, 67)])
@pytest.mark.parametrize("act", [moe.ACT_NONE, moe.ACT_RELU, moe.ACT_SILU, moe.ACT_GELU])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_nan_is_seen_through_every_activation(M, K, N, act, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF)
    W = (torch.randn(K, N, generator=g, device="cuda") * K ** -0.5).to(BF)
    b = torch.randn(N, generator=g, device="cuda")
    r = torch.randn(M, N, generator=g, device="cuda").to(dtype)
    for kw in (dict(), dict(bias=b, residual=r)):
        want, u = moe.linear(x, W, act=act, out_dtype=dtype, pre=True, **kw)
        y = x.clone()
        y[1, 5], y[M - 1, 0] = float("nan"), float("inf")
        got, v = moe.linear(y, W, act=act, out_dtype=dtype, pre=True, **kw)
        assert torch.isnan(got[1]).all() and torch.isnan(v[1]).all()
        assert torch.equal(got[2:M - 1], want[2:M - 1]) and torch.equal(got[0], want[0]) and torch.equal(v[2:M - 1], u[2:M - 1])
        assert not torch.isfinite(v[M - 1]).any()
        up = v[M - 1] == float("inf")
        assert (got[M - 1][up] == float("inf")).all()       # every activation keeps +infinity
        if act == moe.ACT_RELU:                             # and this one makes 0 of -infinity
            rest = torch.zeros(N, device="cuda", dtype=dtype) if not kw else r[M - 1]
            down = v[M - 1] == float("-inf")
            assert torch.equal(got[M - 1][down], rest[down])
    # a NaN in the bias: its column
    b[3] = float("nan")
    got = moe.linear(x, W, bias=b, act=act, out_dtype=dtype)
    assert torch.isnan(got[:, 3]).all() and not torch.isnan(got[:, 4:]).any()
