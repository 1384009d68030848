"""SiLU, GELU and their derivatives to the last bits of fp32, over the arguments where the
results are normal numbers: u goes in exactly, as one bf16 product.

In steps of 2^-24 of the value.  SiLU: expf 4 (2 units in the last place, in the numerator and
the denominator), the sum 1, the division 4, two products 2: below 16.  GELU: erfcf 8 (4 units),
its argument's 1.3 steps move it by (u^2 + 1) times as much, two products 2.  SiLU's derivative
p (1 + u q): p and q 11 each, and the products and the sum. GELU's: both terms, which cancel."""
import pytest
import torch

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")

BF, F32 = torch.bfloat16, torch.float32
STEP = 2.0 ** -24


def _args(act, n):
    lo, hi = (-85.0, 85.0) if act == moe.ACT_SILU else (-12.5, 30.0)
    return torch.cat([torch.linspace(lo, hi, n // 2), torch.linspace(-6, 6, n - n // 2)]).to(BF).cuda()


def _parts(act, u):
    if act == moe.ACT_SILU:
        p, q = torch.sigmoid(u), torch.sigmoid(-u)
        return u * p, 16 * (u * p).abs(), p * (1 + u * q), 30 * p * (1 + u.abs() * q)
    P, f = 0.5 * torch.special.erfc(u * -(0.5 ** 0.5)), torch.exp(-0.5 * u * u) * (2 * torch.pi) ** -0.5
    steps = 12 + 1.5 * u * u
    return u * P, steps * (u * P).abs(), P + u * f, (steps + 2) * P + 10 * u.abs() * f


# without the tensor cores, one tile, and a long sum (its other products are 0)
@pytest.mark.parametrize("M,K,N", [(1, 1, 1000), (16, 3, 1001), (300, 8, 520), (130, 4096, 64)])
@pytest.mark.parametrize("act", [moe.ACT_SILU, moe.ACT_GELU])
def test_activations(M, K, N, act):
    u = _args(act, N)
    x, W = torch.zeros(M, K, dtype=BF, device="cuda"), torch.zeros(K, N, dtype=BF, device="cuda")
    x[:, 0], W[0] = 1, u
    got = moe.linear(x, W, act=act, out_dtype=F32).double()
    want, steps, _, _ = _parts(act, u.double())
    off = (got - want).abs()
    assert (off <= STEP * steps).all(), float((off / (STEP * steps + 1e-300)).max())
    # bf16: its rounding, the fast exponential's steps (of |u| and of u^2 / 2, twice that with the
    # argument's own rounding) and GELU's polynomial, 3.1e-7 = 5.2 steps and 8 roundings
    got = moe.linear(x, W, act=act).double()
    more = STEP * (steps + 2 * u.double().abs() * want.abs())
    if act == moe.ACT_GELU:
        more = STEP * (16 + 2 * u.double() ** 2) * want.abs()
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 1.01 * more).all()


@pytest.mark.parametrize("N", [2000, 1001])
@pytest.mark.parametrize("act", [moe.ACT_SILU, moe.ACT_GELU])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_derivatives(N, act, dtype):
    u = _args(act, N)
    g = torch.Generator(device="cuda").manual_seed(N)
    dout = torch.randn(1, N, generator=g, device="cuda").to(dtype)
    x, W = torch.ones(1, 8, dtype=BF, device="cuda"), torch.zeros(8, N, dtype=BF, device="cuda")
    _, dW, db = moe.linear_backward(dout, x, W, pre=u[None], act=act, want_dbias=True)
    _, _, d, steps = _parts(act, u.double())
    want = dout[0].double() * d
    bound = STEP * dout[0].double().abs() * (steps + d.abs())
    assert ((db.double() - want).abs() <= 1.01 * bound).all()
    # dW takes du as three bf16 terms (2^-24 left), whose products are summed in fp32; bf16's
    # subnormals are 2^-133 apart, so the last term of a du below 2^-110 is off by up to half of that
    assert ((dW.double() - want).abs() <= 1.01 * bound + 5 * STEP * want.abs() + 2.0 ** -134).all()
