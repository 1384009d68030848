"""Sums of one sign over 262144 products with bf16 outputs, whose truncation on the tensor
cores would add up to a bias: forward, dx and dW, at sizes that one block's tile reduces alone.

The mean of (got - want) / want over all outputs.  A run of 16384 products is 1024 additions,
each truncated by at most a step of the partial sum: 1024 * 2^-23 = 2^-13; the 16 runs are
added to nearest: 2^-20.  The outputs' own rounding to bf16 averages out: rows and columns have
factors between 1 and 2, so that its errors, at most 2^-8 and uniform, have a mean of about
2^-8 / sqrt(3 * 2048^2) = 1e-6 over these outputs, 1e-5 with room.  In one run of all products the
truncation would take up to 2^-9."""
import pytest
import torch

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")

BF = torch.bfloat16
LONG, SIDE = 262144, 2304


def _matrix(g, rows, cols, long_rows):
    """Values of (0.5, 1) times a factor of (1, 2) for each place on the short side."""
    t = torch.rand(rows, cols, generator=g, device="cuda").mul_(0.5).add_(0.5)
    f = 1 + torch.rand(1 if long_rows else rows, cols if long_rows else 1, generator=g, device="cuda")
    return t.mul_(f).to(BF)


@pytest.mark.parametrize("what", ["forward", "dx", "dW"])
def test_long_sums_of_one_sign(what):
    g = torch.Generator(device="cuda").manual_seed(3)
    if what == "dW":                       # more elements than the slices' workspace has room for
        a, b = _matrix(g, LONG, SIDE, True), _matrix(g, LONG, SIDE, True)
        W = torch.zeros(SIDE, SIDE, dtype=BF, device="cuda")
        got = moe.linear_backward(b, a, W, dW_dtype=BF, want_dx=False)[1]
    elif what == "dx":
        a, b = _matrix(g, SIDE, LONG, False), _matrix(g, SIDE, LONG, False)
        x = torch.zeros(SIDE, SIDE, dtype=BF, device="cuda")
        got = moe.linear_backward(a, x, b, want_dW=False)[0]
        a, b = a.t(), b.t()
    else:
        a, b = _matrix(g, SIDE, LONG, False), _matrix(g, LONG, SIDE, True)
        got = moe.linear(a, b)
        a = a.t()
    want = torch.zeros(SIDE, SIDE, dtype=torch.float64, device="cuda")
    for i in range(0, LONG, 16384):
        want += a[i:i + 16384].double().t() @ b[i:i + 16384].double()
    off = (got.double() - want) / want
    assert off.abs().max() <= 2.0 ** -8 * (1 + 2.0 ** -12) + 2.0 ** -13 + 2.0 ** -20
    assert abs(float(off.mean())) <= 2.0 ** -13 + 2.0 ** -20 + 1e-5, float(off.mean())
    assert moe.linear_get_status() == moe.MOE_OK
