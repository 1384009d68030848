"""Tensors of more than 2^31 elements: offsets beyond 32 bits in the linear layer, the scored
router and the combine's gradient, checked on rows at both ends and between."""
import pytest
import torch

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")

BF16, F32 = 2.0 ** -8, 2.0 ** -24


def _rows(n):
    return torch.tensor([0, 1, n // 3, n // 2, n - 129, n - 2, n - 1], device="cuda")


def test_linear():
    M, K, N = 70001, 64, 32768
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    W = torch.randn(K, N, generator=g, device="cuda").bfloat16()
    out = moe.linear(x, W)
    r = _rows(M)
    want = x[r].double() @ W.double()
    # 4 truncated additions of the accumulator and the last rounding
    bound = 6 * 2.0 ** -23 * (x[r].double().abs() @ W.double().abs()) + BF16 * want.abs()
    assert ((out[r].double() - want).abs() <= bound).all()


def test_route_scored_and_its_gradient():
    T, E, k = 9_000_001, 256, 4
    z = torch.empty(T, E, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(0, T, 1_000_000):
        z[i:i + 1_000_000].normal_(generator=g)
    idx, gate = moe.route_scored(z, k, score=moe.SCORE_SIGMOID, scale=1.5)
    r = _rows(T)
    top = torch.sort(z[r], dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(idx[r].long(), top)
    p = torch.sigmoid(z[r].double()).gather(1, top)
    want = 1.5 * p / p.sum(1, keepdim=True)
    assert ((gate[r].double() - want).abs() <= 4 * F32 * want).all()
    dz = moe.route_scored_backward(gate, z, idx, score=moe.SCORE_SIGMOID, renorm=False)
    want = torch.zeros(len(r), E, dtype=torch.float64, device="cuda").scatter_(1, top, gate[r].double() * p * (1 - p))
    assert ((dz[r].double() - want).abs() <= 8 * F32 * want.abs()).all()


def test_combine_backward():
    T, k, d = 140_001, 2, 8192
    g = torch.Generator(device="cuda").manual_seed(2)
    dout = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    y = torch.empty(T * k, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    row_of = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
    gate = torch.rand(T, k, generator=g, device="cuda")
    dy, dgate = moe.combine_backward(dout, y, row_of, gate)
    for t in _rows(T).tolist():
        for j in range(k):
            row = int(row_of[t * k + j])
            prod = dout[t].double() * y[row].double()
            assert abs(float(dgate[t, j]) - float(prod.sum())) <= d * F32 * float(prod.abs().sum())
            want = gate[t, j].double() * dout[t].double()
            assert ((dy[row].double() - want).abs() <= (BF16 + 2 * F32) * want.abs()).all()
