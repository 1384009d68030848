"""moe_linear and moe_linear_backward at sizes that take every way through the product:
pairs of blocks, several tiles to a block, reductions split over a cluster or cut into
slices, the lower terms of fp32 gradients; against 64-bit products on the device, element
by element, and in the 2-norm where sums are long."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")

BF, F32 = torch.bfloat16, torch.float32
STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _rand(g, *shape, scale=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _act(kind, u):
    return (u, u.clamp(min=0), u * torch.sigmoid(u), u * torch.special.ndtr(u))[kind]


def _dact(kind, u):
    s = torch.sigmoid(u)
    return (torch.ones_like(u), (u > 0).double(), s * (1 + u * (1 - s)),
            torch.special.ndtr(u) + u * torch.exp(-0.5 * u * u) * (2 * torch.pi) ** -0.5)[kind]


def _within(got, want, bound, what):
    off = (got.double() - want).abs() - bound
    assert not (off > 1e-30).any() and torch.isfinite(got.float()).all(), f"{what}: {int((off > 1e-30).sum())} of {off.numel()}"


# An fp32 output leaves the accumulator every 512 of k: 32 additions of 16 products, each
# truncated by a step (2^-23) of a partial sum that is at most sum|a b|, and then K / 512
# additions rounded to nearest.  A bf16 output is one chain of K / 16.
def _sum_error(K, dtype, size):
    chains = 32 * 2.0 ** -23 + (K // 512 + 2) * 2.0 ** -24
    return (chains if dtype is F32 else (K // 16 + 2) * 2.0 ** -23) * size


SHAPES = [(129, 512, 256), (1024, 512, 1536), (2500, 1000, 776), (4100, 264, 4104), (777, 4104, 130),
          (300, 8192, 264), (3000, 72, 5000), (2048, 1408, 2048), (640, 2048, 31), (17, 4096, 4096), (1200, 130, 1030)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("dtype,act,extras", [(F32, 0, False), (BF, 2, True), (BF, 0, False), (F32, 3, True)])
def test_linear(M, K, N, dtype, act, extras):
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x, W = _rand(g, M, K), _rand(g, K, N, scale=K ** -0.5)
    b = _rand(g, N, dtype=F32) if extras else None
    r = _rand(g, M, N, dtype=dtype) if extras else None
    got = moe.linear(x, W, bias=b, residual=r, act=act, out_dtype=dtype, pre=extras)
    u = x.double() @ W.double()
    e = _sum_error(K, dtype, x.double().abs() @ W.double().abs())
    if extras:
        u = u + b.double()
        e = e + STEP[F32] * u.abs()
        _within(got[1], u, e * (1 + STEP[BF]) + STEP[BF] * u.abs(), "pre")
    # the activation's own roundings: 8 of values up to |u|; |act'| <= 1.13
    e = 1.13 * e + (8 * STEP[F32] * u.abs() if act else 0)
    want = _act(act, u)
    if extras:
        want = want + r.double()
        e = e + STEP[F32] * want.abs()
    _within(got[0] if extras else got, want, e * (1 + STEP[dtype]) + STEP[dtype] * want.abs(), "out")
    assert moe.linear_get_status() == moe.MOE_OK


@pytest.mark.parametrize("M,K,N", [(4096, 8192, 128), (256, 16384, 200), (700, 8200, 60)])
def test_long_sums_keep_32_bits(M, K, N):
    """2-norm: a chain of 32 truncated additions is off by half a step of the partial sums on
    average, which are two thirds of the chain's end in the mean: 32 * 2^-24 * 2/3 = 1.3e-6 of
    the chain's norm at the most.  One chain over all of K would be off by K / 512 times that."""
    g = torch.Generator(device="cuda").manual_seed(K)
    x, W = _rand(g, M, K), _rand(g, K, N, scale=K ** -0.5)
    want = x.double() @ W.double()
    got = moe.linear(x, W, out_dtype=F32).double()
    assert (got - want).norm() <= 1.4e-6 * want.norm()
    dout = _rand(g, K, N, dtype=F32)                    # K tokens: the sums of the weight's gradient
    xt = _rand(g, K, 264)
    dW = moe.linear_backward(dout, xt, _rand(g, 264, N), want_dx=False)[1].double()
    want = xt.double().t() @ dout.double()
    assert (dW - want).norm() <= 1.4e-6 * want.norm()


BACKWARD = [(16384, 512, 128), (8192, 1024, 264), (5000, 776, 1000), (600, 2048, 1408), (3000, 4096, 60),
            (2111, 130, 257), (40000, 64, 8)]


@pytest.mark.parametrize("M,K,N", BACKWARD)
@pytest.mark.parametrize("dout_dtype,dW_dtype,act", [(F32, F32, 0), (BF, BF, 2), (BF, F32, 3), (BF, BF, 0)])
def test_linear_backward(M, K, N, dout_dtype, dW_dtype, act):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    x, W, dout = _rand(g, M, K), _rand(g, K, N), _rand(g, M, N, dtype=dout_dtype)
    pre = _rand(g, M, N, scale=2.0) if act else None
    dx, dW, db = moe.linear_backward(dout, x, W, pre=pre, act=act, dW_dtype=dW_dtype, want_dbias=True)
    du = dout.double() * (_dact(act, pre.double()) if act else 1.0)
    exact = dout_dtype is BF and not act
    # act' in fp32: 10 roundings of values up to 1.13 (1 + |pre|)
    own = 12 * STEP[F32] * dout.double().abs() * (1 + pre.double().abs()) if act else torch.zeros_like(du)
    e = own + (0 if exact else STEP[BF]) * du.abs()     # one bf16 term
    size = du.abs() @ W.double().abs().t()
    want = du @ W.double().t()
    b = e @ W.double().abs().t() + _sum_error(N, BF, size)
    _within(dx, want, b + STEP[BF] * (want.abs() + b), "dx")
    e = own + (0 if exact else STEP[dW_dtype]) * du.abs()    # three terms leave 2^-24
    size = x.double().abs().t() @ du.abs()
    want = x.double().t() @ du
    b = x.double().abs().t() @ e + _sum_error(M, dW_dtype, size)
    _within(dW, want, b + STEP[dW_dtype] * (want.abs() + b), "dW")
    # a column's sum: at most M / 16 additions in a thread, then a few dozen
    _within(db, du.sum(0), own.sum(0) + (M // 16 + 64) * STEP[F32] * du.abs().sum(0), "dbias")
    again = moe.linear_backward(dout, x, W, pre=pre, act=act, dW_dtype=dW_dtype, want_dbias=True)
    assert all(torch.equal(p, q) for p, q in zip((dx, dW, db), again))
    assert moe.linear_get_status() == moe.MOE_OK


def test_two_streams_at_once():
    """Products, and the slices of their reductions, on two streams, each with a workspace of its own."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, W, dout = _rand(g, 8192, 1024), _rand(g, 1024, 264), _rand(g, 8192, 264)
    want = moe.linear(x, W), *moe.linear_backward(dout, x, W)[:2]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[] for _ in streams]
    for _ in range(4):
        for s, to in zip(streams, got):
            to.append((moe.linear(x, W, stream=s), *moe.linear_backward(dout, x, W, stream=s)[:2]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for to in got for r in to for a, b in zip(r, want))


def test_two_graphs_share_a_workspace():
    g = torch.Generator(device="cuda").manual_seed(2)
    x, W, dout = _rand(g, 4096, 777), _rand(g, 777, 60), _rand(g, 4096, 60, dtype=F32)
    ws = torch.empty(moe.linear_backward_workspace_size(4096, 777, 60), dtype=torch.uint8, device="cuda")
    f = lambda d: moe.linear_backward(d, x, W, ws=ws)[:2]  # noqa: E731
    other = -2 * dout
    want = [[t.clone() for t in f(d)] for d in (dout, other)]
    graphs, outs = [], []
    for d in (dout, other):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(f(d))
        graphs.append(gr)
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o, w in zip(outs, want) for a, b in zip(o, w))


def test_first_call_inside_a_capture():
    """Nothing that a first call sets up needs to happen outside a capture."""
    code = """
import torch
from combine_overlap_b200 import moe
x = torch.randn(300, 256, device="cuda").bfloat16(); W = torch.randn(256, 520, device="cuda").bfloat16()
d = torch.randn(300, 520, device="cuda"); z = torch.randn(300, 64, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a = moe.linear(x, W); b = moe.linear_backward(d, x, W)[:2]; c = moe.route_scored(z, 6)
g.replay(); torch.cuda.synchronize()
e = (moe.linear(x, W), *moe.linear_backward(d, x, W)[:2], *moe.route_scored(z, 6))
assert all(torch.equal(p, q) for p, q in zip((a, *b, *c), e))
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
