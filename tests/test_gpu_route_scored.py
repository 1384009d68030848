"""The scored router and its gradient against plain 64-bit references: ids bit for bit,
gates within their rounding; ties, masked experts and rows, groups, extremes; and the
gradient of the combine."""
import numpy as np
import pytest
import torch

import router_ref as ref
from combine_overlap_b200 import synth

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")


def _logits(T, E, seed=0, ties=True, masked=True):
    rng = np.random.default_rng(seed)
    z = rng.normal(size=(T, E)).astype(np.float32) * 2
    if ties:
        z[::3] = np.round(z[::3] * 4) / 4
        if T > 5:
            z[5] = 1.5
    if masked:
        z[rng.random((T, E)) < 0.05] = -np.inf
        z[rng.random((T, E)) < 0.02] = np.nan
        if T > 2:
            z[2] = -np.inf
        if T > 8:
            z[8, 1:] = -np.inf                       # one expert left
    return z


def _gate_bound(E):
    # Z sums E exponentials in fp32 at the worst (E + 8 roundings), the gate is one more
    return (E + 10) * ref.F32


def _check(z, k, kind=0, bias=None, G=1, kg=0, top2=False, renorm=True, scale=1.0):
    T, E = z.shape
    b = None if bias is None else torch.from_numpy(bias).cuda()
    ws = moe.alloc_workspace(T, 256, 128, E, k)
    idx, gate, cnt = moe.route_scored(torch.from_numpy(z).cuda(), k, score=kind, bias=b, n_groups=G, topk_groups=kg,
                                      group_score=int(top2), renorm=renorm, scale=scale, counts=True, ws=ws)
    widx, wgate = ref.route(z, k, kind, bias, G, kg, top2, renorm, scale)
    idx, gate = idx.cpu().numpy(), gate.cpu().numpy()
    bad = np.argwhere((idx != widx).any(1))
    assert not len(bad), (bad[0], idx[bad[0, 0]], widx[bad[0, 0]])
    assert np.all(np.abs(gate - wgate) <= _gate_bound(E) * np.abs(wgate) + 1e-38), np.abs(gate - wgate).max()
    assert np.array_equal(cnt.cpu().numpy(), np.bincount(widx.reshape(-1), minlength=E))
    return idx


SHAPES = [(1, 1, 1), (1, 8, 2), (7, 64, 6), (33, 5, 5), (100, 60, 4), (130, 128, 8), (65, 33, 3), (40, 256, 8),
          (50, 255, 7), (64, 32, 1), (31, 8, 8), (1000, 16, 2)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("biased", [False, True])
def test_route_scored_shapes(T, E, k, kind, biased):
    bias = np.random.default_rng(E).normal(size=E).astype(np.float32) * 0.1 if biased else None
    z = _logits(T, E, T + E)
    _check(z, k, kind, bias, renorm=True, scale=2.5)
    _check(z, k, kind, bias, renorm=False)


@pytest.mark.parametrize("E,G,kg,k", [(8, 2, 1, 4), (8, 8, 3, 3), (64, 8, 4, 6), (256, 8, 4, 8), (60, 4, 2, 5),
                                      (96, 32, 5, 8), (33, 11, 10, 8), (64, 2, 2, 3), (128, 4, 1, 8)])
@pytest.mark.parametrize("top2", [False, True])
@pytest.mark.parametrize("kind,biased", [(0, False), (0, True), (1, False), (1, True)])
def test_route_scored_groups(E, G, kg, k, top2, kind, biased):
    bias = np.random.default_rng(E + G).normal(size=E).astype(np.float32) * 0.2 if biased else None
    _check(_logits(150, E, E + G), k, kind, bias, G, kg, top2, renorm=True, scale=1.5)


@pytest.mark.parametrize("kind", [0, 1])
def test_route_scored_extremes(kind):
    big = float(np.finfo(np.float32).max)
    z = np.array([[big, -big, 0, 1], [-big] * 4, [np.inf, 1, np.inf, 0], [-big, -np.inf, -big, -np.inf],
                  [100, 101, 102, 103], [-100, -101, -102, -103], [-800, -801, -900, -1000], [1e-30, 0, -1e-30, 0],
                  [88, 89, -88, -104]], np.float32)
    for renorm in (True, False):
        _check(z, 2, kind, None, renorm=renorm)
        _check(z, 3, kind, np.array([0.1, 0.1, 0.3, -0.2], np.float32), renorm=renorm)
        _check(z, 2, kind, None, 2, 1, True, renorm=renorm)


@pytest.mark.parametrize("kind", [0, 1])
def test_route_scored_close_keys(kind):
    """Keys that differ by less than fp32 can tell: the choice is the 64-bit one."""
    rng = np.random.default_rng(3)
    T, E = 400, 64
    z = (0.5 + 1e-7 * rng.integers(-8, 9, size=(T, E))).astype(np.float32)
    bias = (0.25 + 1e-8 * rng.integers(-8, 9, size=E)).astype(np.float32)
    _check(z, 6, kind, bias)
    _check(z, 6, kind, bias, 8, 3, True)
    _check(z, 6, kind, None, 8, 3, True)


def test_route_scored_equals_the_plain_router():
    """Renormalised softmax without bias or groups is moe_route's formula."""
    wl = synth.WORKLOADS["fine_grained"]
    logits = synth.make_logits(wl, "cuda")
    ws = moe.alloc_workspace(wl.T, 256, 128, wl.E, wl.k)
    a, b = moe.route(logits, wl.k, ws), moe.route_scored(logits, wl.k)
    assert torch.equal(a[0], b[0])
    assert ((a[1] - b[1]).abs() <= 2 * ref.F32 * a[1] * 1.01).all()


def test_route_scored_needs_no_workspace_and_repeats():
    z = torch.from_numpy(_logits(3000, 128, 1)).cuda()
    a = moe.route_scored(z, 8, score=1, n_groups=8, topk_groups=4, group_score=1)
    for _ in range(3):
        b = moe.route_scored(z, 8, score=1, n_groups=8, topk_groups=4, group_score=1)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(moe.MoEError) as e:
        moe.route_scored(z, 8, counts=True)
    assert e.value.code == moe.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_scored_backward(T, E, k, kind, renorm):
    z = _logits(T, E, T + E + 1)
    idx, _ = ref.route(z, k, kind)
    if T > 30:
        idx[20, 0] = -1                               # a dropped slot
        idx[21, k - 1] = E
    dg = np.random.default_rng(1).normal(size=(T, k)).astype(np.float32)
    out = torch.full((T + 2, E), 7.0, device="cuda")
    view = out[:T]
    moe.route_scored_backward(torch.from_numpy(dg).cuda(), torch.from_numpy(z).cuda(), torch.from_numpy(idx).cuda(),
                              score=kind, renorm=renorm, scale=1.5, dlogits=view)
    want, bound = ref.route_backward(dg, z, idx, kind, renorm, 1.5)
    got = view.cpu().double().numpy()
    assert np.all(np.abs(got - want) <= bound + 1e-37), np.abs(got - want).max()
    assert (out[T:] == 7).all()


@pytest.mark.parametrize("kind", [0, 1])
def test_route_scored_backward_extremes(kind):
    big = float(np.finfo(np.float32).max)
    z = np.array([[big, -big, 0, 1], [-np.inf] * 4, [-800, -801, -900, -1000], [100, 101, 102, 103]], np.float32)
    idx, _ = ref.route(z, 2, kind)
    dg = np.ones((4, 2), np.float32)
    dg[:, 1] = -2
    for renorm in (True, False):
        got = moe.route_scored_backward(torch.from_numpy(dg).cuda(), torch.from_numpy(z).cuda(),
                                        torch.from_numpy(idx).cuda(), score=kind, renorm=renorm)
        want, bound = ref.route_backward(dg, z, idx, kind, renorm)
        assert np.all(np.abs(got.cpu().double().numpy() - want) <= bound + 1e-37)


def _combine_case(T, d, k, dropped, seed=0):
    g = torch.Generator().manual_seed(seed)
    row_of = torch.randperm(T * k, generator=g).to(torch.int32)
    if dropped:
        row_of[torch.rand(T * k, generator=g) < 0.2] = -1
        row_of[0] = T * k                              # out of range: dropped as well
    dout, y = torch.randn(T, d, generator=g).bfloat16(), torch.randn(T * k, d, generator=g).bfloat16()
    return dout, y, row_of, torch.rand(T, k, generator=g)


@pytest.mark.parametrize("T,d,k", [(1, 8, 1), (1, 256, 2), (3, 1032, 8), (33, 512, 6), (9, 4096, 2), (70, 264, 3),
                                   (5, 8200, 5), (17, 2048, 4), (300, 64, 7)])
@pytest.mark.parametrize("dropped", [False, True])
def test_combine_backward(T, d, k, dropped):
    dout, y, row_of, gate = _combine_case(T, d, k, dropped, T + d)
    dy = torch.full((T * k, d), 3.0, dtype=torch.bfloat16, device="cuda")
    got, dgate = moe.combine_backward(dout.cuda(), y.cuda(), row_of.cuda(), gate.cuda(), dy=dy)
    n = [t.double().numpy() for t in (dout, y)]
    want, wgate, bound = ref.combine_backward(*n, row_of.numpy(), gate.double().numpy(), np.full((T * k, d), 3.0))
    assert np.all(np.abs(got.cpu().double().numpy() - want) <= (ref.BF16 + 2 * ref.F32) * np.abs(want))
    assert np.all(np.abs(dgate.cpu().double().numpy() - wgate) <= bound)
    none, again = moe.combine_backward(dout.cuda(), y.cuda(), row_of.cuda(), gate.cuda(), want_dy=False)
    assert none is None and torch.equal(again, dgate)


def test_refusals_of_the_binding():
    z = torch.zeros(4, 8, device="cuda")
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        moe.route_scored(z.t(), 2)
    with pytest.raises(ValueError):
        moe.route_scored(z, 2, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(TypeError):
        moe.route_scored(z, 2, bias=torch.zeros(8, device="cuda").double())
    with pytest.raises(moe.MoEError):
        moe.route_scored(z, 2, n_groups=3)
    with pytest.raises(ValueError):
        moe.route_scored_backward(torch.zeros(4, 3, device="cuda"), z, idx)
    with pytest.raises(TypeError):
        moe.route_scored_backward(torch.zeros(4, 2, device="cuda"), z, idx.long())
    y = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        moe.combine_backward(y, y, idx.view(-1), torch.zeros(4, 2, device="cuda"))
