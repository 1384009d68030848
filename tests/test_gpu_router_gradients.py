"""The router's and the combine's gradients against differences: directional derivatives of
the forward formulas in 64 bits along random directions."""
import numpy as np
import pytest
import torch

import router_ref as ref

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")


def _gates(z, idx, kind, renorm, scale):
    """The chosen experts' gates, the choice held fixed."""
    g = np.zeros(idx.shape)
    for t in range(len(z)):
        w = ref.scores(z[t], kind)[0][idx[t]]
        g[t] = scale * (w / w.sum() if renorm and w.sum() > 0 else w * (not renorm))
    return g


@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (40, 64, 6), (30, 256, 8), (25, 60, 1), (33, 100, 5)])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_scored_gradient(T, E, k, kind, renorm):
    rng = np.random.default_rng(T + E)
    z = rng.normal(size=(T, E)).astype(np.float32)
    if T > 10:
        z[3, : E // 2] = -np.inf
        z[7] = -np.inf
    dg = rng.normal(size=(T, k)).astype(np.float32)
    idx = moe.route_scored(torch.from_numpy(z).cuda(), k, score=kind, renorm=renorm, scale=1.5)[0]
    dz = moe.route_scored_backward(torch.from_numpy(dg).cuda(), torch.from_numpy(z).cuda(), idx, score=kind,
                                   renorm=renorm, scale=1.5).cpu().double().numpy()
    idx = idx.cpu().numpy()
    _, bound = ref.route_backward(dg, z, idx, kind, renorm, 1.5)
    for _ in range(4):
        V = rng.normal(size=(T, E))
        h = 1e-5
        f = lambda s: (dg.astype(np.float64) * _gates(z.astype(np.float64) + s * h * V, idx, kind, renorm, 1.5)).sum()  # noqa: E731
        diff = (f(1) - f(-1)) / (2 * h)
        # central difference: h^2 / 6 of a third derivative that is at most 10 |c| |V|^3 per
        # term, and the sums' own 64-bit rounding over 2 h
        size = 1.5 * np.abs(dg).sum()
        tol = (bound * np.abs(V)).sum() + size * (h * h * 2 * np.abs(V).max() ** 3 + 1e-14 * (E + k * T) / h)
        assert abs((dz * V).sum() - diff) <= tol


@pytest.mark.parametrize("T,d,k", [(5, 64, 2), (40, 512, 6), (17, 1032, 8)])
def test_combine_gradient(T, d, k):
    """sum(dout * combine(y, g)) is linear in y and in g, so its differences are exact."""
    gen = torch.Generator().manual_seed(T)
    row_of = torch.randperm(T * k, generator=gen).to(torch.int32)
    row_of[::7] = -1
    dout, y = torch.randn(T, d, generator=gen).bfloat16(), torch.randn(T * k, d, generator=gen).bfloat16()
    g = torch.rand(T, k, generator=gen)
    dy = torch.zeros(T * k, d, dtype=torch.bfloat16, device="cuda")
    dy, dgate = moe.combine_backward(dout.cuda(), y.cuda(), row_of.cuda(), g.cuda(), dy=dy)
    n = lambda t: t.cpu().double().numpy()  # noqa: E731
    rows = row_of.view(T, k).numpy()

    def loss(yy, gg):
        total = 0.0
        for t in range(T):
            for j in range(k):
                if rows[t, j] >= 0:
                    total += gg[t, j] * (n(dout)[t] * yy[rows[t, j]]).sum()
        return total

    rng = np.random.default_rng(0)
    Vg, Vy = rng.normal(size=(T, k)), rng.normal(size=(T * k, d))
    diff = (loss(n(y), n(g) + Vg) - loss(n(y), n(g) - Vg)) / 2
    _, _, bound = ref.combine_backward(n(dout), n(y), row_of.numpy(), n(g), n(dy))
    assert abs((n(dgate) * Vg).sum() - diff) <= (bound * np.abs(Vg)).sum() + 1e-10 * (1 + abs(diff))
    diff = (loss(n(y) + Vy, n(g)) - loss(n(y) - Vy, n(g))) / 2
    tol = (ref.BF16 + 2 * ref.F32) * 1.01 * (np.abs(n(dy)) * np.abs(Vy)).sum()   # dy's rounding
    assert abs((n(dy) * Vy).sum() - diff) <= tol + 1e-10 * (1 + abs(diff))
