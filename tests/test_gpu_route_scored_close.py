"""The scored router where 32 bits cannot tell: keys and group values next to each other,
many ties, and the sizes between the powers of two; ids bit for bit against 64-bit sorting."""
import numpy as np
import pytest
import torch

import router_ref as ref

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")


def _same(z, k, kind, bias, G=1, kg=0, top2=False, renorm=True):
    b = None if bias is None else torch.from_numpy(bias).cuda()
    idx, gate = moe.route_scored(torch.from_numpy(z).cuda(), k, score=kind, bias=b, n_groups=G, topk_groups=kg,
                                 group_score=int(top2), renorm=renorm)
    widx, wgate = ref.route(z, k, kind, bias, G, kg, top2, renorm)
    bad = np.argwhere((idx.cpu().numpy() != widx).any(1))
    assert not len(bad), (bad[0], idx[int(bad[0, 0])], widx[bad[0, 0]])
    # E exponentials summed in fp32 at the worst, and the gate's own roundings
    bound = (z.shape[1] + 10) * ref.F32
    assert np.all(np.abs(gate.cpu().numpy() - wgate) <= bound * np.abs(wgate) + 1e-38)


@pytest.mark.parametrize("E,G,kg,k", [(256, 8, 4, 8), (256, 1, 1, 8), (128, 4, 2, 8), (160, 8, 3, 6), (200, 4, 2, 7),
                                      (60, 4, 2, 5), (64, 8, 3, 6), (96, 1, 1, 8), (24, 3, 2, 4), (256, 32, 5, 8)])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("top2", [False, True])
def test_keys_and_groups_next_to_each_other(E, G, kg, k, kind, top2):
    """Biases that undo the scores' differences up to a few 1e-7: the 64-bit order decides
    between experts, and between groups."""
    rng = np.random.default_rng(E + k)
    base = rng.normal(size=E).astype(np.float32)
    p, _ = ref.scores(base, kind)
    bias = (1.0 - p + 2e-7 * rng.integers(-3, 4, size=E)).astype(np.float32)
    z = np.stack([base + np.float32(1e-7) * rng.integers(-4, 5, size=E).astype(np.float32) for _ in range(120)])
    z[60:] += (1e-3 * rng.normal(size=(60, E))).astype(np.float32)
    z[5, rng.random(E) < 0.5] = -np.inf
    _same(z.astype(np.float32), k, kind, bias, G, kg, top2)


@pytest.mark.parametrize("E", [2, 31, 32, 33, 64, 65, 100, 128, 129, 192, 250, 256])
@pytest.mark.parametrize("kind,biased", [(0, False), (1, False), (0, True), (1, True)])
def test_many_ties(E, kind, biased):
    """Rows of a few distinct logits, all equal, all masked, one live: ids ascend."""
    rng = np.random.default_rng(E)
    z = rng.integers(0, 3, size=(60, E)).astype(np.float32)
    z[0], z[1], z[2] = 1.0, -np.inf, np.nan
    z[3], z[3, E - 1] = -np.inf, 2.0
    z[4] = np.where(np.arange(E) % 2, 0.0, -0.0)
    bias = (0.5 * rng.integers(0, 2, size=E)).astype(np.float32) if biased else None
    _same(z, min(8, E), kind, bias, renorm=True)
    if E % 2 == 0 and E >= 32:
        _same(z, 6, kind, bias, 2, 1, True)


def test_large_biases():
    """The keys' error grows with the bias: 2^-24 of it is lost when it is added in fp32."""
    rng = np.random.default_rng(0)
    z = rng.normal(size=(200, 64)).astype(np.float32)
    for size in (1e3, 1e6, 1e30):
        bias = (size + 0 * z[0]).astype(np.float32)
        _same(z, 6, 1, bias)
        _same(z, 6, 0, bias, 8, 4, True)
        _same(z, 6, 1, (size * rng.normal(size=64)).astype(np.float32), 8, 4, True)
