"""The router's gates and their gradient where scores are very small or gates constant,
against the formulas with the chosen experts' own largest logit as the reference of the
exponentials (the softmax's normaliser cancels when gates are renormalised)."""
import numpy as np
import pytest
import torch

import router_ref as ref

pytestmark = pytest.mark.gpu
moe = pytest.importorskip("combine_overlap_b200.moe")


def _backward(dg, z, idx, kind, scale=1.0):
    return moe.route_scored_backward(torch.from_numpy(dg).cuda(), torch.from_numpy(z).cuda(),
                                     torch.from_numpy(idx.astype(np.int32)).cuda(), score=kind, renorm=True,
                                     scale=scale).cpu().double().numpy()


def _shares(z, idx, kind):
    """The chosen experts' shares w / S, row by row, without the softmax's normaliser."""
    s = np.take_along_axis(z.astype(np.float64), idx, 1)
    w = np.exp(s - s.max(1, keepdims=True))
    if kind == 1:                          # sigmoid(s) = exp(s) / (1 + exp(s))
        w /= 1 + np.exp(s)
    return w / w.sum(1, keepdims=True), s


def _gradient(dg, z, idx, kind, scale=1.0):
    q, s = _shares(z, idx, kind)
    c = scale * dg.astype(np.float64)
    d = q * (c - (q * c).sum(1, keepdims=True))
    if kind == 1:
        d /= 1 + np.exp(s)                 # 1 - sigmoid(s)
    dz = np.zeros(z.shape)
    np.put_along_axis(dz, idx, d, 1)
    # one rounding to fp32; shares of 64 bits, subnormal ones (from 2^-1029 on) of 44 and more
    return dz, ref.F32 * np.abs(dz) + 1e-12 * np.abs(c).sum(1, keepdims=True) * (dz != 0)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("scale", [1.0, 2.5])
def test_a_constant_gate_has_no_gradient(kind, scale):
    """A renormalised gate of one expert is `scale` whatever the logits: 0, and no rounding of it."""
    rng = np.random.default_rng(kind)
    z = (3 * rng.normal(size=(2000, 24))).astype(np.float32)
    dg = rng.normal(size=(2000, 1)).astype(np.float32)
    assert not _backward(dg, z, ref.route(z, 1, kind)[0].astype(int), kind, scale).any()
    z[:, 1:] = -np.inf                     # one live expert among three chosen
    dg = rng.normal(size=(2000, 3)).astype(np.float32)
    assert not _backward(dg, z, np.tile([0, 1, 2], (2000, 1)), kind, scale).any()


@pytest.mark.parametrize("kind", [0, 1])
def test_gradients_of_sums_whose_reciprocal_overflows(kind):
    """The chosen scores' sum below 2^-1024: by a bias, a group limit or the caller's ids."""
    low = np.array([-709.0, -709.5, -709.2, -709.7]) - (0 if kind else 2)
    z = np.stack([np.r_[0, low, -5], np.r_[0, low[::-1], 1], np.r_[0, low - 0.05, -800]]).astype(np.float32)
    idx = np.array([[1, 2, 3], [4, 1, 2], [3, 4, 1]])
    dg = np.array([[2.5, -5, 1], [1, 1, -3], [0.1, 7, 1]], np.float32)
    want, bound = _gradient(dg, z, idx, kind)
    got = _backward(dg, z, idx, kind)
    assert np.abs(want).max() > 0.5 and np.all(np.abs(got - want) <= bound), (got, want)


FAR = np.array([-715, -716, -714.5, -717, -730, -730.25, -731, -729.5, -743, -744, -744.5, -742], np.float32).reshape(3, 4)


def test_shares_of_experts_far_below_the_largest():
    """Softmax gates of experts 714 to 744 below the row's largest, which a bias leaves out:
    their scores are subnormal in 64 bits, their shares are not."""
    z = np.concatenate([np.zeros((3, 1), np.float32), FAR], 1)
    bias = np.array([-9, 0.4, 0.3, 0.2, 0.1], np.float32)
    dg = np.array([[1, -2, 0.5], [3, 1, -1], [0.25, 2, 1]], np.float32)
    idx, gate = moe.route_scored(torch.from_numpy(z).cuda(), 3, bias=torch.from_numpy(bias).cuda(), scale=1.5)
    chosen = np.tile([1, 2, 3], (3, 1))
    assert np.array_equal(idx.cpu().numpy(), chosen)
    q, _ = _shares(z, chosen, 0)
    # one rounding to fp32, and 64-bit ones
    assert np.all(np.abs(gate.cpu().double().numpy() - 1.5 * q) <= ref.F32 * 1.5 * q * 1.0001)
    want, bound = _gradient(dg, z, chosen, 0, 1.5)
    assert np.all(np.abs(_backward(dg, z, chosen, 0, 1.5) - want) <= bound)


def test_scores_that_underflow_have_neither_gate_nor_gradient():
    """All chosen more than 745.13 below: their sum is 0 in 64 bits, and so are the gates."""
    z = np.array([[0, -746, -747, -748], [0, -746, -1e30, -np.inf], [1e38, 5, 6, 7]], np.float32)
    bias = np.array([-9, 0.4, 0.3, 0.2], np.float32)
    dg = np.ones((3, 2), np.float32)
    idx, gate = moe.route_scored(torch.from_numpy(z).cuda(), 2, bias=torch.from_numpy(bias).cuda())
    assert (idx.cpu().numpy() == [1, 2]).all() and not gate.any()
    assert not _backward(dg, z, idx.cpu().numpy(), 0).any()
    # one of them inside: it has the whole sum
    z[:, 1] = z[:, 0] + np.float32(-744)
    z[2, 0] = 1e4
    z[2, 1:] = [1e4 - 744, 5, 6]
    idx, gate = moe.route_scored(torch.from_numpy(z).cuda(), 2, bias=torch.from_numpy(bias).cuda())
    want = np.array([[np.exp(3.0) / (1 + np.exp(3.0)), 1 / (1 + np.exp(3.0))], [1, 0], [1, 0]])   # -744 and -747
    assert np.all(np.abs(gate.cpu().double().numpy() - want) <= ref.F32 * want * 1.0001)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_gradients_of_masked_and_dropped_slots_are_not_read(kind, renorm, what):
    """NaN and infinities in dgate where the expert is masked or the slot dropped reach nothing."""
    rng = np.random.default_rng(5)
    z = rng.normal(size=(64, 40)).astype(np.float32)
    z[::2, 3:] = -np.inf                   # three live experts among five chosen
    z[5], z[6] = -np.inf, np.nan
    idx = ref.route(z, 5, kind)[0]
    idx[9, 2], idx[11, 4] = -1, 40
    dg = rng.normal(size=(64, 5)).astype(np.float32)
    inside = (idx >= 0) & (idx < 40)
    used = inside & np.isfinite(np.take_along_axis(z, np.where(inside, idx, 0).astype(int), 1))
    run = lambda d: moe.route_scored_backward(torch.from_numpy(d).cuda(), torch.from_numpy(z).cuda(),  # noqa: E731
                                              torch.from_numpy(idx).cuda(), score=kind, renorm=renorm)
    want, got = run(np.where(used, dg, np.float32(0))), run(np.where(used, dg, np.float32(what)))
    assert not used.all() and torch.isfinite(want).all() and torch.equal(got, want)


@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoid_scores_next_to_one(renorm):
    """p (1 - p) of logits up to 80: exp(-z) of 64 bits, where 1 - p has none left from 37 on."""
    z = np.array([[20, 30, 35, 36, -3], [37, 40, 50, 60, 1], [38, 70, 45, 80, 90]], np.float32)
    idx = np.tile([0, 1, 2, 3], (3, 1))
    dg = np.array([[1, -2, 0.5, 1], [3, 1, -1, 2], [0.25, 2, 1, -1]], np.float32)
    got = moe.route_scored_backward(torch.from_numpy(dg).cuda(), torch.from_numpy(z).cuda(),
                                    torch.from_numpy(idx.astype(np.int32)).cuda(), score=1, renorm=renorm).cpu().double().numpy()
    if renorm:
        q, s = _shares(z, idx, 1)
        d = q * (dg - (q * dg).sum(1, keepdims=True)) / (1 + np.exp(s))
    else:
        s = z[:, :4].astype(np.float64)
        d = dg / (1 + np.exp(-s)) / (1 + np.exp(s))
    # a rounding to fp32; 64-bit ones of the sum of 4 shares, of terms up to 4 |d|
    assert np.all(np.abs(got[:, :4] - d) <= (ref.F32 + 1e-14) * np.abs(d)) and not got[:, 4].any()
