"""Pins of the row-loss oracle: finite differences of every loss, closed forms,
and agreement with the row cross-entropy oracle where the two meet."""

import math

import numpy as np
import pytest

import oracle


def _numeric(f, z, h=1e-6):
    g = np.zeros_like(z)
    for i in np.ndindex(*z.shape):
        up, down = z.copy(), z.copy()
        up[i] += h
        down[i] -= h
        g[i] = (f(up) - f(down)) / (2 * h)
    return g


def _near(a, f, z):
    # central differences in float64: rounding of the loss over the step, a few
    # tens of operations of 2^-53 each; h^2 / 6 of the third derivative is below
    far = np.max(np.abs(a - _numeric(f, z)))
    assert far < 64 * 2.0 ** -53 * max(1.0, abs(f(z))) / 1e-6, far


def _z(seed, R=5, C=7):
    return np.random.default_rng(seed).standard_normal((R, C)) * 2


T = np.array([3, -1, 0, 6, 2])


def test_logprob_by_hand_and_differences():
    logp, lse = oracle.logprob_rows([[0.0, math.log(3.0)]], [1], 1.0)
    assert logp[0] == pytest.approx(math.log(0.75)) and lse[0] == pytest.approx(math.log(4.0))
    z, g = _z(0), np.array([0.5, 1.0, -2.0, 0.0, 1.5])
    f = lambda x: float(np.sum(g * oracle.logprob_rows(x, T, 0.7)[0]))
    _near(oracle.logprob_rows_bwd(z, T, g, 0.7), f, z)
    assert np.all(oracle.logprob_rows_bwd(z, T, g, 0.7)[1] == 0)


IDX = np.array([[0, 3, 5], [2, -1, 1], [4, 4, 6], [-1, -1, -1], [6, 0, -1]])
VAL = np.random.default_rng(9).standard_normal((5, 3))


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_distill_differences(rest, weighted):
    z = _z(1)
    lse = np.array([2.5, 2.0, 3.0, 1.0, 2.2]) if rest else None
    w = np.array([1.0, 0.5, 2.0, 1.0, 0.0]) if weighted else None
    f = lambda x: oracle.distill_rows(x, IDX, VAL, lse, 0.8, w)[0]
    _near(oracle.distill_rows(z, IDX, VAL, lse, 0.8, w)[2], f, z)


def test_distill_meets_cross_entropy_and_itself():
    z = _z(2, 4, 6)
    t = np.array([1, 5, 0, 2])
    a = oracle.distill_rows(z, t[:, None], np.zeros((4, 1)), None, 1.5)
    b = oracle.ce_rows(z, t, 1.5)
    assert a[0] == pytest.approx(b[0]) and np.allclose(a[1], b[1]) and np.allclose(a[2], b[2])
    # every column listed, the student's own logits: no divergence
    every = np.tile(np.arange(6), (4, 1))
    for lse in (None, oracle.logprob_rows(z, np.zeros(4, int))[1]):
        loss, rows, grad = oracle.distill_rows(z, every, z, lse)
        assert np.allclose(rows, 0, atol=1e-12) and np.allclose(grad, 0, atol=1e-12)
    # some columns listed with the student's own normaliser: none either
    part = np.tile([1, 4], (4, 1))
    lse = oracle.logprob_rows(z, np.zeros(4, int))[1]
    _, rows, grad = oracle.distill_rows(z, part, np.take_along_axis(z, part, 1), lse)
    assert np.allclose(rows, 0, atol=1e-12) and np.allclose(grad, 0, atol=1e-12)


@pytest.mark.parametrize("kl", [0.0, 0.3])
def test_policy_differences(kl):
    z = _z(3)
    logp = oracle.logprob_rows(z, T, 0.9)[0]
    # off the borders, on both sides of them
    old = logp - np.array([0.1, 0.0, 0.5, -0.5, -0.1])
    adv = np.array([1.5, 1.0, 2.0, -1.0, -0.7])
    ref = logp + np.array([0.2, 0.0, -0.3, 0.1, 0.4]) if kl else None
    w = np.array([1.0, 1.0, 0.5, 2.0, 1.0])
    run = lambda x: oracle.policy_rows(x, T, old, adv, ref, 0.9, 0.2, 0.25, kl, w)
    _near(run(z)[3], lambda x: run(x)[0], z)
    # a positive advantage beyond the upper border, a negative one below the lower: clipped
    if not kl:
        assert run(z)[4][2] == 0 and run(z)[4][3] == 0 and run(z)[4][0] != 0


@pytest.mark.parametrize("kind,margin,smoothing", [
    (oracle.rows.SIGMOID, 0.0, 0.0), (oracle.rows.SIGMOID, 0.4, 0.1),
    (oracle.rows.HINGE, 0.3, 0.0), (oracle.rows.SQUARE, 0.0, 0.0)])
@pytest.mark.parametrize("mean", [False, True])
def test_preference_differences(kind, margin, smoothing, mean):
    z = _z(4, 9, 6)
    t = np.array([1, -1, 0, 5, 2, 3, 3, 4, 0])
    off = [0, 3, 3, 6, 8]                      # an empty sequence, a row behind the last
    c, r = [0, 2, 0, 3, 1], [2, 3, 3, 3, 0]    # one pair of a sequence with itself
    ref = np.array([-5.0, 0.0, -6.0, -4.0])
    w = np.array([1.0, 0.5, 0.0, 1.0, 2.0])
    f = lambda x: oracle.preference_rows(x, t, off, c, r, ref, kind, 0.3, margin, smoothing, mean,
                                         1.1, w)
    _near(f(z)[3], lambda x: f(x)[0], z)
    assert np.all(f(z)[3][8] == 0)


def test_preference_by_hand():
    # two one-token sequences over two columns: d = log(0.75) - log(0.5)
    z = np.array([[0.0, math.log(3.0)], [0.0, 0.0]])
    out = oracle.preference_rows(z, [1, 0], [0, 1, 2], [0], [1], beta=2.0)
    d = math.log(0.75) - math.log(0.5)
    assert out[0] == pytest.approx(math.log1p(math.exp(-2 * d)))
    assert oracle.preference_rows(z, [1, 0], [0, 1, 2], [0], [1], kind=oracle.rows.SQUARE,
                                  beta=2.0)[0] == pytest.approx((d - 0.25) ** 2)


@pytest.mark.parametrize("kind", [oracle.rows.SIGMOID, oracle.rows.HINGE, oracle.rows.SQUARE])
def test_preference_nan_reaches_its_pairs(kind):
    # sequence 1 holds a NaN: its pairs, one of them with itself, and their sequences
    z = _z(6, 4, 5)
    z[1, 3] = np.nan
    _, pairs, seq, grad, _ = oracle.preference_rows(z, [1, 2, 0, 4], [0, 1, 2, 3, 4], [1, 0, 2],
                                                    [1, 2, 3], kind=kind)
    assert np.array_equal(np.isnan(pairs), [True, False, False]) and np.isnan(seq[1])
    assert np.array_equal(np.isnan(grad).all(1), [False, True, False, False])
    assert np.isfinite(grad[[0, 2, 3]]).all()
