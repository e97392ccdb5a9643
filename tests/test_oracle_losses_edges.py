"""Pins of the oracle's losses (oracle/losses.py) where plain forms lose their
digits or their meaning."""
import math

import numpy as np
import pytest

from oracle import losses


def test_near_certain_tokens():
    """Two logits a gap apart: logp = -log1p(exp(-gap)), to the last digits of
    fp64 however small (two roundings and the exponential's: 4 x 2^-53)."""
    for gap in (1.0, 20.0, 40.0, 300.0):
        for t, y in ((0, [0.0, -gap]), (1, [-gap, 0.0])):
            want = -math.log1p(math.exp(-gap))
            assert losses.token_logp(np.array([y]), np.array([t]))[0] == pytest.approx(want, rel=2.0 ** -51, abs=0)


def test_near_certain_gradients():
    """The target's gradient c (1 - p) and the others' -c p sum to zero to their
    own precision: with two logits they are each other's opposite."""
    for gap in (1.0, 20.0, 40.0, 300.0):
        y, t = np.array([[0.0, -gap], [-gap, 0.0]]), np.array([0, 1])
        _, _, g, coef = losses.policy(y, t, np.zeros(2), np.array([1.0, -0.5]), np.ones(2))
        p = math.exp(-gap) / (1 + math.exp(-gap))
        for m in range(2):
            assert g[m, t[m]] == pytest.approx(coef[m] * p, rel=2.0 ** -50, abs=0)
            assert g[m, 1 - t[m]] == pytest.approx(-coef[m] * p, rel=2.0 ** -50, abs=0)


def test_an_unknown_advantage_is_not_a_zero_one():
    """A NaN advantage (normalised by a zero deviation) or an infinite one at a
    ratio of zero makes the loss and its row's gradient NaN; other rows keep
    theirs.  No advantage is no gain, also where the old policy had the token
    masked."""
    y, t, w = np.zeros((4, 3)), np.array([0, 1, 2, 0]), np.array([0.5, 0.5, 0.5, 0.0])
    y[3] = np.nan
    old = np.full(4, -math.log(3))
    for A, o in ((math.nan, old[0]), (math.inf, math.inf)):
        old[0] = o
        loss, _, g, coef = losses.policy(y, t, old, np.array([A, 1.0, -1.0, math.nan]), w)
        assert math.isnan(loss) and math.isnan(coef[0]) and np.isnan(g[0]).all()
        assert np.isfinite(g[1:]).all() and g[1:3].any(1).all() and not g[3].any()
    old[0] = -math.inf
    with np.errstate(over="ignore"):
        loss, _, g, _ = losses.policy(y, t, old, np.array([0.0, 1.0, -1.0, 0.0]), w)
    assert loss == pytest.approx(0.0) and not g[0].any()


def test_infinite_margins_are_decided():
    """A masked token in the rejected answer: -log sigma(inf) = 0 and no
    gradient; in the chosen one an infinite loss and the limit's slope."""
    y = np.zeros((4, 4))
    y[1, 2] = y[2, 0] = -np.inf
    t, w, off = np.array([1, 2, 0, 3]), np.ones(4), np.array([0, 1, 2, 3, 4])
    loss, h, _, g, coef = losses.preference(y[:2], t[:2], w[:2], off[:3], beta=0.3)
    assert h[0] == np.inf and loss == 0.0 and not g.any()
    loss, h, _, g, coef = losses.preference(y, t, w, off, beta=0.3)
    assert h[1] == -np.inf and loss == np.inf
    assert coef[2] == pytest.approx(-0.15) and coef[3] == pytest.approx(0.15) and np.isfinite(g).all()
    loss, h, _, g, coef = losses.preference(y[:2], t[:2], w[:2], off[:3], beta=0.3, smoothing=0.1)
    assert loss == np.inf and coef[0] == pytest.approx(0.03)


def test_a_masked_token_is_infinitely_far_from_its_reference():
    y, t = np.zeros((2, 4)), np.array([1, 2])
    y[0, 1] = -np.inf
    old, ref = np.array([-1.4, -1.4]), np.array([-2.0, -1.4])
    for A in (1.0, -1.0):
        loss, lp, g, coef = losses.policy(y, t, old, np.array([A, 0.0]), np.ones(2), ref, beta=0.1)
        assert lp[0] == -np.inf and loss == np.inf and coef[0] == -np.inf and np.isfinite(g[1]).all()
    # the other way round the reference's mask costs as much, with a finite slope
    loss, _, _, coef = losses.policy(np.zeros((1, 4)), t[:1], old[:1], np.ones(1), np.ones(1), np.array([-np.inf]), beta=0.1)
    assert loss == np.inf and np.isfinite(coef[0])
