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
