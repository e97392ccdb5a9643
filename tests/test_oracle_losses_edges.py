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
