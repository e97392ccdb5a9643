"""Pins of the oracle's token log probabilities and post-training losses
(oracle/losses.py): gradients against central differences, closed forms, the
clip's borders, rows that carry no loss."""
import math

import numpy as np
import pytest

from oracle import losses
from oracle.softmax import cross_entropy


def _batch(M, V, seed):
    rng = np.random.default_rng(seed)
    y = rng.normal(0, 2, (M, V))
    t = rng.integers(0, V, M)
    logp = losses.token_logp(y, t)
    return rng, y, t, logp


def _differences(f, y, h=1e-5):
    g = np.zeros_like(y)
    for idx in np.ndindex(*y.shape):
        up, down = y.copy(), y.copy()
        up[idx] += h
        down[idx] -= h
        g[idx] = (f(up) - f(down)) / (2 * h)
    return g


@pytest.mark.parametrize("beta", [0.0, 0.3])
def test_policy_gradient_is_the_derivative(beta):
    rng, y, t, logp = _batch(6, 7, 1)
    args = dict(old_logp=logp - np.array([0.5, -0.6, 0.05, -0.05, 0.4, -0.4]), ref_logp=logp + rng.normal(0, 0.3, 6),
                advantages=np.array([1.0, -1.5, 0.7, -0.7, -2.0, 2.0]), weights=np.array([.2, .3, .1, 0., .5, .4]),
                beta=beta, eps_low=0.2, eps_high=0.28)
    _, _, g, coef = losses.policy(y, t, **args)
    d = _differences(lambda x: losses.policy(x, t, **args)[0], y)
    # truncation h^2 and cancellation eps / h, each far below 1e-8
    assert np.abs(g - d).max() < 1e-8
    assert not g[3].any()
    if beta == 0.0:  # rho > 1 + eps with A > 0 and rho < 1 - eps with A < 0 are clipped away
        assert coef[0] == 0.0 and coef[1] == 0.0 and (coef[[2, 4, 5]] != 0).all()
    assert np.abs(g.sum(1)).max() < 1e-12


def test_preference_gradient_is_the_derivative():
    rng, y, t, logp = _batch(9, 5, 2)
    args = dict(weights=np.array([1, 1, 0, 1, 1, 1, .5, 1, 1.]), offsets=np.array([0, 2, 5, 5, 8]), ref_logp=logp +
                rng.normal(0, 0.5, 9), beta=0.7, smoothing=0.1)
    _, _, _, g, _ = losses.preference(y, t, **args)
    d = _differences(lambda x: losses.preference(x, t, **args)[0], y)
    assert np.abs(g - d).max() < 1e-8
    assert not g[8].any() and not g[2].any()


def test_closed_forms():
    # equal logits: logp = -ln V; old = ref = logp: rho = 1, no KL, loss = -sum w A
    y, t = np.zeros((3, 8)), np.array([0, 3, 7])
    lp = losses.token_logp(y, t)
    assert np.allclose(lp, -math.log(8), rtol=0, atol=1e-14)
    # against the cross-entropy oracle, and at the lowest values fp32 holds
    rng = np.random.default_rng(0)
    x, u = rng.normal(0, 3, (5, 40)), rng.integers(0, 40, 5)
    assert np.allclose(losses.token_logp(x, u), -cross_entropy(x, u), rtol=0, atol=1e-12)
    assert np.allclose(losses.token_logp(np.full((2, 9), -3.4e38), np.array([0, 8])), -math.log(9))
    A, w = np.array([1.0, -2.0, 0.5]), np.array([0.5, 0.25, 0.25])
    loss, _, g, _ = losses.policy(y, t, lp, A, w, ref_logp=lp, beta=0.5)
    assert loss == pytest.approx(-(A * w).sum(), abs=1e-14)
    assert g[0, 0] == pytest.approx(-0.5 * 7 / 8) and g[0, 1] == pytest.approx(0.5 / 8)
    # no margin: ln 2; two empty answers likewise
    loss, h, _, _, _ = losses.preference(y[:2], t[:2], np.ones(2), np.array([0, 1, 2]), beta=0.3)
    assert h[0] == pytest.approx(0.0, abs=1e-15) and loss == pytest.approx(math.log(2))
    assert losses.preference(y[:0], t[:0], np.ones(0), np.array([0, 0, 0]))[0] == pytest.approx(math.log(2))


def test_rows_without_weight_and_bad_targets():
    y = np.array([[np.nan, np.inf], [0.0, 1.0], [0.0, 0.0]])
    loss, lp, g, _ = losses.policy(y, np.array([-100, 1, 2]), np.zeros(3), np.ones(3), np.array([0.0, 1.0, 0.0]))
    assert np.isfinite(loss) and lp[0] == 0 and not g[0].any() and not g[2].any()
    loss, lp, g, _ = losses.policy(y, np.array([0, 1, 2]), np.zeros(3), np.ones(3), np.array([0.0, 1.0, 1.0]))
    assert np.isnan(loss) and np.isnan(lp[2]) and np.isnan(g[2]).all() and np.isfinite(g[1]).all()
