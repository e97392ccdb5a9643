"""Pins of oracle/embedding.py: the one-hot products and differences."""
import numpy as np

from oracle import embedding


def _case():
    rng = np.random.default_rng(0)
    V, d = 7, 5
    tokens = np.array([3, 0, 3, -1, 6, 2, 3, 7, -5, 2])
    return V, rng.normal(0, 1, (V, d)), tokens, rng.normal(0, 1, (len(tokens), d))


def test_lookup_is_the_one_hot_product():
    V, table, tokens, _ = _case()
    got = embedding.lookup(table, tokens, 0.5, pad=2)
    hot = np.array([[float(t == v and t != 2) for v in range(V)] for t in tokens])
    lost = np.array([t != 2 and not 0 <= t < V for t in tokens])
    assert np.isnan(got[lost]).all()
    assert np.allclose(got[~lost], (0.5 * hot @ table)[~lost], rtol=1e-15, atol=0)


def test_gradient_is_the_one_hot_product_and_the_differences():
    V, table, tokens, dout = _case()
    grad, size, count = embedding.gradient(dout, tokens, V, 0.5, pad=2)
    hot = np.array([[float(t == v and t != 2) for v in range(V)] for t in tokens])
    assert np.allclose(grad, 0.5 * hot.T @ dout, rtol=1e-14, atol=0)
    assert np.array_equal(count, hot.sum(0)) and np.all(np.abs(grad) <= size * (1 + 1e-12))

    def loss(table):
        out = embedding.lookup(table, tokens, 0.5, pad=2)
        return np.nansum(out * dout)

    for v in range(V):
        for j in range(table.shape[1]):
            step = np.zeros_like(table)
            step[v, j] = 1e-4
            assert abs((loss(table + step) - loss(table - step)) / 2e-4 - grad[v, j]) < 1e-9
