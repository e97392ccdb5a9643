"""Pins of oracle/norm.py: closed forms, differences, scale invariance, and bf16
rounding against torch's."""
import numpy as np
import torch

from oracle import norm


def test_bf16_rounding_is_torchs():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(0, 1, 4096), rng.normal(0, 1e-30, 64), [0.0, -0.0, 1.00390625, 1.01171875]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
    assert np.array_equal(norm.to_bf16(x).view(np.uint32), want.view(np.uint32))


def test_closed_forms():
    h = np.array([[3.0, -4.0], [1.0, 1.0]])
    w = np.array([2.0, 0.5])
    y = norm.forward(h, w, 0.0, 0.0)
    assert np.allclose(y[0], [3 / np.sqrt(12.5) * 2, -4 / np.sqrt(12.5) / 2], rtol=1e-15)
    assert np.allclose(y[1], w, rtol=1e-15)
    assert np.allclose(norm.forward(h, w, 0.0, 1.0), norm.forward(h, w + 1.0, 0.0, 0.0), rtol=1e-15)
    # without eps the norm does not change with the row's scale, so its gradient is orthogonal to the row
    rng = np.random.default_rng(1)
    h, w, u = rng.normal(0, 1, (5, 33)), rng.normal(1, 0.2, 33), rng.normal(0, 1, (5, 33))
    assert np.allclose(norm.forward(7.0 * h, w, 0.0, 0.0), norm.forward(h, w, 0.0, 0.0), rtol=1e-13)
    dh, _, _ = norm.backward(u, h, w, 0.0, 0.0)
    assert np.abs(np.sum(dh * h, axis=1)).max() < 1e-13


def test_gradients_are_the_differences():
    rng = np.random.default_rng(2)
    for d, eps, offset in ((1, 0.1, 0.0), (5, 1e-6, 1.0), (48, 1e-2, 0.0)):
        h, w = rng.normal(0, 1.5, (3, d)), rng.normal(1, 0.3, d)
        u, through = rng.normal(0, 1, (3, d)), rng.normal(0, 1, (3, d))

        def loss(h, w):
            return np.sum(u * norm.forward(h, w, eps, offset)) + np.sum(through * h)

        dh, dw, size = norm.backward(u, h, w, eps, offset, dres=through)
        assert np.all(np.abs(dh) <= size * (1 + 1e-12))
        e = 1e-5
        for m in range(3):
            for j in range(d):
                step = np.zeros_like(h)
                step[m, j] = e
                assert abs((loss(h + step, w) - loss(h - step, w)) / (2 * e) - dh[m, j]) < 1e-7
        for j in range(d):
            step = np.zeros(d)
            step[j] = e
            assert abs((loss(h, w + step) - loss(h, w - step)) / (2 * e) - dw[j]) < 1e-7


def test_the_sum_is_rounded_as_it_is_stored():
    x, r = np.array([[1.0, 2.0 ** -9]], dtype=np.float32), np.array([[2.0 ** -8, 1.0]], dtype=np.float32)
    assert np.array_equal(norm.add(x, r, True), [[1.0, 1.0]])  # ties to even, and below half a step
    assert np.array_equal(norm.add(x, r, False), [[1.0 + 2.0 ** -8, 1.0 + 2.0 ** -9]])
