"""Pins of the oracle's 8-bit matrices (oracle/fp8.py)."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import fp8


def test_codes_against_torch():
    import torch
    c = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(c.copy()).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp8.decode(c), t, equal_nan=True)
    ok = (c & 127) != 127
    assert np.array_equal(fp8.encode(fp8.decode(c[ok])), c[ok])
    x = np.random.default_rng(0).normal(0, 40, 20000).astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8.encode(x.astype(np.float64)), want)


def test_ties_and_ends():
    v = fp8.decode(np.arange(127, dtype=np.uint8))
    mid = (v[1:] + v[:-1]) / 2
    even = np.arange(126) + (np.arange(126) % 2)
    assert np.array_equal(fp8.encode(mid), even)
    assert np.array_equal(fp8.encode(np.nextafter(mid, 0)), np.arange(126))
    assert np.array_equal(fp8.encode(-np.nextafter(mid, 1e9)), np.arange(1, 127) + 128)
    assert fp8.encode(np.array([1e30, -1e30])).tolist() == [126, 254]


@pytest.mark.parametrize("amax", [1.0, 3.1415927, 448.0, 1e-30, 6.5e30, 1.5e-44])
def test_nearest_of_the_exact_quotient(amax):
    """Codes of every kind of value against exact fractions."""
    rng = np.random.default_rng(1)
    x = (rng.uniform(-1, 1, (1, 128)).astype(np.float32) * np.float32(amax)).astype(np.float32)
    x[0, 0] = np.float32(amax)
    codes, s = fp8.quantize(x)
    table = [Fraction(float(t)) for t in fp8.decode(np.arange(127, dtype=np.uint8))]
    for j in range(0, 128, 5):
        q = abs(Fraction(float(x[0, j])) / Fraction(float(s[0, 0])))
        best = min(range(127), key=lambda i: (abs(table[i] - q), i % 2))
        assert codes[0, j] & 127 == best


def test_product_of_small_integers_is_exact():
    rng = np.random.default_rng(2)
    a, b = rng.integers(-7, 8, (5, 272)).astype(float), rng.integers(-7, 8, (300, 272)).astype(float)
    sa, sb = 2.0 ** rng.integers(-3, 3, (3, 5)), 2.0 ** rng.integers(-3, 3, (3, 3))
    out, bound = fp8.matmul(fp8.encode(a), sa.astype(np.float32), fp8.encode(b), sb.astype(np.float32))
    want = np.zeros((5, 300))
    for k in range(272):
        for n in range(300):
            want[:, n] += a[:, k] * sa[k // 128] * b[n, k] * sb[n // 128, k // 128]
    assert np.array_equal(out, want) and (bound >= np.abs(out)).all()
    z, s = fp8.quantize(np.zeros((2, 16)))
    assert not z.any() and not s.any()
