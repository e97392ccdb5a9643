"""The root-mean-square norm with the residual's addition, and its backward --
TEST INFRASTRUCTURE.

Defined in include/archead.h.  fp64 throughout but for the sum h, which is taken
in fp32 and rounded to the residual's type, as it is stored; the norm is the
stored sum's.  Pins live in tests/test_oracle_norm.py.
"""
from __future__ import annotations

import numpy as np


def to_bf16(x: np.ndarray) -> np.ndarray:
    """fp32 values rounded to bf16 (nearest even), as fp32; finite inputs."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32)


def add(x: np.ndarray, residual: np.ndarray, bf16: bool) -> np.ndarray:
    h = np.asarray(x, dtype=np.float32) + np.asarray(residual, dtype=np.float32)
    return (to_bf16(h) if bf16 else h).astype(np.float64)


def rms(h: np.ndarray, eps: float) -> np.ndarray:
    return np.sqrt(np.mean(np.square(h), axis=1, keepdims=True) + float(np.float32(eps)))


def forward(h: np.ndarray, weight: np.ndarray, eps: float, offset: float) -> np.ndarray:
    return h / rms(h, eps) * (weight + offset)


def backward(dy, h, weight, eps: float, offset: float, dres=None):
    """(dh, dweight, size): the gradients, and the sum of the magnitudes that dh is formed from."""
    r = 1.0 / rms(h, eps)
    g = dy * (weight + offset)
    c = np.mean(g * h, axis=1, keepdims=True)
    dh = r * (g - h * r ** 2 * c)
    size = r * (np.abs(g) + np.abs(h) * r ** 2 * np.mean(np.abs(g * h), axis=1, keepdims=True))
    if dres is not None:
        dh, size = dh + dres, size + np.abs(dres)
    return dh, np.sum(dy * h * r, axis=0), size
