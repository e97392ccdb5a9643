"""Rows of an embedding table by token, and the table's gradient -- TEST
INFRASTRUCTURE.

Defined in include/archead.h; fp64, one token at a time.  Pins live in
tests/test_oracle_embedding.py.
"""
from __future__ import annotations

import numpy as np


def lookup(table: np.ndarray, tokens: np.ndarray, scale: float, pad: int = -1) -> np.ndarray:
    out = np.full((len(tokens), table.shape[1]), np.nan)
    for i, t in enumerate(tokens):
        if t == pad:
            out[i] = 0.0
        elif 0 <= t < table.shape[0]:
            out[i] = scale * table[t]
    return out


def gradient(dout: np.ndarray, tokens: np.ndarray, V: int, scale: float, pad: int = -1):
    """(gradient, sums of the terms' magnitudes, number of terms of each row)."""
    grad, size, count = np.zeros((V, dout.shape[1])), np.zeros((V, dout.shape[1])), np.zeros(V, dtype=np.int64)
    for i, t in enumerate(tokens):
        if t != pad and 0 <= t < V:
            grad[t] += scale * dout[i]
            size[t] += abs(scale) * np.abs(dout[i])
            count[t] += 1
    return grad, size, count
