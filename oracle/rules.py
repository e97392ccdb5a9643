"""Penalties, biases and masks on logits, and the draw from what they leave --
TEST INFRASTRUCTURE.

Defined in include/archead.h.  One row, one token at a time; every operation in
fp32, as the definition rounds them (numpy's fp32 operations are correctly
rounded), so the kernels are held to it bit for bit.  The draw is fp64.  Pins
live in tests/test_oracle_rules.py.
"""
from __future__ import annotations

import numpy as np

f32 = np.float32


def adjust(y, history=(), prompt=0, repetition=1.0, frequency=0.0, presence=0.0, bias=(), mask=None):
    """One row: y fp32 V; history the tokens in use; bias a list of (id, value); mask V truth values."""
    y = np.array(y, dtype=f32)
    V = len(y)
    with np.errstate(all="ignore"):
        for v in sorted({int(t) for t in history if 0 <= t < V}):
            y[v] = y[v] / f32(repetition) if y[v] > 0 else y[v] * f32(repetition)
        count = {}
        for t in history[max(prompt, 0):]:
            if 0 <= t < V:
                count[int(t)] = count.get(int(t), 0) + 1
        for v, c in count.items():
            y[v] = (y[v] - f32(frequency) * f32(c)) - f32(presence)
        for v, b in {int(i): f32(b) for i, b in bias if 0 <= i < V}.items():
            y[v] = f32(-np.inf) if b == -np.inf else y[v] + b
    if mask is not None:
        y[~np.asarray(mask, dtype=bool)] = -np.inf
    return y


def top(y, K: int):
    """(values, indices) of the K largest: larger first, NaN before all, equal values by index."""
    y = np.asarray(y, dtype=f32)
    nan = np.isnan(y)
    rank = np.lexsort((np.arange(len(y)), np.where(nan, f32(0), -y), ~nan))[:K]
    return y[rank], rank.astype(np.int32)


def draw(values, indices, u, temperature) -> int:
    v = np.asarray(values, dtype=np.float64)
    if not v[0] > -np.inf:
        return -1
    if v[0] == np.inf or not temperature > 0:
        return int(indices[0])
    with np.errstate(invalid="ignore"):
        w = np.where(v > -np.inf, np.exp((v - v[0]) / np.float64(temperature)), 0.0)
    run = np.cumsum(w)
    over = np.nonzero(run > np.float64(u) * run[-1])[0]
    return int(indices[over[0] if len(over) else np.nonzero(w > 0)[0][-1]])


def bits(mask: np.ndarray) -> np.ndarray:
    """Truth values R x V -> int32 words R x ceil(V / 32), bit v % 32 of word v / 32."""
    R, V = mask.shape
    wide = np.zeros((R, -(-V // 32) * 32), dtype=np.uint8)
    wide[:, :V] = mask
    return np.packbits(wide, axis=1, bitorder="little").view("<u4").astype(np.uint32).view(np.int32)
