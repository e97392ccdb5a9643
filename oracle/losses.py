"""Token log probabilities and post-training losses over logits, with the
logits' gradients -- TEST INFRASTRUCTURE.

fp64, one row at a time, from the definitions in include/archead.h: rows of
weight 0 (or outside every answer) are not looked at, a target outside
[0, V) gives NaN.  Pins live in tests/test_oracle_losses.py: gradients against
central differences of the losses, closed forms, the clip's borders.
"""
from __future__ import annotations

import numpy as np


def _row_logp(row, target):
    if not 0 <= target < row.shape[0]:
        return np.nan
    with np.errstate(invalid="ignore", divide="ignore"):
        away = row - row.max()  # taken first: at the type's lowest values lse - y would lose everything
        top = int(away.argmax())
        rest = np.exp(np.delete(away, top)).sum()  # next to the largest's 1 a sum would round off small terms
        return away[target] - (np.log1p(rest) + away[top])  # away[top] is 0, or the row's NaN


def token_logp(logits, targets):
    """logp[m] = logits[m, t] - log sum exp, NaN for a target that is no column."""
    y = np.asarray(logits, dtype=np.float64)
    return np.array([_row_logp(y[m], int(targets[m])) for m in range(y.shape[0])])


def _gradient(y, targets, coef):
    g = np.zeros_like(y)
    for m in range(y.shape[0]):
        if coef[m] == 0.0:
            continue
        if np.isnan(coef[m]):
            g[m] = np.nan
            continue
        e = np.exp(y[m] - y[m].max())
        others = np.delete(e, int(targets[m])).sum()  # 1 - p of the target, however near p is to 1
        with np.errstate(invalid="ignore"):  # an infinite coefficient at a probability of 0
            g[m] = -coef[m] * e / e.sum()
            g[m, int(targets[m])] = coef[m] * (others / e.sum())
    return g


def policy(logits, targets, old_logp, advantages, weights, ref_logp=None, beta=0.0, eps_low=0.2, eps_high=0.2,
           grad_scale=1.0):
    """(loss, logp, dlogits, coef) of the clipped policy loss with a KL term."""
    y = np.asarray(logits, dtype=np.float64)
    M = y.shape[0]
    loss, logp, coef = 0.0, np.zeros(M), np.zeros(M)
    for m in range(M):
        w = float(weights[m])
        if w == 0.0:
            continue
        lp = _row_logp(y[m], int(targets[m]))
        A = float(advantages[m])
        with np.errstate(over="ignore", invalid="ignore"):
            rho = np.exp(lp - float(old_logp[m]))
        kept = np.clip(rho, 1.0 - eps_low, 1.0 + eps_high)
        gain = float(rho) * A if A != 0.0 else 0.0  # no advantage, no gain: also at an infinite ratio
        known = rho == rho and gain == gain  # min and the comparison drop a NaN
        value = -min(gain, kept * A) if known else np.nan
        slope = (-gain if gain <= kept * A else 0.0) if known else np.nan
        if beta:
            r = float(ref_logp[m]) - lp
            value += beta * (np.expm1(r) - r if r != np.inf else r)  # exp(r) - r - 1 grows without end
            slope -= beta * np.expm1(r)
        loss += w * value
        logp[m], coef[m] = lp, w * slope
    return loss, logp, _gradient(y, targets, coef) * grad_scale, coef


def preference(logits, targets, weights, offsets, ref_logp=None, beta=0.1, smoothing=0.0, grad_scale=1.0):
    """(loss, margins, logp, dlogits, coef) of the preference loss over answer pairs."""
    y = np.asarray(logits, dtype=np.float64)
    M, P = y.shape[0], (len(offsets) - 1) // 2
    logp, coef, h = np.zeros(M), np.zeros(M), np.zeros(P)
    loss = 0.0
    for p in range(P):
        s = []
        for i in (2 * p, 2 * p + 1):
            total = 0.0
            for m in range(int(offsets[i]), int(offsets[i + 1])):
                if float(weights[m]) != 0.0:
                    logp[m] = _row_logp(y[m], int(targets[m]))
                    total += float(weights[m]) * (logp[m] - (float(ref_logp[m]) if ref_logp is not None else 0.0))
            s.append(total)
        h[p] = beta * (s[0] - s[1])
        loss += (1 - smoothing) * np.logaddexp(0.0, -h[p]) / P
        if smoothing:  # else an infinite margin would make 0 times infinity of it
            loss += smoothing * np.logaddexp(0.0, h[p]) / P
        slope = beta / P * (np.exp(-np.logaddexp(0.0, -h[p])) - (1 - smoothing))
        for i, sign in ((2 * p, 1.0), (2 * p + 1, -1.0)):
            for m in range(int(offsets[i]), int(offsets[i + 1])):
                if float(weights[m]) != 0.0:
                    coef[m] = sign * slope * float(weights[m])
    return loss, h, logp, _gradient(y, targets, coef) * grad_scale, coef
