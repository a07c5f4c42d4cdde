"""The gated linear recurrence, written plainly in numpy float64, position by
position (formulas in include/recur.h).  Shares no code with the HIP path."""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def gates(r, i, lam, c):
    """(a, m, g, rho)."""
    rho = sigmoid(np.asarray(r, np.float64))
    z = -c * softplus(np.asarray(lam, np.float64)) * rho
    return np.exp(z), np.sqrt(-np.expm1(2.0 * z)), sigmoid(np.asarray(i, np.float64)), rho


def _spans(T, offsets):
    return [(0, T)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))


def forward(x, r, i, lam, c, offsets=None, h0=None):
    """(h [T][D], 0 outside the sequences; hT [n][D]; h_{t-1} [T][D])."""
    x = np.asarray(x, np.float64)
    a, m, g, _ = gates(r, i, lam, c)
    T, D = x.shape
    spans = _spans(T, offsets)
    y, before, hT = np.zeros((T, D)), np.zeros((T, D)), np.zeros((len(spans), D))
    for k, (lo, hi) in enumerate(spans):
        h = np.zeros(D) if h0 is None else np.asarray(h0[k], np.float64)
        for t in range(lo, hi):
            before[t] = h
            h = a[t] * h + m[t] * g[t] * x[t]
            y[t] = h
        hT[k] = h
    return y, hT, before


def backward(x, r, i, lam, c, dy, offsets=None, h0=None, dhT=None):
    """{"dx", "dr", "di", "dlam", "dh0"}, 0 outside the sequences."""
    x, dy, lam = (np.asarray(v, np.float64) for v in (x, dy, lam))
    a, m, g, rho = gates(r, i, lam, c)
    T, D = x.shape
    spans = _spans(T, offsets)
    before = forward(x, r, i, lam, c, offsets, h0)[2]
    G, dh0 = np.zeros((T, D)), np.zeros((len(spans), D))
    for k, (lo, hi) in enumerate(spans):
        d = np.zeros(D) if dhT is None else np.asarray(dhT[k], np.float64)
        for t in range(hi - 1, lo - 1, -1):
            G[t] = dy[t] + d
            d = a[t] * G[t]
        dh0[k] = d
    with np.errstate(divide="ignore", invalid="ignore"):
        over = np.where(m > 0, a * a / m, 0.0)
    dz = a * G * before - G * g * x * over
    return {"dx": G * m * g, "di": G * m * x * g * (1.0 - g), "dr": -c * softplus(lam) * dz * rho * (1.0 - rho),
            "dlam": sigmoid(lam) * (-c * rho * dz).sum(0), "dh0": dh0}


def step(x, r, i, lam, c, state, slots=None):
    """(y, the states after it)."""
    x = np.asarray(x, np.float64)
    a, m, g, _ = gates(r, i, lam, c)
    state, y = np.array(state, np.float64), np.zeros(x.shape)
    for k in range(x.shape[0]):
        s = k if slots is None else int(slots[k])
        if 0 <= s < state.shape[0]:
            state[s] = y[k] = a[k] * state[s] + m[k] * g[k] * x[k]
    return y, state
