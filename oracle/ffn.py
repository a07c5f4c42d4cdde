"""The gated feed-forward block, written plainly in numpy float64 (formulas in
include/ffn.h).  Shares no code with the HIP path."""
from __future__ import annotations

import numpy as np


def act(g, kind: str):
    """(a(g), a'(g))."""
    if kind == "silu":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if kind == "gelu":
        c = np.sqrt(2.0 / np.pi)
        t = np.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)
    if kind == "relu2":
        r = np.maximum(g, 0.0)
        return r * r, 2.0 * r
    raise ValueError(kind)


def forward(X, Wg, Wu, Wd, kind: str, factor=None, res=None):
    """Y; factor: the dropout's 0 or c of each element ([T][D])."""
    X, Wg, Wu, Wd = (np.asarray(v, np.float64) for v in (X, Wg, Wu, Wd))
    y = (act(X @ Wg.T, kind)[0] * (X @ Wu.T)) @ Wd.T
    if factor is not None:
        y = y * factor
    return y if res is None else y + np.asarray(res, np.float64)


def backward(X, Wg, Wu, Wd, dY, kind: str, factor=None):
    """{"dX", "dWg", "dWu", "dWd"}."""
    X, Wg, Wu, Wd, dY = (np.asarray(v, np.float64) for v in (X, Wg, Wu, Wd, dY))
    if factor is not None:
        dY = dY * factor
    G, U = X @ Wg.T, X @ Wu.T
    a, da = act(G, kind)
    dH = dY @ Wd
    dG, dU = dH * U * da, dH * a
    return {"dX": dG @ Wg + dU @ Wu, "dWg": dG.T @ X, "dWu": dU.T @ X, "dWd": dY.T @ (a * U)}
