"""The norms around a block, written plainly in numpy float64 (formulas in
include/norm.h).  Shares no code with the HIP path."""
from __future__ import annotations

import numpy as np


def _f(a):
    return None if a is None else np.asarray(a, np.float64)


def norm(x, kind: str, eps: float):
    """(xh, rho) of each row."""
    x = _f(x)
    mu = x.mean(1, keepdims=True) if kind == "layer" else 0.0
    rho = 1.0 / np.sqrt(((x - mu) ** 2).mean(1, keepdims=True) + eps)
    return (x - mu) * rho, rho


def affine(xh, w=None, b=None):
    y = xh if w is None else xh * _f(w)
    return y if b is None else y + _f(b)


def forward(R, kind, eps, w=None, b=None):
    return affine(norm(R, kind, eps)[0], w, b)


def sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0, e) / (1.0 + e)


def _gamma(gate, token):
    return np.float64(1.0) if gate is None else sigmoid(_f(gate)) if token else _f(gate)


def join(R, B, kind, eps, post=True, post_w=None, post_b=None, gate=None, token=False, scale=None, w=None, b=None):
    """(R1, X)."""
    N = affine(norm(B, kind, eps)[0], post_w, post_b) if post else _f(B)
    R1 = (1.0 if scale is None else _f(scale)) * _f(R) + _gamma(gate, token) * N
    return R1, forward(R1, kind, eps, w, b)


def _through(xh, rho, d, kind):
    out = d - xh * (d * xh).mean(1, keepdims=True)
    return rho * (out - d.mean(1, keepdims=True) if kind == "layer" else out)


def backward(R, dX, kind, eps, w=None, dR1=None):
    """{"dR", "dw", "db"}."""
    xh, rho = norm(R, kind, eps)
    dX = _f(dX)
    dR = _through(xh, rho, affine(dX, w), kind)
    return {"dR": dR if dR1 is None else _f(dR1) + dR, "dw": (dX * xh).sum(0), "db": dX.sum(0)}


def join_backward(R, B, R1, dX, dR1, kind, eps, pre=True, post=True, post_w=None, post_b=None, gate=None, token=False,
                  scale=None, w=None):
    """All gradients, of a scalar gate or scale (shape [1]) too."""
    out = {}
    if pre:
        g = backward(R1, dX, kind, eps, w, dR1)
        E, out["dw"], out["db"] = g["dR"], g["dw"], g["db"]
    else:
        E = _f(dR1)
    out["dR"] = E if scale is None else E * _f(scale)
    if scale is not None:
        ds = (E * _f(R)).sum(0)
        out["dscale"] = ds.sum(keepdims=True) if np.size(scale) == 1 and E.shape[1] != 1 else ds
    if post:
        nh, rho = norm(B, kind, eps)
        N = affine(nh, post_w, post_b)
    else:
        N = _f(B)
    gam = _gamma(gate, token)
    if gate is not None and token:
        out["dgate"] = E * N * gam * sigmoid(-_f(gate))
    elif gate is not None:
        dg = (E * N).sum(0)
        out["dgate"] = dg.sum(keepdims=True) if np.size(gate) == 1 and E.shape[1] != 1 else dg
    dN = E * gam
    if post:
        out["dpost_w"], out["dpost_b"] = (dN * nh).sum(0), dN.sum(0)
        out["dB"] = _through(nh, rho, affine(dN, post_w), kind)
    else:
        out["dB"] = dN
    return out
