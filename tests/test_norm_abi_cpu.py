"""CPU checks of the norms' C ABI (include/norm.h): exports, layout, and refusals
before any HIP call."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "norm.h")
WS = 1 << 40
A = [(k + 1) << 30 for k in range(20)]      # fake device addresses, far apart


@pytest.fixture(scope="module")
def N():
    from sparse_hashed_gram_amd import norm
    return norm


def test_exports_layout_version(N):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(norm_[a-z_]+)\s*\(", src)))
    assert names == ["norm_abi_version", "norm_bwd", "norm_config_check", "norm_fwd", "norm_join_bwd", "norm_join_fwd",
                     "norm_status_string", "norm_workspace_bytes"]
    for n in names:
        assert hasattr(N.lib(), n)
    assert N.lib().norm_abi_version() == 1
    assert ctypes.sizeof(N.NormConfig) == 40 and N.NormConfig.eps.offset == 36
    assert ctypes.sizeof(N.NormParams) == 48 and ctypes.sizeof(N.NormGrads) == 48
    for s in range(-6, 1):
        assert N.status_string(s) not in ("", "unknown status")
    assert N.status_string(-99) == "unknown status"


@pytest.mark.parametrize("field,value", [
    ("dim", 0), ("dim", 4097), ("dim", -3), ("kind", 2), ("kind", -1), ("x_dtype", 2), ("r_dtype", -1), ("p_dtype", 2),
    ("dp_dtype", 5), ("gate", 4), ("gate", -1), ("scale", 3), ("scale", -1), ("options", 8), ("eps", 0.0), ("eps", -1.0),
    ("eps", 2.0), ("eps", float("nan")), ("eps", 1e-13)])
def test_config_rejects(N, field, value):
    c = N.config(768, gate="vector")
    assert N.config_check(c) == 0
    setattr(c, field, value)
    L = N.lib()
    n = ctypes.c_uint64()
    assert N.config_check(c) == -3 and L.norm_workspace_bytes(ctypes.byref(c), ctypes.byref(n)) == -3
    p, g = N.NormParams(), N.NormGrads()
    assert L.norm_fwd(c, A[0], None, None, 4, A[1], None) == -3
    assert L.norm_bwd(c, WS, 1 << 30, A[0], A[1], None, None, 4, A[2], None, None, None) == -3
    assert L.norm_join_fwd(c, A[0], A[1], p, 4, A[2], A[3], None) == -3
    assert L.norm_join_bwd(c, WS, 1 << 30, A[0], A[1], A[2], A[3], None, p, 4, A[4], A[5], g, None) == -3


def test_config_types(N):
    assert N.config_check(N.config(768, x_dtype="f32", r_dtype="f32")) == 0
    assert N.config_check(N.config(768, x_dtype="f32", r_dtype="bf16")) == -3
    assert N.config_check(N.config(768, x_dtype="bf16", r_dtype="bf16")) == 0
    assert N.lib().norm_config_check(None) == -1


def test_workspace_bytes(N):
    for D in (1, 768, 1001, 4096):
        assert 0 < N.workspace_bytes(N.config(D)) <= 10300 * (D + 3) + 1024
    assert N.lib().norm_workspace_bytes(N.config(8), None) == -1


def test_norm_refusals(N):
    L, c = N.lib(), N.config(64)
    f = L.norm_fwd
    assert f(None, A[0], None, None, 4, A[1], None) == -1
    assert f(c, None, None, None, 4, A[1], None) == -1
    assert f(c, A[0], None, None, 4, None, None) == -1
    assert f(c, A[0] + 2, None, None, 4, A[1], None) == -2     # fp32 at a 2-byte address
    assert f(c, A[0], A[2] + 2, None, 4, A[1], None) == -2
    assert f(c, A[0], None, A[2] + 1, 4, A[1], None) == -2
    assert f(c, A[0], None, None, 4, A[1] + 1, None) == -2
    assert f(c, A[0], None, None, -1, A[1], None) == -4
    assert f(c, A[0], None, None, 1 << 31, A[1], None) == -4
    assert f(c, A[0], None, None, 4, A[0] + 64, None) == -5
    assert f(c, A[0], A[1] + 8, None, 4, A[1], None) == -5     # w inside the result
    assert f(c, None, None, None, 0, None, None) == 0
    need = N.workspace_bytes(c)
    g = L.norm_bwd

    def bwd(ws=WS, n=need, R=A[0], dX=A[1], dR1=None, w=A[3], T=4, dR=A[4], dw=A[5], db=A[6]):
        return g(c, ws, n, R, dX, dR1, w, T, dR, dw, db, None)

    assert bwd(ws=None) == -1 and bwd(R=None) == -1 and bwd(dX=None) == -1 and bwd(dR=None) == -1
    assert bwd(ws=WS + 128) == -2 and bwd(n=need - 1) == -4 and bwd(T=-1) == -4
    assert bwd(dw=A[5] + 2) == -2
    assert bwd(dR=A[0]) == -5 and bwd(dR=A[1]) == -5 and bwd(dR1=A[4] + 64) == -5
    assert bwd(dw=A[6]) == -5 and bwd(dw=A[4]) == -5 and bwd(dw=WS + 512) == -5 and bwd(R=WS) == -5
    assert g(None, WS, need, A[0], A[1], None, None, 4, A[4], None, None, None) == -1


def test_join_refusals(N):
    L, c = N.lib(), N.config(64, gate="token", scale="vector")
    need = N.workspace_bytes(c)
    P, G = N.NormParams, N.NormGrads
    p = dict(post_w=A[6], post_b=A[7], gate=A[8], scale=A[9], w=A[10], b=A[11])

    def fwd(R=A[0], B=A[1], T=4, R1=A[2], X=A[3], **kw):
        return L.norm_join_fwd(c, R, B, P(**{**p, **kw}), T, R1, X, None)

    for k in ("R", "B", "R1", "X", "gate", "scale"):
        assert fwd(**{k: None}) == -1, k
    for k in ("R", "R1", "post_w", "post_b", "scale", "w", "b"):
        assert fwd(**{k: A[15] + 2}) == -2, k
    assert fwd(gate=A[15] + 1) == -2
    assert fwd(T=-1) == -4
    assert fwd(R1=A[1]) == -5 and fwd(R1=A[0] + 4) == -5 and fwd(X=A[0]) == -5 and fwd(X=A[2] + 8) == -5
    assert fwd(gate=A[3]) == -5 and fwd(w=A[2]) == -5
    assert L.norm_join_fwd(c, A[0], A[1], None, 4, A[2], A[3], None) == -1
    assert fwd(R=None, B=None, R1=None, X=None, gate=None, T=0) == 0

    gr = dict(dpost_w=A[12], dpost_b=A[13], dgate=A[14], dscale=A[15], dw=A[16], db=A[17])

    def bwd(ws=WS, n=need, R=A[0], B=A[1], R1=A[2], dX=A[3], dR1=None, T=4, dR=A[4], dB=A[5], cfg=c, **kw):
        q = P(**{k: kw.get(k, v) for k, v in p.items()})
        h = G(**{k: kw.get(k, v) for k, v in gr.items()})
        return L.norm_join_bwd(cfg, ws, n, R, B, R1, dX, dR1, q, T, dR, dB, h, None)

    for k in ("ws", "R", "B", "R1", "dX", "dR", "dB", "gate", "scale"):
        assert bwd(**{k: None}) == -1, k
    assert bwd(ws=WS + 8) == -2 and bwd(n=need - 1) == -4 and bwd(T=1 << 31) == -4
    for k in gr:
        assert bwd(**{k: A[18] + 1}) == -2, k
    for k in ("dB", "dgate", "dw"):
        assert bwd(**{k: A[0]}) == -5, k
        assert bwd(**{k: WS + 256}) == -5, k
    assert bwd(dB=A[4] + 64) == -5 and bwd(dR=A[2]) == -5 and bwd(dR1=A[4] + 4) == -5 and bwd(dw=A[17]) == -5
    nopre = N.config(64, gate="token", scale="vector", pre=False)
    assert bwd(cfg=nopre) == -1        # no gradient comes in at all
    assert L.norm_join_bwd(c, WS, need, A[0], A[1], A[2], A[3], None, None, 4, A[4], A[5], G(), None) == -1
    assert L.norm_join_bwd(c, WS, need, A[0], A[1], A[2], A[3], None, P(), 4, A[4], A[5], None, None) == -1


def test_binding_refuses(N):
    c = N.config(8, gate="vector", scale="scalar")
    t = torch.zeros(3, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        N.fwd(c, t)
    with pytest.raises(ValueError, match="shape"):
        N.fwd(c, torch.zeros(3, 9))
    with pytest.raises(ValueError, match="shape"):
        N.fwd(c, torch.zeros(8))
    with pytest.raises(KeyError):
        N.config(8, kind="mean")
    with pytest.raises(KeyError):
        N.config(8, x_dtype="f16")
    w = object.__new__(N.Workspace)
    w.tensor = torch.zeros(1)
    with pytest.raises(ValueError, match="scale needs R"):
        N.join_bwd(c, w, None, t, t, t)
    with pytest.raises(ValueError, match="R1 and dX"):
        N.join_bwd(N.config(8), w, None, t, None, t)
    with pytest.raises(ValueError, match="dR1 is needed"):
        N.join_bwd(N.config(8, pre=False), w, None, t, None, None)
