"""CPU checks of the feed-forward C ABI (include/ffn.h): exports, config
layout, and refusals before any HIP call."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ffn.h")
WS = 1 << 40
A = [(i + 1) << 30 for i in range(12)]      # fake device addresses, far apart


@pytest.fixture(scope="module")
def F():
    from sparse_hashed_gram_amd import ffn
    return ffn


def test_exports_layout_version(F):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ffn_[a-z_]+)\s*\(", src)))
    assert len(names) == 6
    for n in names:
        assert hasattr(F.lib(), n)
    assert F.lib().ffn_abi_version() == 1
    assert ctypes.sizeof(F.FfnConfig) == 32 and F.FfnConfig.max_tokens.offset == 24
    for s in range(-6, 1):
        assert F.status_string(s) not in ("", "unknown status")
    assert F.status_string(-99) == "unknown status"


@pytest.mark.parametrize("field,value", [("dim", 512), ("hidden", 0), ("hidden", 4), ("hidden", 2050),
                                         ("hidden", 65544), ("act", -1), ("act", 3), ("y_dtype", 2), ("dw_dtype", -1),
                                         ("options", 2), ("max_tokens", 0), ("max_tokens", (1 << 24) + 1)])
def test_config_rejects(F, field, value):
    c = F.config(2048, 256)
    assert F.config_check(c) == 0
    setattr(c, field, value)
    assert F.config_check(c) == -3
    n = ctypes.c_uint64()
    assert F.lib().ffn_workspace_bytes(ctypes.byref(c), 0, ctypes.byref(n)) == -3
    assert F.lib().ffn_fwd(c, WS, 1 << 34, *A[:4], None, None, 8, A[4], None) == -3
    assert F.lib().ffn_bwd(c, WS, 1 << 34, *A[:5], None, 8, *A[5:9], None) == -3


def test_workspace_bytes(F):
    c = F.config(2048, 49152)
    fwd, bwd = F.workspace_bytes(c, False), F.workspace_bytes(c)
    assert 2 * 49152 * 2048 <= fwd <= 2 * 49152 * 2048 + 33_600_000
    assert 6 * 49152 * 2048 < bwd <= 6 * 49152 * 2048 + 1536 * 49152 + 73728 * 2048 + 4096
    n = ctypes.c_uint64()
    assert F.lib().ffn_workspace_bytes(c, 2, ctypes.byref(n)) == -5
    assert F.lib().ffn_workspace_bytes(c, 0, None) == -1


def test_forward_rejections(F):
    from sparse_hashed_gram_amd import drop
    c = F.config(64, 256)
    n = F.workspace_bytes(c, False)
    f = F.lib().ffn_fwd

    def call(ws=WS, nbytes=n, X=A[0], Wg=A[1], Wu=A[2], Wd=A[3], res=None, d=None, T=100, Y=A[4]):
        return f(c, ws, nbytes, X, Wg, Wu, Wd, res, d, T, Y, None)

    assert f(None, WS, n, *A[:4], None, None, 100, A[4], None) == -1
    for k in ("ws", "X", "Wg", "Wu", "Wd", "Y"):
        assert call(**{k: None}) == -1, k
        assert call(**{k: A[9] + 8}) == -2, k
    assert call(res=A[9] + 4) == -2
    assert call(T=257) == -4 and call(T=-1) == -4
    assert call(nbytes=n - 1) == -4
    assert call(d=drop.DropSpec(1.5, 0, 0, 0, None)) == -5
    assert call(d=drop.DropSpec(0.5, 0, 0, 0, 8)) == -2
    assert call(Y=A[0]) == -5                       # Y over X
    assert call(Y=A[1] + 64) == -5                  # over a weight
    assert call(res=A[4] + 16) == -5                # res over part of Y
    assert call(Y=WS + 256) == -5 and call(X=WS) == -5 and call(res=WS + 16) == -5
    assert call(T=0, X=None, Y=None) == 0           # nothing to do


def test_backward_rejections(F):
    c = F.config(64, 256)
    n = F.workspace_bytes(c)
    f = F.lib().ffn_bwd
    names = ["X", "Wg", "Wu", "Wd", "dY", "dX", "dWg", "dWu", "dWd"]

    def call(nbytes=n, ws=WS, T=100, **kw):
        a = [kw.get(k, A[i]) for i, k in enumerate(names)]
        return f(c, ws, nbytes, *a[:5], None, T, *a[5:], None)

    for k in names:
        assert call(**{k: None}) == -1, k
        assert call(**{k: A[9] + 8}) == -2, k
    assert call(nbytes=F.workspace_bytes(c, False)) == -4
    assert call(T=257) == -4
    assert call(dX=A[4]) == -5                      # dX over dY
    assert call(dWg=A[7]) == -5                     # one buffer for two gradients
    assert call(dWd=A[3]) == -5
    c.options = 1
    assert call(T=0) == 0                           # accumulating nothing


def test_binding_refuses(F):
    with pytest.raises(KeyError):
        F.config(64, 8, act="tanh")
    c = F.config(64, 8)
    z = torch.zeros
    ws = type("W", (), {"tensor": z(1), "ptr": 0, "nbytes": 0})()
    with pytest.raises(ValueError, match="X must be a GPU tensor"):
        F.fwd(c, ws, z(4, 768, dtype=torch.bfloat16), z(64, 768), z(64, 768), z(768, 64))
    with pytest.raises(ValueError, match="X must have shape"):
        F.fwd(c, ws, z(768, dtype=torch.bfloat16), z(64, 768), z(64, 768), z(768, 64))


def test_generator_state_inside_results_or_workspace_is_refused(F):
    from sparse_hashed_gram_amd import drop
    c = F.config(64, 256)
    n = F.workspace_bytes(c)
    for at in (A[4], A[4] + 100 * 1536 - 16, WS + 512):
        assert F.lib().ffn_fwd(c, WS, n, *A[:4], None, drop.DropSpec(0.5, 0, 0, 0, at), 100, A[4], None) == -5
    for at in (A[5], A[6], A[7], A[8] + 64, WS + n - 16):
        assert F.lib().ffn_bwd(c, WS, n, *A[:5], drop.DropSpec(0.5, 0, 0, 0, at), 100, *A[5:9], None) == -5
