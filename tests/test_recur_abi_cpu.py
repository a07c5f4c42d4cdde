"""CPU checks of the recurrence's C ABI (include/recur.h): exports, layout, and
refusals before any HIP call."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "recur.h")
WS = 1 << 44
A = [(k + 1) << 32 for k in range(20)]      # fake device addresses, far apart


@pytest.fixture(scope="module")
def M():
    from sparse_hashed_gram_amd import recur
    return recur


def test_exports_layout_version(M):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(recur_[a-z_]+)\s*\(", src)))
    assert names == ["recur_abi_version", "recur_bwd", "recur_config_check", "recur_fwd", "recur_saved_bytes",
                     "recur_status_string", "recur_step", "recur_workspace_bytes"]
    for n in names:
        assert hasattr(M.lib(), n)
    assert M.lib().recur_abi_version() == 1
    assert ctypes.sizeof(M.RecurConfig) == 24 and M.RecurConfig.max_tokens.offset == 16
    assert ctypes.sizeof(M.RecurInputs) == 48 and ctypes.sizeof(M.RecurGrads) == 48
    assert int(re.search(r"#define RECUR_CHUNK (\d+)", src)[1]) == M.CHUNK
    for s in range(-6, 1):
        assert M.status_string(s) not in ("", "unknown status")
    assert M.status_string(-99) == "unknown status"


@pytest.mark.parametrize("field,value", [
    ("dim", 0), ("dim", 16385), ("dtype", 2), ("dtype", -1), ("c", 0.0), ("c", -1.0), ("c", 65.0), ("c", float("nan")),
    ("options", 2), ("max_tokens", 0), ("max_tokens", (1 << 24) + 1)])
def test_config_rejects(M, field, value):
    c = M.config(768, 100)
    assert M.config_check(c) == 0
    setattr(c, field, value)
    L, n, i, g = M.lib(), ctypes.c_uint64(), M.RecurInputs(), M.RecurGrads()
    assert M.config_check(c) == -3
    assert L.recur_workspace_bytes(c, 0, ctypes.byref(n)) == -3 and L.recur_saved_bytes(c, 8, ctypes.byref(n)) == -3
    assert L.recur_fwd(c, WS, 1 << 40, i, A[0], None, 1, None, 8, A[1], None, None, None) == -3
    assert L.recur_bwd(c, WS, 1 << 40, i, A[0], None, 1, None, A[1], A[2], None, 8, g, A[3], None, None) == -3
    assert L.recur_step(c, i, A[0], A[1], 8, None, 8, A[2], None) == -3


def test_sizes(M):
    c = M.config(768, 49152)
    f, b = M.workspace_bytes(c, False), M.workspace_bytes(c)
    assert 0 < f <= b <= 768 * 49152 * 0.41 + (1 << 16)
    n, L = ctypes.c_uint64(), M.lib()
    assert L.recur_workspace_bytes(c, 2, ctypes.byref(n)) == -5 and L.recur_workspace_bytes(c, 0, None) == -1
    for T in (0, 1, M.CHUNK, M.CHUNK + 1, 49152):
        assert L.recur_saved_bytes(c, T, ctypes.byref(n)) == 0 and n.value == -(-T // M.CHUNK) * 768 * 4
    assert L.recur_saved_bytes(c, 49153, ctypes.byref(n)) == -4 and L.recur_saved_bytes(c, -1, ctypes.byref(n)) == -4
    assert L.recur_saved_bytes(c, 1, None) == -1


def test_forward_refusals(M):
    L, c = M.lib(), M.config(64, 100)
    need = M.workspace_bytes(c, False)

    def call(ws=WS, nb=need, x=A[0], r=A[1], i=A[2], ldx=64, ldr=64, ldi=64, lam=A[3], off=A[4], n=3, h0=A[5], T=100,
             y=A[6], hT=A[7], saved=A[8]):
        return L.recur_fwd(c, ws, nb, M.RecurInputs(x, r, i, ldx, ldr, ldi), lam, off, n, h0, T, y, hT, saved, None)

    assert L.recur_fwd(None, WS, need, M.RecurInputs(), A[3], None, 1, None, 8, A[6], None, None, None) == -1
    assert L.recur_fwd(c, WS, need, None, A[3], None, 1, None, 8, A[6], None, None, None) == -1
    for k in ("ws", "x", "r", "i", "lam", "y"):
        assert call(**{k: None}) == -1, k
    for k in ("x", "r", "i", "y"):
        assert call(**{k: A[9] + 1}) == -2, k
    for k in ("ws", "lam", "off", "h0", "hT", "saved"):
        assert call(**{k: A[9] + 2}) == -2, k
    assert call(ws=A[9] + 128) == -2
    assert call(T=101) == -4 and call(T=-1) == -4 and call(n=-1) == -4 and call(n=(1 << 24) + 1) == -4
    assert call(off=None) == -4 and call(off=None, n=0) == -4
    for k in ("ldx", "ldr", "ldi"):
        assert call(**{k: 63}) == -4 and call(**{k: 1 << 31}) == -4, k
    assert call(nb=need - 1) == -4
    for k in ("y", "hT", "saved"):
        for bad in (A[0], A[0] + 2 * 64 * 100 - 64, A[3], A[4], A[5], WS):
            assert call(**{k: bad}) == -5, (k, bad)
    assert call(y=A[7]) == -5 and call(hT=A[8]) == -5 and call(x=WS) == -5
    assert call(n=0, off=A[4], y=A[6]) == 0       # no sequence, nothing to do


def test_backward_refusals(M):
    L, c = M.lib(), M.config(64, 100)
    need = M.workspace_bytes(c)

    def call(ws=WS, nb=need, x=A[0], r=A[1], i=A[2], lam=A[3], off=A[4], n=3, h0=A[5], saved=A[6], dy=A[7], dhT=A[8],
             T=100, dx=A[9], dr=A[10], di=A[11], lddx=64, lddr=64, lddi=64, dlam=A[12], dh0=A[13]):
        return L.recur_bwd(c, ws, nb, M.RecurInputs(x, r, i, 64, 64, 64), lam, off, n, h0, saved, dy, dhT, T,
                           M.RecurGrads(dx, dr, di, lddx, lddr, lddi), dlam, dh0, None)

    for k in ("ws", "x", "r", "i", "lam", "saved", "dy", "dx", "dr", "di", "dlam"):
        assert call(**{k: None}) == -1, k
    for k in ("lam", "off", "h0", "saved", "dhT", "dlam", "dh0"):
        assert call(**{k: A[14] + 2}) == -2, k
    for k in ("dy", "dx", "dr", "di"):
        assert call(**{k: A[14] + 1}) == -2, k
    assert call(T=101) == -4 and call(lddx=63) == -4 and call(lddr=0) == -4 and call(lddi=-64) == -4
    assert call(nb=need - 1) == -4 and call(off=None) == -4
    for k in ("dx", "dr", "di", "dlam", "dh0"):
        for bad in (A[0], A[2], A[3], A[5], A[6], A[7], A[8], WS + 128 * 256):
            if bad == WS + 128 * 256 and need <= 128 * 256:
                continue
            assert call(**{k: bad}) == -5, (k, bad)
    assert call(dx=A[10]) == -5 and call(dlam=A[13]) == -5
    assert L.recur_bwd(c, WS, need, M.RecurInputs(A[0], A[1], A[2], 64, 64, 64), A[3], None, 1, None, A[6], A[7], None, 8,
                       None, A[12], None, None) == -1
    # columns of one array: side by side is apart, one element nearer is not
    e = 2
    assert call(dx=A[9], dr=A[9] + 64 * e, di=A[9] + 127 * e, lddx=192, lddr=192, lddi=192) == -5
    assert call(dx=A[9], dr=A[9] + 63 * e, di=A[9] + 128 * e, lddx=192, lddr=192, lddi=192) == -5
    assert call(dx=A[9], dr=A[9] + 64 * e, di=A[9] + 129 * e, lddx=192, lddr=192, lddi=192) == -5   # wraps onto dx's next row
    assert call(dx=A[9], dr=A[9] + 64 * e, di=A[11], lddx=192, lddr=200, lddi=192) == -5             # rows drift apart


def test_too_many_pieces(M):
    # T and D in their ranges, but over 2^23 - 1 blocks
    c = M.config(16384, 1 << 24)
    n = M.workspace_bytes(c)
    i = M.RecurInputs(1 << 50, 1 << 51, 1 << 52, 16384, 16384, 16384)
    assert M.lib().recur_fwd(c, 1 << 53, n, i, A[0], None, 1, None, 1 << 24, 1 << 54, None, None, None) == -4
    g = M.RecurGrads(1 << 55, 1 << 56, 1 << 57, 16384, 16384, 16384)
    assert M.lib().recur_bwd(c, 1 << 53, n, i, A[0], None, 1, None, 1 << 58, 1 << 54, None, 1 << 24, g, A[1], None,
                             None) == -4
    # the backward of fp32 takes half the channels to a block: too many where the forward's are not
    f = M.config(1024, 1 << 24, "f32")
    n, g = M.workspace_bytes(f), M.RecurGrads(1 << 55, 1 << 56, 1 << 57, 1024, 1024, 1024)
    i = M.RecurInputs(1 << 50, 1 << 51, 1 << 52, 1024, 1024, 1024)
    assert M.lib().recur_bwd(f, 1 << 53, n, i, A[0], None, 1, None, 1 << 58, 1 << 54, None, 1 << 24, g, A[1], None,
                             None) == -4


def test_step_refusals(M):
    L, c = M.lib(), M.config(64, 100)

    def call(x=A[0], r=A[1], i=A[2], ldx=64, lam=A[3], state=A[4], states=50, slots=A[5], n=20, y=A[6]):
        return L.recur_step(c, M.RecurInputs(x, r, i, ldx, 64, 64), lam, state, states, slots, n, y, None)

    for k in ("x", "r", "i", "lam", "state", "y"):
        assert call(**{k: None}) == -1, k
    assert L.recur_step(None, M.RecurInputs(), A[3], A[4], 4, None, 4, A[6], None) == -1
    assert L.recur_step(c, None, A[3], A[4], 4, None, 4, A[6], None) == -1
    for k in ("lam", "state", "slots"):
        assert call(**{k: A[7] + 2}) == -2, k
    assert call(n=-1) == -4 and call(n=(1 << 16) + 1) == -4 and call(states=-1) == -4 and call(ldx=63) == -4
    assert call(slots=None, states=19) == -4
    for k in ("y", "state"):
        for bad in (A[0], A[1] + 64, A[3], A[5]):
            assert call(**{k: bad}) == -5, (k, bad)
    assert call(y=A[4] + 256) == -5
    assert call(n=0) == 0


def test_binding_refuses(M):
    c = M.config(8, 10)
    t, lam = torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(8)
    w = object.__new__(M.Workspace)
    w.tensor = t
    with pytest.raises(ValueError, match="GPU tensor"):
        M.fwd(c, w, t, t, t, lam)
    with pytest.raises(ValueError, match="shape"):
        M.fwd(c, w, torch.zeros(3, 9), t, t, lam)
    with pytest.raises(ValueError, match="GPU tensor"):
        M.step(c, t, t, t, lam, torch.zeros(3, 8))
    with pytest.raises(KeyError):
        M.config(8, 10, dtype="f16")
