"""Python binding of the gated linear recurrence (ctypes).  Argument marshalling
only: every function forwards to the C ABI in ``include/recur.h`` of the same
name, inside the in-tree libngram.so; PyTorch supplies device memory and the
current HIP stream.  Importing this module raises if the library is missing.

    cfg = recur.config(768, max_tokens=T)
    ws = recur.Workspace(cfg)                        # of the backward's size, serves both
    y, _, saved = recur.fwd(cfg, ws, x, r, i, lam, offsets=starts, keep=True)
    g = recur.bwd(cfg, ws, x, r, i, lam, saved, dy, offsets=starts)       # dx, dr, di, dlam
    y, state, _ = recur.fwd(cfg, ws, x, r, i, lam, offsets=starts, final=True)   # a prompt
    y = recur.step(cfg, x1, r1, i1, lam, state)      # one token of each sequence, state in place
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _marshal

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libngram.so")

DTYPE_F32 = 0
DTYPE_BF16 = 1
_DTYPES = {"f32": DTYPE_F32, "bf16": DTYPE_BF16}
_TORCH = (torch.float32, torch.bfloat16)
OPT_ACCUM = 0x1
PASS_FWD = 0
PASS_BWD = 1
CHUNK = 32


class RecurConfig(ctypes.Structure):
    _fields_ = [
        ("dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("c", ctypes.c_float),
        ("options", ctypes.c_int32),
        ("max_tokens", ctypes.c_int64),
    ]


class RecurInputs(ctypes.Structure):
    _fields_ = ([(k, ctypes.c_void_p) for k in ("x", "r", "i")] + [(k, ctypes.c_int64) for k in ("ldx", "ldr", "ldi")])


class RecurGrads(ctypes.Structure):
    _fields_ = ([(k, ctypes.c_void_p) for k in ("dx", "dr", "di")]
                + [(k, ctypes.c_int64) for k in ("lddx", "lddr", "lddi")])


def config(dim: int, max_tokens: int, dtype: str = "bf16", c: float = 8.0, accumulate: bool = False) -> RecurConfig:
    """dtype: of x, r, i, y and their gradients; c: the decay's factor;
    accumulate: bwd adds to the dlam it is given."""
    f = RecurConfig()
    f.dim = int(dim)
    f.dtype = _DTYPES[dtype]
    f.c = c
    f.options = OPT_ACCUM if accumulate else 0
    f.max_tokens = int(max_tokens)
    return f


class RecurError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} (status {status})")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        vp, i64, i, u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint64
        cp, ip, gp = ctypes.POINTER(RecurConfig), ctypes.POINTER(RecurInputs), ctypes.POINTER(RecurGrads)
        _lib = _marshal.library(_LIB_PATH, {
            "recur_abi_version": ([], i),
            "recur_status_string": ([i], ctypes.c_char_p),
            "recur_config_check": ([cp], i),
            "recur_workspace_bytes": ([cp, i, vp], i),
            "recur_saved_bytes": ([cp, i64, vp], i),
            "recur_fwd": ([cp, vp, u64, ip, vp, vp, i64, vp, i64, vp, vp, vp, vp], i),
            "recur_bwd": ([cp, vp, u64, ip, vp, vp, i64, vp, vp, vp, vp, i64, gp, vp, vp, vp], i),
            "recur_step": ([cp, ip, vp, vp, i64, vp, i64, vp, vp], i),
        })
    return _lib


lib()   # fail at import time if the HIP library is missing: there is no fallback


def status_string(status: int) -> str:
    return lib().recur_status_string(status).decode()


def _check(fn: str, status: int):
    if status != 0:
        raise RecurError(fn, status)


def config_check(cfg: RecurConfig) -> int:
    return lib().recur_config_check(ctypes.byref(cfg))


def workspace_bytes(cfg: RecurConfig, backward: bool = True) -> int:
    n = ctypes.c_uint64()
    _check("recur_workspace_bytes", lib().recur_workspace_bytes(
        ctypes.byref(cfg), PASS_BWD if backward else PASS_FWD, ctypes.byref(n)))
    return int(n.value)


class Workspace:
    """Device workspace (a uint8 tensor, 256-byte aligned); backward=False:
    of the forward's size only (serving)."""

    def __init__(self, cfg: RecurConfig, device="cuda", backward: bool = True):
        self.cfg = cfg
        self.nbytes = workspace_bytes(cfg, backward)
        self._buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device)
        off = (-self._buf.data_ptr()) % 256
        self.tensor = self._buf[off:off + self.nbytes]
        self.ptr = self.tensor.data_ptr()


def _columns(t: torch.Tensor, name: str, dev, dtype, shape):
    """(address, distance between rows) of a [T, D] tensor whose rows are contiguous."""
    if t.is_cuda and t.device == dev and t.dtype is dtype and t.shape == shape:
        rows, one = t.stride()
        if one == 1 or shape[1] <= 1 or shape[0] == 0:
            return t.data_ptr(), shape[1] if shape[0] <= 1 else rows
        raise ValueError(f"the rows of {name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _inputs(cfg: RecurConfig, x, r, i, lam):
    if x.dim() != 2 or x.shape[1] != cfg.dim:
        raise ValueError(f"x must have shape (T, {cfg.dim}), got {tuple(x.shape)}")
    dev, shape, dt = x.device, x.shape, _TORCH[cfg.dtype]
    px, lx = _columns(x, "x", dev, dt, shape)
    pr, lr = _columns(r, "r", dev, dt, shape)
    pi, li = _columns(i, "i", dev, dt, shape)
    return dev, shape, dt, RecurInputs(px, pr, pi, lx, lr, li), _marshal.ptr(lam, "lam", dev, torch.float32, (cfg.dim,))


def _sequences(cfg: RecurConfig, ws: Workspace, dev, offsets, h0):
    """(address of offsets, number of sequences, shape of their states, address of h0)."""
    if ws.tensor.device != dev:
        raise ValueError(f"the workspace is on {ws.tensor.device}, x on {dev}")
    n, po = 1, None
    if offsets is not None:
        if offsets.dim() != 1 or offsets.numel() < 1:
            raise ValueError(f"offsets must have shape (n + 1,), got {tuple(offsets.shape)}")
        n = offsets.numel() - 1
        po = _marshal.ptr(offsets, "offsets", dev, torch.int32)
    shape = (n, cfg.dim)
    return po, n, shape, None if h0 is None else _marshal.ptr(h0, "h0", dev, torch.float32, shape)


def _result(t, name, dev, dtype, shape):
    """(the tensor, its address) of a result, allocated if it is not given."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=dev)
        return t, t.data_ptr()
    return t, _marshal.ptr(t, name, dev, dtype, shape)


def _rows(t, name, x, dt):
    """The same for [T, D] rows shaped as x (empty_like of contiguous rows: 1 us less)."""
    if t is None and x.is_contiguous():
        t = torch.empty_like(x)
        return t, t.data_ptr()
    return _result(t, name, x.device, dt, x.shape)


def fwd(cfg: RecurConfig, ws: Workspace, x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, lam: torch.Tensor,
        offsets: torch.Tensor | None = None, h0: torch.Tensor | None = None, keep: bool = False,
        final: bool = False, out: torch.Tensor | None = None):
    """(y, hT, saved).  x, r, i: [T, D] of cfg's dtype, rows contiguous (columns of
    one tensor will do); lam: fp32 [D]; offsets: int32 [n + 1] or None for one
    sequence; h0, hT: fp32 [n, D].  hT is None unless final, saved (for bwd) unless
    keep.  Rows of y outside the sequences are left as they were (uninitialised
    unless out is given)."""
    dev, shape, dt, inputs, pl = _inputs(cfg, x, r, i, lam)
    po, n, states, ph = _sequences(cfg, ws, dev, offsets, h0)
    out, py = _rows(out, "out", x, dt)
    hT = saved = pT = ps = None
    if final:
        hT = torch.empty(states, dtype=torch.float32, device=dev)
        pT = hT.data_ptr()
    if keep:
        saved = torch.empty(((shape[0] + CHUNK - 1) // CHUNK, cfg.dim), dtype=torch.float32, device=dev)
        ps = saved.data_ptr()
    rc = _marshal.enqueue(lib().recur_fwd, dev, cfg, ws.ptr, ws.nbytes, inputs, pl, po, n, ph, shape[0], py, pT, ps)
    if rc:
        raise RecurError("recur_fwd", rc)
    return out, hT, saved


def bwd(cfg: RecurConfig, ws: Workspace, x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, lam: torch.Tensor,
        saved: torch.Tensor, dy: torch.Tensor, offsets: torch.Tensor | None = None, h0: torch.Tensor | None = None,
        dhT: torch.Tensor | None = None, dx: torch.Tensor | None = None, dr: torch.Tensor | None = None,
        di: torch.Tensor | None = None, dlam: torch.Tensor | None = None,
        dh0: torch.Tensor | None = None) -> dict[str, torch.Tensor]:
    """{"dx", "dr", "di", "dlam"}, and "dh0" where h0 is given, under the forward's
    inputs and its saved.  dx, dr, di may be columns of one tensor.  With cfg's
    accumulate dlam must be given; it is added to."""
    dev, shape, dt, inputs, pl = _inputs(cfg, x, r, i, lam)
    po, n, states, ph = _sequences(cfg, ws, dev, offsets, h0)
    ps = _marshal.ptr(saved, "saved", dev, torch.float32, ((shape[0] + CHUNK - 1) // CHUNK, cfg.dim))
    pd = _marshal.ptr(dy, "dy", dev, dt, shape)
    pT = None if dhT is None else _marshal.ptr(dhT, "dhT", dev, torch.float32, states)
    if cfg.options & OPT_ACCUM and dlam is None:
        raise ValueError("an accumulating backward needs the gradient it adds to: dlam")
    if dh0 is not None and h0 is None:
        raise ValueError("dh0 is the gradient of an h0 that is not given")
    got, at = {}, []
    for name, t in (("dx", dx), ("dr", dr), ("di", di)):
        if t is None:
            got[name], p = _rows(None, name, x, dt)
            at.append((p, shape[1]))
        else:
            got[name] = t
            at.append(_columns(t, name, dev, dt, shape))
    g = RecurGrads(*(p for p, _ in at), *(ld for _, ld in at))
    got["dlam"], pm = _rows(dlam, "dlam", lam, torch.float32)
    p0 = None
    if h0 is not None:
        got["dh0"], p0 = _result(dh0, "dh0", dev, torch.float32, states)
    rc = _marshal.enqueue(lib().recur_bwd, dev, cfg, ws.ptr, ws.nbytes, inputs, pl, po, n, ph, ps, pd, pT, shape[0], g,
                          pm, p0)
    if rc:
        raise RecurError("recur_bwd", rc)
    return got


def step(cfg: RecurConfig, x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, lam: torch.Tensor, state: torch.Tensor,
         slots: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """y [n, D]: the next position of each row's state, which moves on in place.
    x, r, i: [n, D]; state: fp32 [states, D]; slots: int32 [n], the row of state
    (None: its own); a slot outside the states is an unused row, its y is 0; rows
    of the same slot follow one another."""
    dev, shape, dt, inputs, pl = _inputs(cfg, x, r, i, lam)
    if state.dim() != 2 or state.shape[1] != cfg.dim:
        raise ValueError(f"state must have shape (states, {cfg.dim}), got {tuple(state.shape)}")
    p = _marshal.ptr(state, "state", dev, torch.float32)
    pk = None if slots is None else _marshal.ptr(slots, "slots", dev, torch.int32, (shape[0],))
    out, py = _rows(out, "out", x, dt)
    rc = _marshal.enqueue(lib().recur_step, dev, cfg, inputs, pl, p, state.shape[0], pk, shape[0], py)
    if rc:
        raise RecurError("recur_step", rc)
    return out
