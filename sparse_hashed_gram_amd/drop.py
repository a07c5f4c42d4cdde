"""Python binding of counter-based dropout (ctypes).  Argument marshalling
only: every function forwards to the C ABI in ``include/drop.h`` of the same
name, inside the in-tree libngram.so; PyTorch supplies device memory and the
current HIP stream.  Importing this module raises if the library is missing.

    s = drop.spec(0.1, seed, offset)          # offset: another one for each dropped tensor
    y = drop.fwd(s, x, residual=r)            # r + dropout(x)
    dx = drop.bwd(s, dy)                      # the same mask again, never stored
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _marshal

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libngram.so")

DTYPE_F32 = 0
DTYPE_BF16 = 1
_U64 = 1 << 64
_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}


class DropSpec(ctypes.Structure):
    _fields_ = [
        ("p", ctypes.c_float),
        ("reserved", ctypes.c_int32),
        ("seed", ctypes.c_uint64),
        ("offset", ctypes.c_uint64),
        ("rng", ctypes.c_void_p),
    ]


class DropError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} (status {status})")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        vp, i64, i = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        sp = ctypes.POINTER(DropSpec)
        _lib = _marshal.library(_LIB_PATH, {
            "drop_abi_version": ([], i),
            "drop_status_string": ([i], ctypes.c_char_p),
            "drop_fwd": ([sp, vp, i, vp, vp, i, i64, i64, vp], i),
            "drop_bwd": ([sp, vp, i, vp, i, i64, i64, vp], i),
        })
    return _lib


lib()   # fail at import time if the HIP library is missing: there is no fallback


def status_string(status: int) -> str:
    return lib().drop_status_string(status).decode()


def rng_state(seed: int, offset: int, out: torch.Tensor | None = None, device="cuda") -> torch.Tensor:
    """A generator state in device memory (drop_rng: int64 [2], the bits of
    seed and offset), for spec(rng=...); written in place if `out` is given (an
    ordinary copy on the current stream)."""
    host = torch.tensor([_signed(seed), _signed(offset)], dtype=torch.int64)
    if out is None:
        out = torch.empty(2, dtype=torch.int64, device=device)
    out.copy_(host)
    return out


def _signed(v: int) -> int:
    v = int(v)
    if not 0 <= v < _U64:
        raise ValueError("seed and offset are 64-bit unsigned numbers")
    return v - (1 << 64) if v >> 63 else v


def spec(p: float, seed: int = 0, offset: int = 0, rng: torch.Tensor | None = None) -> DropSpec:
    """What to drop: the share p and the mask's seed and offset, or `rng`, a
    generator state in device memory (rng_state) that the kernels read when
    they run, so a captured graph replays with the mask of whatever it holds
    then.  Calls need offsets of their own, or they get the same mask."""
    seed, offset = int(seed), int(offset)
    if not (0 <= seed < _U64 and 0 <= offset < _U64):
        raise ValueError("seed and offset are 64-bit unsigned numbers")
    s = DropSpec(p, 0, seed, offset, None)
    if rng is not None:
        if rng.dtype != torch.int64 or rng.numel() != 2:
            raise ValueError("rng must be an int64 [2] tensor")
        s.rng = _marshal.ptr(rng, "rng", rng.device)
        s.rng_tensor = rng   # kept alive with the spec
    return s


def _check_rng(s: DropSpec, device: torch.device):
    if s.rng:
        t = getattr(s, "rng_tensor", None)   # None: a DropSpec filled in by hand
        if t is not None and t.device != device:
            raise ValueError(f"rng is on {t.device}, the call's other tensors on {device}")


def _dtype(t, name: str) -> int:
    if t not in _DTYPES:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t}")
    return _DTYPES[t]


def _rows_cols(x: torch.Tensor):
    """Rows are the last dimension's: any shape is taken as [rows][cols]."""
    if x.dim() == 0:
        raise ValueError("a dropped tensor has at least one dimension")
    cols = x.shape[-1]
    return (x.numel() // cols if cols else 0), cols


def fwd(s: DropSpec, x: torch.Tensor, residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
        out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """(residual +) dropout(x).  residual and the result have one dtype: out's,
    residual's, out_dtype, or x's, whichever is given first.  out may be x
    (same dtype) or residual."""
    dev = x.device
    yt = out.dtype if out is not None else residual.dtype if residual is not None else out_dtype or x.dtype
    rows, cols = _rows_cols(x)
    px = _marshal.ptr(x, "x", dev)
    dx, dy = _dtype(x.dtype, "x"), _dtype(yt, "the result")
    pr = None if residual is None else _marshal.ptr(residual, "residual", dev, yt, x.shape)
    if out is None:
        out = torch.empty_like(x, dtype=yt)
        po = out.data_ptr()
    else:
        po = _marshal.ptr(out, "out", dev, yt, x.shape)
    _check_rng(s, dev)
    rc = _marshal.enqueue(lib().drop_fwd, dev, s, px, dx, pr, po, dy, rows, cols)
    if rc:
        raise DropError("drop_fwd", rc)
    return out


def bwd(s: DropSpec, dy: torch.Tensor, out: torch.Tensor | None = None,
        out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """The gradient of x: dropout(dy) under the forward's spec.  out may be dy
    (same dtype)."""
    dev = dy.device
    xt = out.dtype if out is not None else out_dtype or dy.dtype
    rows, cols = _rows_cols(dy)
    py = _marshal.ptr(dy, "dy", dev)
    ty, tx = _dtype(dy.dtype, "dy"), _dtype(xt, "the result")
    if out is None:
        out = torch.empty_like(dy, dtype=xt)
        po = out.data_ptr()
    else:
        po = _marshal.ptr(out, "out", dev, xt, dy.shape)
    _check_rng(s, dev)
    rc = _marshal.enqueue(lib().drop_bwd, dev, s, py, ty, po, tx, rows, cols)
    if rc:
        raise DropError("drop_bwd", rc)
    return out
