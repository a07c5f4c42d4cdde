"""Python binding of the gated feed-forward block (ctypes).  Argument
marshalling only: every function forwards to the C ABI in ``include/ffn.h`` of
the same name, inside the in-tree libngram.so; PyTorch supplies device memory
and the current HIP stream.  Importing this module raises if the library is
missing.

    cfg = ffn.config(2048, max_tokens=T, act="silu")
    ws = ffn.Workspace(cfg)                                  # of the backward's size, serves both
    Y = ffn.fwd(cfg, ws, X, Wg, Wu, Wd, residual=R, drop=drop.spec(0.1, seed, offset))
    g = ffn.bwd(cfg, ws, X, Wg, Wu, Wd, dY, drop=...)        # dX, dWg, dWu, dWd
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _marshal
from .drop import DropSpec, _check_rng

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libngram.so")

DIM = 768

ACTS = {"silu": 0, "gelu": 1, "relu2": 2}
DTYPE_F32 = 0
DTYPE_BF16 = 1
_DTYPES = {"f32": DTYPE_F32, "bf16": DTYPE_BF16}
OPT_ACCUM = 0x1
PASS_FWD = 0
PASS_BWD = 1


class FfnConfig(ctypes.Structure):
    _fields_ = [
        ("dim", ctypes.c_int32),
        ("hidden", ctypes.c_int32),
        ("act", ctypes.c_int32),
        ("y_dtype", ctypes.c_int32),
        ("dw_dtype", ctypes.c_int32),
        ("options", ctypes.c_int32),
        ("max_tokens", ctypes.c_int64),
    ]

    @property
    def y_torch_dtype(self):
        return torch.float32 if self.y_dtype == DTYPE_F32 else torch.bfloat16

    @property
    def dw_torch_dtype(self):
        return torch.float32 if self.dw_dtype == DTYPE_F32 else torch.bfloat16


def config(hidden: int, max_tokens: int, act: str = "silu", y_dtype: str = "bf16", dw_dtype: str = "bf16",
           accumulate: bool = False) -> FfnConfig:
    """act: "silu", "gelu" (tanh form) or "relu2"; y_dtype: of the residual,
    Y, dY and dX; dw_dtype: of the weights' gradients; accumulate: bwd adds to
    the weight gradients it is given."""
    c = FfnConfig()
    c.dim = DIM
    c.hidden = int(hidden)
    c.act = ACTS[act]
    c.y_dtype = _DTYPES[y_dtype]
    c.dw_dtype = _DTYPES[dw_dtype]
    c.options = OPT_ACCUM if accumulate else 0
    c.max_tokens = int(max_tokens)
    return c


class FfnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} (status {status})")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        vp, i64, i, u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint64
        cp, sp = ctypes.POINTER(FfnConfig), ctypes.POINTER(DropSpec)
        _lib = _marshal.library(_LIB_PATH, {
            "ffn_abi_version": ([], i),
            "ffn_status_string": ([i], ctypes.c_char_p),
            "ffn_config_check": ([cp], i),
            "ffn_workspace_bytes": ([cp, i, vp], i),
            "ffn_fwd": ([cp, vp, u64, vp, vp, vp, vp, vp, sp, i64, vp, vp], i),
            "ffn_bwd": ([cp, vp, u64, vp, vp, vp, vp, vp, sp, i64, vp, vp, vp, vp, vp], i),
        })
    return _lib


lib()   # fail at import time if the HIP library is missing: there is no fallback


def status_string(status: int) -> str:
    return lib().ffn_status_string(status).decode()


def _check(fn: str, status: int):
    if status != 0:
        raise FfnError(fn, status)


def config_check(cfg: FfnConfig) -> int:
    return lib().ffn_config_check(ctypes.byref(cfg))


def workspace_bytes(cfg: FfnConfig, backward: bool = True) -> int:
    n = ctypes.c_uint64()
    _check("ffn_workspace_bytes", lib().ffn_workspace_bytes(ctypes.byref(cfg), PASS_BWD if backward else PASS_FWD,
                                                            ctypes.byref(n)))
    return int(n.value)


class Workspace:
    """Device workspace (a uint8 tensor, 256-byte aligned); backward=False:
    of the forward's size only (serving)."""

    def __init__(self, cfg: FfnConfig, device="cuda", backward: bool = True):
        self.cfg = cfg
        self.nbytes = workspace_bytes(cfg, backward)
        self._buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device)
        off = (-self._buf.data_ptr()) % 256
        self.tensor = self._buf[off:off + self.nbytes]
        self.ptr = self.tensor.data_ptr()


def _weights(cfg: FfnConfig, Wg, Wu, Wd, dev, dtype, prefix=""):
    up, down = (cfg.hidden, DIM), (DIM, cfg.hidden)
    return (_marshal.ptr(Wg, prefix + "Wg", dev, dtype, up), _marshal.ptr(Wu, prefix + "Wu", dev, dtype, up),
            _marshal.ptr(Wd, prefix + "Wd", dev, dtype, down))


def _common(ws: Workspace, X: torch.Tensor, drop: DropSpec | None):
    dev = X.device
    if X.dim() != 2:
        raise ValueError(f"X must have shape (T, {DIM}), got {tuple(X.shape)}")
    if X.is_cuda and ws.tensor.device != dev:
        raise ValueError(f"the workspace is on {ws.tensor.device}, X on {dev}")
    if drop is not None:
        _check_rng(drop, dev)
    return dev, X.shape[0]


def fwd(cfg: FfnConfig, ws: Workspace, X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor,
        residual: torch.Tensor | None = None, drop: DropSpec | None = None,
        out: torch.Tensor | None = None) -> torch.Tensor:
    """Y = (residual +) dropout((a(X Wg^T) * (X Wu^T)) Wd^T).  X: bf16 [T, 768];
    Wg, Wu: bf16 [F, 768]; Wd: bf16 [768, F]; residual and Y: [T, 768] of
    cfg.y_dtype.  out may be residual."""
    dev, T = _common(ws, X, drop)
    px = _marshal.ptr(X, "X", dev, torch.bfloat16, (T, DIM))
    pg, pu, pd = _weights(cfg, Wg, Wu, Wd, dev, torch.bfloat16)
    pr = None if residual is None else _marshal.ptr(residual, "residual", dev, cfg.y_torch_dtype, (T, DIM))
    if out is None:
        out = torch.empty_like(X, dtype=cfg.y_torch_dtype)
        po = out.data_ptr()
    else:
        po = _marshal.ptr(out, "out", dev, cfg.y_torch_dtype, (T, DIM))
    _check("ffn_fwd", _marshal.enqueue(lib().ffn_fwd, dev, cfg, ws.ptr, ws.nbytes, px, pg, pu, pd, pr, drop, T, po))
    return out


def bwd(cfg: FfnConfig, ws: Workspace, X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor,
        dY: torch.Tensor, drop: DropSpec | None = None, dX: torch.Tensor | None = None,
        dWg: torch.Tensor | None = None, dWu: torch.Tensor | None = None,
        dWd: torch.Tensor | None = None) -> dict[str, torch.Tensor]:
    """The gradients {"dX", "dWg", "dWu", "dWd"} under the forward's inputs and
    drop (dY, dX: [T, 768] of cfg.y_dtype).  The residual's gradient is dY.
    With cfg's accumulate the weight gradients must be given; they are added
    to."""
    dev, T = _common(ws, X, drop)
    px = _marshal.ptr(X, "X", dev, torch.bfloat16, (T, DIM))
    pg, pu, pd = _weights(cfg, Wg, Wu, Wd, dev, torch.bfloat16)
    py = _marshal.ptr(dY, "dY", dev, cfg.y_torch_dtype, (T, DIM))
    wt = cfg.dw_torch_dtype
    if cfg.options & OPT_ACCUM and (dWg is None or dWu is None or dWd is None):
        raise ValueError("an accumulating backward needs the gradients it adds to: dWg, dWu, dWd")
    if dX is None:
        dX = torch.empty_like(dY)
    if dWg is None:
        dWg = torch.empty_like(Wg, dtype=wt)
    if dWu is None:
        dWu = torch.empty_like(Wu, dtype=wt)
    if dWd is None:
        dWd = torch.empty_like(Wd, dtype=wt)
    _check("ffn_bwd", _marshal.enqueue(
        lib().ffn_bwd, dev, cfg, ws.ptr, ws.nbytes, px, pg, pu, pd, py, drop, T,
        _marshal.ptr(dX, "dX", dev, cfg.y_torch_dtype, (T, DIM)), *_weights(cfg, dWg, dWu, dWd, dev, wt, "d")))
    return {"dX": dX, "dWg": dWg, "dWu": dWu, "dWd": dWd}
