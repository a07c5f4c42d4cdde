"""Python binding of the norms around a block (ctypes).  Argument marshalling
only: every function forwards to the C ABI in ``include/norm.h`` of the same
name, inside the in-tree libngram.so; PyTorch supplies device memory and the
current HIP stream.  Importing this module raises if the library is missing.

    cfg = norm.config(768, kind="rms", gate="token")         # fp32 residual stream, bf16 blocks
    X = norm.fwd(cfg, R, w)                                  # in front of a block
    R1, X1 = norm.join_fwd(cfg, R, B, post_w=pw, gate=G, w=w1)   # behind it, and in front of the next
    ws = norm.Workspace(cfg)
    g = norm.join_bwd(cfg, ws, None, B, R1, dX1, dR1, post_w=pw, gate=G, w=w1)  # dR, dB, dgate, dpost_w, dw
    h = norm.bwd(cfg, ws, R, dX, w, dR1=g["dR"])             # dR, dw
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _marshal

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libngram.so")

KINDS = {"rms": 0, "layer": 1}
DTYPE_F32 = 0
DTYPE_BF16 = 1
_DTYPES = {"f32": DTYPE_F32, "bf16": DTYPE_BF16}
_TORCH = (torch.float32, torch.bfloat16)
BY = {"none": 0, "scalar": 1, "vector": 2, "token": 3}
OPT_PRE = 0x1
OPT_POST = 0x2
OPT_ACCUM = 0x4


class NormConfig(ctypes.Structure):
    _fields_ = [
        ("dim", ctypes.c_int32),
        ("kind", ctypes.c_int32),
        ("x_dtype", ctypes.c_int32),
        ("r_dtype", ctypes.c_int32),
        ("p_dtype", ctypes.c_int32),
        ("dp_dtype", ctypes.c_int32),
        ("gate", ctypes.c_int32),
        ("scale", ctypes.c_int32),
        ("options", ctypes.c_int32),
        ("eps", ctypes.c_float),
    ]


class NormParams(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("post_w", "post_b", "gate", "scale", "w", "b")]


class NormGrads(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("dpost_w", "dpost_b", "dgate", "dscale", "dw", "db")]


def config(dim: int, kind: str = "rms", x_dtype: str = "bf16", r_dtype: str = "f32", p_dtype: str = "f32",
           dp_dtype: str = "f32", gate: str = "none", scale: str = "none", pre: bool = True, post: bool = True,
           eps: float = 1e-6, accumulate: bool = False) -> NormConfig:
    """kind: "rms" or "layer"; x_dtype: of the blocks' inputs and outputs and of
    a token gate; r_dtype: of the residual stream ("f32" where x_dtype is);
    p_dtype, dp_dtype: of the parameters and their gradients; gate: "none",
    "scalar", "vector" or "token" (sigmoid of a [T, D] tensor); scale: of the
    residual stream, "none", "scalar" or "vector"; pre, post: the join has the
    norm in front of the next block, of the block's output; accumulate: the
    backward adds to the parameters' gradients it is given."""
    c = NormConfig()
    c.dim = int(dim)
    c.kind = KINDS[kind]
    c.x_dtype = _DTYPES[x_dtype]
    c.r_dtype = _DTYPES[r_dtype]
    c.p_dtype = _DTYPES[p_dtype]
    c.dp_dtype = _DTYPES[dp_dtype]
    c.gate = BY[gate]
    c.scale = BY[scale]
    c.options = (OPT_PRE if pre else 0) | (OPT_POST if post else 0) | (OPT_ACCUM if accumulate else 0)
    c.eps = eps
    return c


class NormError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} (status {status})")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        vp, i64, i, u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint64
        cp, pp, gp = ctypes.POINTER(NormConfig), ctypes.POINTER(NormParams), ctypes.POINTER(NormGrads)
        _lib = _marshal.library(_LIB_PATH, {
            "norm_abi_version": ([], i),
            "norm_status_string": ([i], ctypes.c_char_p),
            "norm_config_check": ([cp], i),
            "norm_workspace_bytes": ([cp, vp], i),
            "norm_fwd": ([cp, vp, vp, vp, i64, vp, vp], i),
            "norm_bwd": ([cp, vp, u64, vp, vp, vp, vp, i64, vp, vp, vp, vp], i),
            "norm_join_fwd": ([cp, vp, vp, pp, i64, vp, vp, vp], i),
            "norm_join_bwd": ([cp, vp, u64, vp, vp, vp, vp, vp, pp, i64, vp, vp, gp, vp], i),
        })
    return _lib


lib()   # fail at import time if the HIP library is missing: there is no fallback


def status_string(status: int) -> str:
    return lib().norm_status_string(status).decode()


def _check(fn: str, status: int):
    if status != 0:
        raise NormError(fn, status)


def config_check(cfg: NormConfig) -> int:
    return lib().norm_config_check(ctypes.byref(cfg))


def workspace_bytes(cfg: NormConfig) -> int:
    n = ctypes.c_uint64()
    _check("norm_workspace_bytes", lib().norm_workspace_bytes(ctypes.byref(cfg), ctypes.byref(n)))
    return int(n.value)


class Workspace:
    """Device workspace of the backward (a uint8 tensor, 256-byte aligned)."""

    def __init__(self, cfg: NormConfig, device="cuda"):
        self.cfg = cfg
        self.nbytes = workspace_bytes(cfg)
        self._buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device)
        off = (-self._buf.data_ptr()) % 256
        self.tensor = self._buf[off:off + self.nbytes]
        self.ptr = self.tensor.data_ptr()


def _rows(t: torch.Tensor, cfg: NormConfig, name: str):
    if t.dim() != 2 or t.shape[1] != cfg.dim:
        raise ValueError(f"{name} must have shape (T, {cfg.dim}), got {tuple(t.shape)}")
    return t.device, t.shape


def _opt(t, name, dev, dtype, shape):
    return None if t is None else _marshal.ptr(t, name, dev, dtype, shape)


def _result(t, name, dev, dtype, shape):
    """(the tensor, its address) of a result, allocated if it is not given."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=dev)
        return t, t.data_ptr()
    return t, _marshal.ptr(t, name, dev, dtype, shape)


def _like(t, name, like, dtype):
    """The same for a result shaped as a tensor of the call (empty_like: 1 us less)."""
    if t is None:
        t = torch.empty_like(like, dtype=dtype)
        return t, t.data_ptr()
    return t, _marshal.ptr(t, name, like.device, dtype, like.shape)


def _by_shape(cfg: NormConfig, by: int, shape):
    return shape if by == 3 else (cfg.dim,) if by == 2 else (1,)


def _params(cfg: NormConfig, dev, shape, post_w, post_b, gate, scale, w, b) -> NormParams:
    pt, col = _TORCH[cfg.p_dtype], (cfg.dim,)
    if (gate is None) != (cfg.gate == 0):
        raise ValueError("gate has to be given where the config names one, and only there")
    if (scale is None) != (cfg.scale == 0):
        raise ValueError("scale has to be given where the config names one, and only there")
    if not cfg.options & OPT_POST and (post_w is not None or post_b is not None):
        raise ValueError("the config has no norm behind the block: post_w and post_b do not belong to it")
    if not cfg.options & OPT_PRE and (w is not None or b is not None):
        raise ValueError("the config has no norm in front of the next block: w and b do not belong to it")
    return NormParams(
        _opt(post_w, "post_w", dev, pt, col), _opt(post_b, "post_b", dev, pt, col),
        _opt(gate, "gate", dev, _TORCH[cfg.x_dtype] if cfg.gate == 3 else pt, _by_shape(cfg, cfg.gate, shape)),
        _opt(scale, "scale", dev, pt, _by_shape(cfg, cfg.scale, shape)),
        _opt(w, "w", dev, pt, col), _opt(b, "b", dev, pt, col))


def _check_ws(ws: Workspace, t: torch.Tensor):
    if t.is_cuda and ws.tensor.device != t.device:
        raise ValueError(f"the workspace is on {ws.tensor.device}, the call's tensors on {t.device}")


def fwd(cfg: NormConfig, R: torch.Tensor, w: torch.Tensor | None = None, b: torch.Tensor | None = None,
        out: torch.Tensor | None = None) -> torch.Tensor:
    """X = norm(R; w, b).  R: [T, D] of cfg's r_dtype, X of its x_dtype."""
    dev, shape = _rows(R, cfg, "R")
    pt, col = _TORCH[cfg.p_dtype], (cfg.dim,)
    pr = _marshal.ptr(R, "R", dev, _TORCH[cfg.r_dtype])
    pw, pb = _opt(w, "w", dev, pt, col), _opt(b, "b", dev, pt, col)
    out, po = _like(out, "out", R, _TORCH[cfg.x_dtype])
    rc = _marshal.enqueue(lib().norm_fwd, dev, cfg, pr, pw, pb, shape[0], po)
    if rc:
        raise NormError("norm_fwd", rc)
    return out


def _grad(g, name, like, cfg, dev, shape, got):
    """The address of a parameter's gradient; None where there is no parameter."""
    if like is None:
        if g is not None:
            raise ValueError(f"{name} is the gradient of a parameter that is not given")
        return None
    if g is None and cfg.options & OPT_ACCUM:
        raise ValueError(f"an accumulating backward needs the gradients it adds to: {name}")
    dt = _TORCH[cfg.dp_dtype]
    g, p = _like(g, name, like, dt) if like.shape == shape else _result(g, name, dev, dt, shape)
    got[name] = g
    return p


def bwd(cfg: NormConfig, ws: Workspace, R: torch.Tensor, dX: torch.Tensor, w: torch.Tensor | None = None,
        b: torch.Tensor | None = None, dR1: torch.Tensor | None = None, dR: torch.Tensor | None = None,
        dw: torch.Tensor | None = None, db: torch.Tensor | None = None) -> dict[str, torch.Tensor]:
    """{"dR", "dw", "db"} (those of the parameters that are given) under the
    forward's inputs.  dR = dR1 + the gradient through the norm; dR may be dR1."""
    dev, shape = _rows(R, cfg, "R")
    _check_ws(ws, R)
    rt, col = _TORCH[cfg.r_dtype], (cfg.dim,)
    pr = _marshal.ptr(R, "R", dev, rt)
    px = _marshal.ptr(dX, "dX", dev, _TORCH[cfg.x_dtype], shape)
    p1 = _opt(dR1, "dR1", dev, rt, shape)
    pw = _opt(w, "w", dev, _TORCH[cfg.p_dtype], col)
    _opt(b, "b", dev, _TORCH[cfg.p_dtype], col)
    dR, po = _like(dR, "dR", R, rt)
    got = {"dR": dR}
    gw, gb = _grad(dw, "dw", w, cfg, dev, col, got), _grad(db, "db", b, cfg, dev, col, got)
    _check("norm_bwd", _marshal.enqueue(lib().norm_bwd, dev, cfg, ws.ptr, ws.nbytes, pr, px, p1, pw, shape[0], po,
                                        gw, gb))
    return got


def join_fwd(cfg: NormConfig, R: torch.Tensor, B: torch.Tensor, post_w: torch.Tensor | None = None,
             post_b: torch.Tensor | None = None, gate: torch.Tensor | None = None,
             scale: torch.Tensor | None = None, w: torch.Tensor | None = None, b: torch.Tensor | None = None,
             out_R: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """(R1, X): R1 = scale R + g norm(B; post_w, post_b), X = norm(R1; w, b) (None
    without cfg's pre).  gate: [1], [D], or [T, D] before its sigmoid; scale: [1]
    or [D].  out_R may be R."""
    dev, shape = _rows(R, cfg, "R")
    rt, xt = _TORCH[cfg.r_dtype], _TORCH[cfg.x_dtype]
    pr = _marshal.ptr(R, "R", dev, rt)
    pb = _marshal.ptr(B, "B", dev, xt, shape)
    p = _params(cfg, dev, shape, post_w, post_b, gate, scale, w, b)
    out_R, p1 = _like(out_R, "out_R", R, rt)
    px = None
    if cfg.options & OPT_PRE:
        out, px = _like(out, "out", R, xt)
    elif out is not None:
        raise ValueError("the config has no norm in front of the next block: there is no out")
    rc = _marshal.enqueue(lib().norm_join_fwd, dev, cfg, pr, pb, p, shape[0], p1, px)
    if rc:
        raise NormError("norm_join_fwd", rc)
    return out_R, out


def join_bwd(cfg: NormConfig, ws: Workspace, R: torch.Tensor | None, B: torch.Tensor, R1: torch.Tensor | None,
             dX: torch.Tensor | None, dR1: torch.Tensor | None = None, post_w: torch.Tensor | None = None,
             post_b: torch.Tensor | None = None, gate: torch.Tensor | None = None,
             scale: torch.Tensor | None = None, w: torch.Tensor | None = None, b: torch.Tensor | None = None,
             dR: torch.Tensor | None = None, dB: torch.Tensor | None = None,
             grads: dict[str, torch.Tensor] | None = None) -> dict[str, torch.Tensor]:
    """{"dR", "dB"} and the gradients of the parameters that are given:
    "dpost_w", "dpost_b", "dgate", "dscale", "dw", "db" (written into grads where
    it has them).  R may be None without a scale; R1 and dX without cfg's pre;
    dR1, the gradient that reaches R1 from elsewhere, with it.  dR may be dR1."""
    dev, shape = _rows(B, cfg, "B")
    _check_ws(ws, B)
    rt, xt, pre = _TORCH[cfg.r_dtype], _TORCH[cfg.x_dtype], cfg.options & OPT_PRE
    if cfg.scale and R is None:
        raise ValueError("the gradient of scale needs R")
    if pre and (R1 is None or dX is None):
        raise ValueError("R1 and dX are needed where the config has the norm in front of the next block")
    if not pre and dR1 is None:
        raise ValueError("dR1 is needed where the config has no norm in front of the next block")
    pb = _marshal.ptr(B, "B", dev, xt)
    pr = _opt(R, "R", dev, rt, shape) if cfg.scale else None
    p1 = _opt(R1, "R1", dev, rt, shape) if pre else None
    px = _opt(dX, "dX", dev, xt, shape) if pre else None
    pd = _opt(dR1, "dR1", dev, rt, shape)
    p = _params(cfg, dev, shape, post_w, post_b, gate, scale, w, b)
    dR, po = _like(dR, "dR", B, rt)
    dB, qo = _like(dB, "dB", B, xt)
    got = {"dR": dR, "dB": dB}
    have = dict(grads or {})
    col = (cfg.dim,)
    if cfg.gate == 3:   # a whole tensor: overwritten, of x_dtype
        got["dgate"], pg = _like(have.pop("dgate", None), "dgate", B, xt)
    else:
        pg = _grad(have.pop("dgate", None), "dgate", gate, cfg, dev, _by_shape(cfg, cfg.gate, shape), got)
    g = NormGrads(
        _grad(have.pop("dpost_w", None), "dpost_w", post_w, cfg, dev, col, got),
        _grad(have.pop("dpost_b", None), "dpost_b", post_b, cfg, dev, col, got), pg,
        _grad(have.pop("dscale", None), "dscale", scale, cfg, dev, _by_shape(cfg, cfg.scale, shape), got),
        _grad(have.pop("dw", None), "dw", w, cfg, dev, col, got),
        _grad(have.pop("db", None), "db", b, cfg, dev, col, got))
    if have:
        raise ValueError(f"unknown gradients: {sorted(have)}")
    _check("norm_join_bwd", _marshal.enqueue(lib().norm_join_bwd, dev, cfg, ws.ptr, ws.nbytes, pr, pb, p1, px, pd, p,
                                             shape[0], po, qo, g))
    return got
