"""Loading of the library, shared by the bindings, and the checks of tensors and
the stream of a call of ``drop``, ``ffn`` and ``ngram.embed_fwd_drop``.

A call runs on its tensors' device, on that device's current stream, whatever
device is current in the calling thread."""
from __future__ import annotations

import ctypes
import os

import torch

# the stream's handle without the object around it (2 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def library(path: str, signatures: dict) -> ctypes.CDLL:
    """The library at `path` with {name: (argument types, result type)} set."""
    if not os.path.exists(path):
        raise RuntimeError(f"libngram is not built ({path} missing): run "
                           "`python -m sparse_hashed_gram_amd.build`")
    L = ctypes.CDLL(path)
    for name, (args, res) in signatures.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    return L


def ptr(t: torch.Tensor, name: str, device: torch.device, dtype=None, shape=None) -> int:
    """The address of a contiguous GPU tensor on `device`, after the checks."""
    if (t.is_cuda and t.device == device and t.is_contiguous() and (dtype is None or t.dtype is dtype)
            and (shape is None or t.shape == shape)):
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def enqueue(f, device: torch.device, *args) -> int:
    """f(*args, stream) on the device's current stream; its status."""
    if device.index == _device():
        return f(*args, _raw_stream(device.index))
    with torch.cuda.device(device):
        return f(*args, _raw_stream(device.index))
