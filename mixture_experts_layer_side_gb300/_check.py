"""Checks of tensor arguments, shared by the wrappers whose calls take them
from serving and training code directly (the C ABI sees only pointers)."""

from __future__ import annotations

import torch

from . import _lib


class MokArgError(_lib.MokError, ValueError):
    """An argument the wrapper refuses before any call."""

    def __init__(self, what):
        _lib.MokError.__init__(self, 1, what)


def require(ok, what):
    if not ok:
        raise MokArgError(what)


def tensor(t, name, shape, dtypes, device, rows_apart=False):
    """``t`` is a tensor of this shape, one of these types, on this device and
    dense in row-major order (``rows_apart``: a matrix whose rows may be
    further apart than its columns)."""
    require(isinstance(t, torch.Tensor), f"{name}: a tensor is wanted")
    require(tuple(t.shape) == tuple(shape), f"{name}: shape {tuple(t.shape)}, wanted {tuple(shape)}")
    require(t.dtype in dtypes, f"{name}: {t.dtype}, wanted {' or '.join(str(d) for d in dtypes)}")
    require(t.device == device, f"{name}: on {t.device}, wanted {device}")
    if rows_apart:
        dense = t.shape[1] <= 1 or t.stride(1) == 1
        dense = dense and (t.shape[0] <= 1 or t.stride(0) >= t.shape[1])
    else:
        dense = t.is_contiguous()
    require(dense, f"{name}: strides {tuple(t.stride())} are not row-major")
    return t


def on(device):
    """``device`` with its index, as tensors name it."""
    d = torch.device(device)
    return torch.device(d.type, torch.cuda.current_device()) if d.type == "cuda" and d.index is None else d
