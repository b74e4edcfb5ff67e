"""Checks of tensor arguments, shared by the wrappers whose calls take them
from serving and training code directly (the C ABI sees only pointers)."""

from __future__ import annotations

import contextlib

import torch

from . import _lib

# (without the look whether CUDA is initialised: a call's tensors are there)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


class MokArgError(_lib.MokError, ValueError):
    """An argument the wrapper refuses before any call."""

    def __init__(self, what):
        _lib.MokError.__init__(self, 1, what)


def require(ok, what):
    if not ok:
        raise MokArgError(what)


def fits(t, shape, dtype, device):
    """Whether ``t`` is a dense tensor as described: what a call asks of its
    arguments each time, without the cost of saying what is wrong."""
    return (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.device == device and
            t.is_contiguous())


def rows_fit(t, shape, dtype, device):
    """As ``fits``, for a matrix whose rows may be further apart than its columns."""
    return (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.device == device and
            (t.is_contiguous() or ((t.stride(1) == 1 or shape[1] <= 1) and
                                   (t.stride(0) >= shape[1] or shape[0] <= 1))))


def tensor(t, name, shape, dtypes, device, rows_apart=False):
    """Raises unless ``t`` is a tensor of this shape, one of these types, on
    this device and dense in row-major order (``rows_apart``: see ``rows_fit``)."""
    require(isinstance(t, torch.Tensor), f"{name}: a tensor is wanted")
    require(tuple(t.shape) == tuple(shape), f"{name}: shape {tuple(t.shape)}, wanted {tuple(shape)}")
    require(t.dtype in dtypes, f"{name}: {t.dtype}, wanted {' or '.join(str(d) for d in dtypes)}")
    require(t.device == device, f"{name}: on {t.device}, wanted {device}")
    dense = t.is_contiguous()
    if rows_apart and not dense:
        dense = (t.stride(1) == 1 or t.shape[1] <= 1) and (t.stride(0) >= t.shape[1] or t.shape[0] <= 1)
    require(dense, f"{name}: strides {tuple(t.stride())} are not row-major")
    return t


def on(device):
    """``device`` with its index, as tensors name it."""
    d = torch.device(device)
    return torch.device(d.type, torch.cuda.current_device()) if d.type == "cuda" and d.index is None else d


def workspace(size, device, what):
    """size() bytes of zeros on ``device``, there for every stream.  (The size
    goes by the device's SMs: it is asked for with that device current.)"""
    with torch.cuda.device(device) if device.type == "cuda" else contextlib.nullcontext():
        n = size()
        if n == 0:
            raise _lib.MokError(2, what)
        ws = torch.zeros(n, dtype=torch.uint8, device=device)
        if device.type == "cuda" and not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()
    return ws


def _handle(stream):
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def away(device, stream):
    """Whether a call on ``device`` and ``stream`` (None: the current one) is
    to be made by ``run_on``: it is not on the current device and stream."""
    if device.type != "cuda":
        return False
    return (_current_device() != device.index or
            stream is not None and _handle(stream) != torch.cuda.current_stream().cuda_stream)


def run_on(owner, stream, call, *args):
    """call(*args) with the owner's device and ``stream`` current, as under
    torch.cuda.stream: what the call allocates is the stream's own, so that it
    takes no memory that another stream still reads, and what it returns may
    be used and dropped on the caller's stream."""
    d = owner.device
    if stream is None:
        with torch.cuda.device(d):
            return call(*args)
    if not isinstance(stream, torch.cuda.Stream):
        h = int(stream)
        stream = torch.cuda.default_stream(d) if h == 0 else torch.cuda.ExternalStream(h, device=d)
    require(stream.device == d, f"stream: on {stream.device}, wanted {d}")
    caller = torch.cuda.current_stream(d)
    if type(stream) is torch.cuda.Stream:  # (a foreign stream may be gone when the workspace is freed)
        for ws in (owner.ws, getattr(owner, "ctx", None)):
            if ws is not None:
                ws.record_stream(stream)
    with torch.cuda.stream(stream):
        got = call(*args)
    for t in got if isinstance(got, tuple) else got.values() if isinstance(got, dict) else (got,):
        if isinstance(t, torch.Tensor):  # (a dict is the caller's, who may keep other things in it)
            t.record_stream(caller)
    return got
