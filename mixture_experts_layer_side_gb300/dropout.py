"""Dropout whose mask is never stored (mok_dropout; no compute here)."""

from __future__ import annotations

import numbers

import torch

from . import _lib
from ._check import MokArgError, away, on, require, rows_fit, run_on, tensor

_TYPES = (torch.bfloat16, torch.float32)


class MoKDropout:
    """x / (1 - p) where an element is kept, else 0, for bf16 or f32 tensors:
    dense ones of any shape, or matrices whose rows are apart.  Which elements
    are kept follows from ``seed``, the number of the ``call`` and the
    element's place alone: the backward pass, with the same call, makes the
    mask again.  ``call`` is a whole number, or an int64 tensor of one element
    on the device, read when the kernel runs (a captured graph that counts it
    up gets another mask each time).  p is rounded to a multiple of 2^-16."""

    ws = None  # (nothing is kept between calls)

    def __init__(self, p, seed=0, device="cuda"):
        require(isinstance(p, numbers.Real) and 0.0 <= p <= 1.0, f"p: {p}, wanted a number from 0 to 1")
        require(isinstance(seed, numbers.Integral) and 0 <= seed < 2**64, f"seed: {seed}, wanted 64 bits")
        self.p, self.seed = float(p), int(seed)
        self.device = on(device)

    def drop(self, call):
        """The mok_drop of one call."""
        if isinstance(call, torch.Tensor):
            require(call.numel() == 1, "call: a tensor of one element is wanted")
            tensor(call, "call", call.shape, (torch.int64,), self.device)
            return _lib.mok_drop(self.p, self.seed, 0, call)
        if not ((type(call) is int or isinstance(call, numbers.Integral)) and 0 <= call < 2**63):
            raise MokArgError(f"call: {call}, wanted a whole number")
        return _lib.mok_drop(self.p, self.seed, int(call))

    def forward(self, x, call=0, out=None, stream=None):
        """A tensor like x, or ``out``, which may be x itself."""
        if away(self.device, stream):
            return run_on(self, stream, self.forward, x, call, out)
        d = self.device
        require(isinstance(x, torch.Tensor), "x: a tensor is wanted")
        matrix = x.dim() == 2
        if not (matrix and x.dtype in _TYPES and rows_fit(x, x.shape, x.dtype, d)):
            tensor(x, "x", x.shape, _TYPES, d, rows_apart=matrix)
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=d)
        elif not (matrix and rows_fit(out, x.shape, x.dtype, d)):
            tensor(out, "out", x.shape, (x.dtype,), d, rows_apart=matrix)
        drop = self.drop(call)
        if matrix:
            _lib.mok_dropout(x, drop, out, stream)
        else:
            _lib.mok_dropout(x.view(1, -1), drop, out.view(1, -1), stream)
        return out

    def backward(self, dout, call=0, out=None, stream=None):
        """The gradient of the forward's x from that of its result."""
        return self.forward(dout, call, out, stream)
