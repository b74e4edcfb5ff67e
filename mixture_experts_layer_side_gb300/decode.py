"""The layer for a few tokens of a serving step (mok_few_*; no compute here)."""

from __future__ import annotations

import torch

from . import _lib
from ._check import on, require, tensor
from .inputs import Shape
from .layer import PRECISIONS


class MoKDecoder:
    """Owns the workspace of the few-token layer for up to ``shape.T`` tokens
    (at most 128); a call takes any number from 0 to that.

    Weights as for ``MoKLayer.forward``: bf16 tensors, or in MXFP8 mode the
    forward descriptors of ``quantize_weights``.  Calls on one object must not
    overlap (they share the workspace).  Errors found on the device (an expert
    id outside [0, E)) are raised by ``check``."""

    def __init__(self, shape: Shape, precision="bf16", device="cuda"):
        self.shape = shape
        self.prec = PRECISIONS[precision]
        self.device = on(device)
        n = _lib.mok_few_workspace_size(_lib.shape_of(shape.T, shape.H, shape.I, shape.E, shape.k), self.prec)
        if n == 0:
            raise _lib.MokError(2, "unsupported shape")
        self.ws = torch.zeros(n, dtype=torch.uint8, device=self.device)

    def _weights(self, W1, W3, W2):
        s = self.shape
        for name, W, rows, cols in (("W1", W1, s.H, s.I), ("W3", W3, s.H, s.I), ("W2", W2, s.I, s.H)):
            if self.prec == _lib.MOK_BF16:
                tensor(W, name, (s.E, rows, cols), (torch.bfloat16,), self.device)
            else:
                require(isinstance(W, _lib.MokMx), f"{name}: an MXFP8 descriptor is wanted")

    def _begin(self, x, out):
        s = self.shape
        require(isinstance(x, torch.Tensor) and x.dim() == 2 and x.shape[0] <= s.T,
                f"x: at most {s.T} rows of {s.H} are wanted")
        T = x.shape[0]
        tensor(x, "x", (T, s.H), (torch.bfloat16,), self.device)
        if out is None:
            out = torch.empty((T, s.H), dtype=torch.bfloat16, device=self.device)
        tensor(out, "out", (T, s.H), (torch.bfloat16,), self.device)
        return T, out, _lib.shape_of(T, s.H, s.I, s.E, s.k)

    def forward(self, x, topk_idx, scores, W1, W3, W2, out=None, stream=None):
        """out [T, H] for the routing given (int32 ids and f32 scores [T, k])."""
        T, out, cshape = self._begin(x, out)
        self._weights(W1, W3, W2)
        tensor(topk_idx, "topk_idx", (T, self.shape.k), (torch.int32,), self.device)
        tensor(scores, "scores", (T, self.shape.k), (torch.float32,), self.device)
        if T:
            _lib.mok_few_forward(cshape, self.prec, self.ws, topk_idx, x, scores, W1, W3, W2, out, stream)
        return out

    def layer(self, x, Wr, W1, W3, W2, bias=None, out=None, stream=None):
        """(out, topk_idx, scores), the router included: Wr bf16 [H, E], bias
        f32 [E] or None (selection only)."""
        s = self.shape
        T, out, cshape = self._begin(x, out)
        self._weights(W1, W3, W2)
        tensor(Wr, "Wr", (s.H, s.E), (torch.bfloat16,), self.device)
        if bias is not None:
            tensor(bias, "bias", (s.E,), (torch.float32,), self.device)
        idx = torch.empty((T, s.k), dtype=torch.int32, device=self.device)
        scores = torch.empty((T, s.k), dtype=torch.float32, device=self.device)
        if T:
            _lib.mok_few_layer(cshape, self.prec, self.ws, x, Wr, bias, W1, W3, W2, idx, scores, out, stream)
        return out, idx, scores

    def check(self, stream=None):
        """Synchronise and raise if the device recorded an error."""
        st = _lib.mok_check(self.ws, stream)
        if st != 0:
            raise _lib.MokError(st, "few tokens: device status")
