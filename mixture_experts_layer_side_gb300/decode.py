"""The layer for a few tokens of a serving step (mok_few_*; no compute here)."""

from __future__ import annotations

import math

import torch

from . import _lib
from ._check import away, fits, on, require, run_on, tensor, workspace
from .inputs import Shape
from .layer import PRECISIONS


class MoKDecoder:
    """Owns the workspace of the few-token layer for up to ``shape.T`` tokens
    (at most 128); a call takes any number from 0 to that.

    Weights as for ``MoKLayer.forward``: bf16 tensors, or in MXFP8 mode the
    forward descriptors of ``quantize_weights`` (or of ``_lib.mx``; one that was
    filled with bare addresses names no tensors to check).  Calls on one object must not
    overlap (they share the workspace).  Errors found on the device (an expert
    id outside [0, E)) are raised by ``check``.  After a timeout the results
    of all calls since the last ``check`` are void; ``check`` raises it and
    makes the workspace ready again."""

    def __init__(self, shape: Shape, precision="bf16", device="cuda"):
        self.shape = shape
        self.prec = PRECISIONS[precision]
        self.device = on(device)
        cshape = _lib.shape_of(shape.T, shape.H, shape.I, shape.E, shape.k)
        self.ws = workspace(lambda: _lib.mok_few_workspace_size(cshape, self.prec), self.device, "unsupported shape")
        self._w13, self._w2 = (shape.E, shape.H, shape.I), (shape.E, shape.I, shape.H)
        self._mx13, self._mx2 = (((E, r, c), (E, r // 32, c), self.device) for E, r, c in (self._w13, self._w2))

    def _weights(self, W1, W3, W2):
        d, bf16 = self.device, torch.bfloat16
        if self.prec == _lib.MOK_BF16:
            if not (fits(W1, self._w13, bf16, d) and fits(W3, self._w13, bf16, d) and fits(W2, self._w2, bf16, d)):
                for name, W, shape in (("W1", W1, self._w13), ("W3", W3, self._w13), ("W2", W2, self._w2)):
                    tensor(W, name, shape, (bf16,), d)
        elif not (type(W1) is type(W3) is type(W2) is _lib.MokMx and
                  W1.made_of == W3.made_of == self._mx13 and W2.made_of == self._mx2):
            for name, W, (codes, scales, _) in (("W1", W1, self._mx13), ("W3", W3, self._mx13), ("W2", W2, self._mx2)):
                require(isinstance(W, _lib.MokMx), f"{name}: an MXFP8 descriptor is wanted")
                if W.tensors is None:
                    continue
                for part, t, shape in (("codes", W.tensors[0], codes), ("scales", W.tensors[1], scales)):
                    require(t.element_size() == 1, f"{name}: {part} of {t.dtype}, wanted bytes")
                    # (as one long row, or as a matrix, they are the same bytes)
                    same = t.dim() != 3 and t.is_contiguous() and t.numel() == math.prod(shape)
                    tensor(t.view(shape) if same else t, f"{name}: {part}", shape, (t.dtype,), d)

    def _begin(self, x, out):
        s, d = self.shape, self.device
        if type(x) is not torch.Tensor or x.dim() != 2 or x.shape[0] > s.T:
            require(isinstance(x, torch.Tensor) and x.dim() == 2 and x.shape[0] <= s.T,
                    f"x: at most {s.T} rows of {s.H} are wanted")
        T = x.shape[0]
        rows = (T, s.H)
        if not fits(x, rows, torch.bfloat16, d):
            tensor(x, "x", rows, (torch.bfloat16,), d)
        if out is None:
            out = torch.empty(rows, dtype=torch.bfloat16, device=d)
        elif not fits(out, rows, torch.bfloat16, d):
            tensor(out, "out", rows, (torch.bfloat16,), d)
        return T, out, _lib.shape_of(T, s.H, s.I, s.E, s.k)

    def forward(self, x, topk_idx, scores, W1, W3, W2, out=None, stream=None):
        """out [T, H] for the routing given (int32 ids and f32 scores [T, k])."""
        if away(self.device, stream):
            return run_on(self, stream, self.forward, x, topk_idx, scores, W1, W3, W2, out)
        T, out, cshape = self._begin(x, out)
        self._weights(W1, W3, W2)
        rows, d = (T, self.shape.k), self.device
        if not (fits(topk_idx, rows, torch.int32, d) and fits(scores, rows, torch.float32, d)):
            tensor(topk_idx, "topk_idx", rows, (torch.int32,), d)
            tensor(scores, "scores", rows, (torch.float32,), d)
        if T:
            _lib.mok_few_forward(cshape, self.prec, self.ws, topk_idx, x, scores, W1, W3, W2, out, stream)
        return out

    def layer(self, x, Wr, W1, W3, W2, bias=None, out=None, stream=None):
        """(out, topk_idx, scores), the router included: Wr bf16 [H, E], bias
        f32 [E] or None (selection only)."""
        if away(self.device, stream):
            return run_on(self, stream, self.layer, x, Wr, W1, W3, W2, bias, out)
        s, d = self.shape, self.device
        T, out, cshape = self._begin(x, out)
        self._weights(W1, W3, W2)
        if not fits(Wr, (s.H, s.E), torch.bfloat16, d):
            tensor(Wr, "Wr", (s.H, s.E), (torch.bfloat16,), d)
        if bias is not None and not fits(bias, (s.E,), torch.float32, d):
            tensor(bias, "bias", (s.E,), (torch.float32,), d)
        idx = torch.empty((T, s.k), dtype=torch.int32, device=d)
        scores = torch.empty((T, s.k), dtype=torch.float32, device=d)
        if T:
            _lib.mok_few_layer(cshape, self.prec, self.ws, x, Wr, bias, W1, W3, W2, idx, scores, out, stream)
        return out, idx, scores

    def check(self, stream=None):
        """Synchronise and raise if the device recorded an error."""
        if away(self.device, stream):
            return run_on(self, stream, self.check)
        st = _lib.mok_check(self.ws, stream)
        if st == _lib.MOK_ERR_TIMEOUT:
            # a call that gave up leaves the abort word and counts of arrivals behind
            self.ws.zero_()
            if self.device.type == "cuda":
                torch.cuda.current_stream(self.device).synchronize()
        if st != 0:
            raise _lib.MokError(st, "few tokens: device status")
