"""The join of a block with its residual stream (mok_residual_*; no compute here)."""

from __future__ import annotations

import math

import torch

from . import _lib
from ._check import MokArgError, away, fits, on, require, rows_fit, run_on, tensor, workspace
from .dropout import MoKDropout

_TYPES = (torch.bfloat16, torch.float32)


class MoKResidual:
    """Norms before and after a block, fused with its gate, scale, dropout and
    the addition to the stream, for up to ``rows`` rows of ``hidden``:

        z  = y / sqrt(mean y^2 + eps) * w_out            (y itself without w_out)
        x' = x + scale * gate * dropout(z)
        n  = x' / sqrt(mean x'^2 + eps) * w_next

    The stream (x, x') is bf16 or f32, the branch (y, n, the weights and the
    gate) bf16, or f32 with an f32 stream.  ``gate`` is [hidden], or [G, hidden]
    with G dividing the rows, each serving as many consecutive ones.  Matrices
    may have their rows apart.  Calls on one object must not overlap (the
    backward passes share its workspace)."""

    def __init__(self, hidden, rows, eps=1e-6, device="cuda"):
        self.hidden, self.rows, self.eps = hidden, rows, float(eps)
        require(0.0 < self.eps < math.inf, f"eps: {eps}, wanted a positive number")
        self.device = on(device)
        self.ws = workspace(lambda: _lib.mok_residual_workspace_size(rows, hidden), self.device, "unsupported sizes")

    def _matrix(self, t, name, T, types):
        if not (getattr(t, "dtype", None) in types and rows_fit(t, (T, self.hidden), t.dtype, self.device)):
            tensor(t, name, (T, self.hidden), types, self.device, rows_apart=True)

    def _begin(self, x, w_out, gate, w_next, scale, dropout, call, branch):
        """(T, branch type, mok_residual) of a call whose stream is like ``x``."""
        # (what is wrong is put into words only where something is)
        d = self.device
        if not (isinstance(x, torch.Tensor) and x.dim() == 2 and x.shape[0] <= self.rows):
            raise MokArgError(f"a matrix of at most {self.rows} rows of {self.hidden} is wanted")
        T, S = x.shape[0], x.dtype
        self._matrix(x, "x", T, _TYPES)
        B = branch
        if not (B is torch.bfloat16 or S is B is torch.float32):
            raise MokArgError(f"a branch of {B} beside a stream of {S}: wanted bf16, or both f32")
        for w, name in ((w_out, "w_out"), (w_next, "w_next")):
            if w is not None and not fits(w, (self.hidden,), B, d):
                tensor(w, name, (self.hidden,), (B,), d)
        G = 0
        if gate is not None:
            require(isinstance(gate, torch.Tensor) and gate.dim() in (1, 2), "gate: one or two dimensions are wanted")
            G = 1 if gate.dim() == 1 else gate.shape[0]
            if not (1 <= G <= max(T, 1) and T % G == 0):
                raise MokArgError(f"gate: {G} rows for {T} rows")
            shape = (self.hidden,) if gate.dim() == 1 else (G, self.hidden)
            if not fits(gate, shape, B, d):
                tensor(gate, "gate", shape, (B,), d)
        scale = float(scale)
        if not math.isfinite(scale):
            raise MokArgError(f"scale: {scale}, wanted a finite number")
        drop = None
        if dropout is not None:
            if not (isinstance(dropout, MoKDropout) and dropout.device == d):
                raise MokArgError(f"dropout: a MoKDropout on {d} is wanted")
            drop = dropout.drop(call)
        return T, _lib.mok_residual(T, self.hidden, _lib.dtype_of(x), _lib._DTYPES[B], self.eps, scale, w_out, gate, G,
                                    w_next, drop)

    def _out(self, out, name, T, dtype):
        if out is None:
            return torch.empty((T, self.hidden), dtype=dtype, device=self.device)
        self._matrix(out, name, T, (dtype,))
        return out

    def norm(self, x, w_next, out=None, stream=None):
        """n of x alone, of the weight's type: the norm before the first block."""
        if away(self.device, stream):
            return run_on(self, stream, self.norm, x, w_next, out)
        require(getattr(w_next, "dtype", None) in _TYPES, "w_next: a bf16 or f32 tensor is wanted")
        T, r = self._begin(x, None, None, w_next, 1.0, None, 0, w_next.dtype)
        out = self._out(out, "out", T, w_next.dtype)
        _lib.mok_residual_forward(r, x, None, None, out, stream)
        return out

    def norm_backward(self, dn, x, w_next, dx_new=None, out=None, stream=None):
        """(dx, dw_next) of ``norm``, dw_next f32; ``dx_new``, the gradient that
        reaches x beside the norm, is added to dx."""
        if away(self.device, stream):
            return run_on(self, stream, self.norm_backward, dn, x, w_next, dx_new, out)
        require(getattr(w_next, "dtype", None) in _TYPES, "w_next: a bf16 or f32 tensor is wanted")
        T, r = self._begin(x, None, None, w_next, 1.0, None, 0, w_next.dtype)
        self._matrix(dn, "dn", T, (w_next.dtype,))
        if dx_new is not None:
            self._matrix(dx_new, "dx_new", T, (x.dtype,))
        dx = self._out(out, "out", T, x.dtype)
        dw = torch.empty(self.hidden, dtype=torch.float32, device=self.device)
        _lib.mok_residual_backward(r, x, None, dx_new, dn, dx, None, None, None, dw, self.ws, stream)
        return dx, dw

    def forward(self, x, y, w_out=None, gate=None, w_next=None, scale=1.0, dropout=None, call=0, out=None,
                out_next=None, stream=None):
        """(x', n), n None without w_next.  ``out`` may be x, ``out_next`` y.
        ``dropout`` is a MoKDropout; ``call`` numbers its call."""
        if away(self.device, stream):
            return run_on(self, stream, self.forward, x, y, w_out, gate, w_next, scale, dropout, call, out, out_next)
        require(getattr(y, "dtype", None) in _TYPES, "y: a bf16 or f32 tensor is wanted")
        T, r = self._begin(x, w_out, gate, w_next, scale, dropout, call, y.dtype)
        self._matrix(y, "y", T, (y.dtype,))
        out = self._out(out, "out", T, x.dtype)
        if w_next is None:
            require(out_next is None, "out_next: there is no n without w_next")
            n = None
        else:
            n = self._out(out_next, "out_next", T, y.dtype)
        _lib.mok_residual_forward(r, x, y, out, n, stream)
        return out, n

    def backward(self, dx_new, dn, x_new, y, w_out=None, gate=None, w_next=None, scale=1.0, dropout=None, call=0,
                 dx=None, dy=None, stream=None):
        """Gradients of the forward with the same arguments: a dict of dx, dy,
        dw_out and dw_next (f32 [hidden]) and dgate (like gate), None where there is
        nothing to have one.  ``dx_new`` and ``dn`` are the gradients of x' and n
        (None: zero), ``x_new`` is x'.  The dx given to write to may be dx_new,
        dy may be dn or y."""
        if away(self.device, stream):
            return run_on(self, stream, self.backward, dx_new, dn, x_new, y, w_out, gate, w_next, scale, dropout, call,
                          dx, dy)
        require(getattr(y, "dtype", None) in _TYPES, "y: a bf16 or f32 tensor is wanted")
        T, r = self._begin(x_new, w_out, gate, w_next, scale, dropout, call, y.dtype)
        S, B, d = x_new.dtype, y.dtype, self.device
        self._matrix(y, "y", T, (B,))
        require((dn is None) or (w_next is not None), "dn: there is no n without w_next")
        require(dx_new is not None or dn is not None, "dx_new, dn: one of them is wanted")
        if dx_new is not None:
            self._matrix(dx_new, "dx_new", T, (S,))
        if dn is not None:
            self._matrix(dn, "dn", T, (B,))
        dx, dy = self._out(dx, "dx", T, S), self._out(dy, "dy", T, B)
        f32 = dict(dtype=torch.float32, device=d)
        dw_out = None if w_out is None else torch.empty(self.hidden, **f32)
        dgate = None if gate is None else torch.empty(gate.shape, dtype=B, device=d)
        dw_next = None if w_next is None else \
            torch.empty(self.hidden, **f32) if dn is not None else torch.zeros(self.hidden, **f32)
        _lib.mok_residual_backward(r, x_new, y, dx_new, dn, dx, dy, dw_out, dgate, dw_next if dn is not None else None,
                                   self.ws, stream)
        return dict(dx=dx, dy=dy, dw_out=dw_out, dgate=dgate, dw_next=dw_next)
