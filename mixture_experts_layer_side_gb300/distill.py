"""Distillation loss from a teacher's top logits (mok_distill_*; no compute here)."""

from __future__ import annotations

import torch

from . import _lib
from ._check import away, fits, on, require, rows_fit, run_on, tensor, workspace

_TYPES = (torch.bfloat16, torch.float32)


class DistillLoss:
    """KL(p || softmax(z / temperature)) per row, p the softmax of the
    teacher's listed logits / temperature over the list, for up to ``rows``
    rows of ``vocab`` student logits (bf16 or f32, rows any distance apart)
    and lists of up to ``top`` (id, value) pairs; an id of -1 leaves its entry
    out.  Rows are weighted by ``dloss`` in the gradient.  Errors found on the
    device (an id outside the vocabulary) are raised by ``check``."""

    def __init__(self, rows, vocab, top, device="cuda"):
        self.rows, self.vocab, self.top = rows, vocab, top
        self.device = on(device)
        self.ws = workspace(lambda: _lib.mok_distill_workspace_size(rows, vocab, top), self.device, "unsupported sizes")

    def _begin(self, z, ids, vals, temperature):
        d = self.device
        if not (type(z) is type(ids) is torch.Tensor and z.dim() == ids.dim() == 2):
            require(isinstance(z, torch.Tensor) and z.dim() == 2, "z: a matrix is wanted")
            require(isinstance(ids, torch.Tensor) and ids.dim() == 2, "ids: a matrix is wanted")
        T, K = z.shape[0], ids.shape[1]
        if T > self.rows:
            require(False, f"z: at most {self.rows} rows are wanted")
        if not 1 <= K <= self.top:
            require(False, f"ids: lists of 1 to {self.top} entries are wanted")
        if not (rows_fit(z, (T, self.vocab), z.dtype, d) and z.dtype in _TYPES and fits(ids, (T, K), torch.int32, d) and
                fits(vals, (T, K), torch.float32, d)):
            tensor(z, "z", (T, self.vocab), _TYPES, d, rows_apart=True)
            tensor(ids, "ids", (T, K), (torch.int32,), d)
            tensor(vals, "vals", (T, K), (torch.float32,), d)
        tau = float(temperature)
        if not 0.0 < tau < float("inf"):
            require(False, f"temperature: {tau}, wanted a positive number")
        return T, tau

    def _row_values(self, T, name, t):
        if not fits(t, (T,), torch.float32, self.device):
            tensor(t, name, (T,), (torch.float32,), self.device)

    def _gradient(self, z, out):
        if out is None:
            return torch.empty(z.shape, dtype=z.dtype, device=z.device)
        if not rows_fit(out, z.shape, z.dtype, self.device):
            tensor(out, "out", z.shape, (z.dtype,), self.device, rows_apart=True)
        return out

    def forward(self, z, ids, vals, temperature=1.0, stream=None):
        """(loss, lse), f32 [T] each."""
        if away(self.device, stream):
            return run_on(self, stream, self.forward, z, ids, vals, temperature)
        T, tau = self._begin(z, ids, vals, temperature)
        loss = torch.empty(T, dtype=torch.float32, device=self.device)
        lse = torch.empty(T, dtype=torch.float32, device=self.device)
        _lib.mok_distill_forward(z, ids, vals, tau, loss, lse, self.ws, stream)
        return loss, lse

    def backward(self, z, ids, vals, lse, dloss, temperature=1.0, out=None, stream=None):
        """dz of z's type, from the forward's ``lse``; ``out`` may be z itself,
        but not overlap it in part."""
        if away(self.device, stream):
            return run_on(self, stream, self.backward, z, ids, vals, lse, dloss, temperature, out)
        T, tau = self._begin(z, ids, vals, temperature)
        self._row_values(T, "lse", lse)
        self._row_values(T, "dloss", dloss)
        dz = self._gradient(z, out)
        _lib.mok_distill_backward(z, ids, vals, tau, lse, dloss, dz, self.ws, stream)
        return dz

    def forward_backward(self, z, ids, vals, dloss, temperature=1.0, out=None, stream=None):
        """(loss, dz) in one call; ``out`` as in ``backward``."""
        if away(self.device, stream):
            return run_on(self, stream, self.forward_backward, z, ids, vals, dloss, temperature, out)
        T, tau = self._begin(z, ids, vals, temperature)
        self._row_values(T, "dloss", dloss)
        dz = self._gradient(z, out)
        loss = torch.empty(T, dtype=torch.float32, device=self.device)
        _lib.mok_distill_step(z, ids, vals, tau, dloss, loss, None, dz, self.ws, stream)
        return loss, dz

    def check(self, stream=None):
        """Synchronise and raise if the device recorded an error."""
        if away(self.device, stream):
            return run_on(self, stream, self.check)
        st = _lib.mok_check(self.ws, stream)
        if st != 0:
            raise _lib.MokError(st, "distillation: device status")
