"""Token embedding and its gradient (mok_embed_*; no compute here)."""

from __future__ import annotations

import torch

from . import _lib
from ._check import away, fits, on, require, run_on, tensor, workspace

_TYPES = (torch.bfloat16, torch.float32)


class MoKEmbedding:
    """scale * table[ids] and its gradient, for a [vocab, hidden] table (bf16
    or f32) and up to ``tokens`` int32 ids a call (of any shape).  Tokens with
    ``pad_id`` take no part in the gradient.  The gradient is summed in f32 in
    ascending token order (bitwise reproducible).  Calls on one object must
    not overlap (they share the workspace).  Errors found on the device (an id
    outside the table) are raised by ``check``."""

    def __init__(self, vocab, hidden, tokens, pad_id=None, device="cuda"):
        self.vocab, self.hidden, self.tokens = vocab, hidden, tokens
        self._table = (vocab, hidden)
        self.pad_id = _lib.MOK_EMBED_NO_PAD if pad_id is None else int(pad_id)
        # (a wider number would name another id in the call; the lowest says that there is none)
        require(pad_id is None or -2**31 < self.pad_id < 2**31, f"pad_id: {pad_id}, wanted an int32 above the lowest")
        self.device = on(device)
        self.ws = workspace(lambda: _lib.mok_embed_workspace_size(vocab, hidden, tokens), self.device,
                            "unsupported sizes")

    def _ids(self, ids):
        if not (type(ids) is torch.Tensor and ids.numel() <= self.tokens and
                fits(ids, ids.shape, torch.int32, self.device)):
            require(isinstance(ids, torch.Tensor) and ids.numel() <= self.tokens,
                    f"ids: at most {self.tokens} are wanted")
            tensor(ids, "ids", ids.shape, (torch.int32,), self.device)
        return (*ids.shape, self.hidden)

    def forward(self, table, ids, scale=1.0, out=None, stream=None):
        """[*ids.shape, hidden] of the table's type."""
        if away(self.device, stream):
            return run_on(self, stream, self.forward, table, ids, scale, out)
        d = self.device
        shape = self._ids(ids)
        if not (getattr(table, "dtype", None) in _TYPES and fits(table, self._table, table.dtype, d)):
            tensor(table, "table", self._table, _TYPES, d)
        if out is None:
            out = torch.empty(shape, dtype=table.dtype, device=d)
        elif not fits(out, shape, table.dtype, d):
            tensor(out, "out", shape, (table.dtype,), d)
        _lib.mok_embed_forward(table, ids, self.pad_id, float(scale), out, self.ws, stream)
        return out

    def backward(self, dx, ids, scale=1.0, out=None, accumulate=False, stream=None):
        """The table's gradient [vocab, hidden] in ``out`` (bf16 or f32; f32 by
        default): written whole, or with ``accumulate`` added to the rows that
        ``ids`` names."""
        if away(self.device, stream):
            return run_on(self, stream, self.backward, dx, ids, scale, out, accumulate)
        d = self.device
        shape = self._ids(ids)
        if not (getattr(dx, "dtype", None) in _TYPES and fits(dx, shape, dx.dtype, d)):
            tensor(dx, "dx", shape, _TYPES, d)
        if out is None:
            require(not accumulate, "out: wanted to accumulate into")
            out = torch.empty(self._table, dtype=torch.float32, device=d)
        elif not (getattr(out, "dtype", None) in _TYPES and fits(out, self._table, out.dtype, d)):
            tensor(out, "out", self._table, _TYPES, d)
        _lib.mok_embed_backward(dx, ids, self.pad_id, float(scale), out, accumulate, self.ws, stream)
        return out

    def check(self, stream=None):
        """Synchronise and raise if the device recorded an error."""
        if away(self.device, stream):
            return run_on(self, stream, self.check)
        st = _lib.mok_check(self.ws, stream)
        if st != 0:
            raise _lib.MokError(st, "embedding: device status")
