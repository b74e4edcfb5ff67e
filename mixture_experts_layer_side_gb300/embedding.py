"""Token embedding and its gradient (mok_embed_*; no compute here)."""

from __future__ import annotations

import torch

from . import _lib
from ._check import on, require, tensor

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
        self.pad_id = _lib.MOK_EMBED_NO_PAD if pad_id is None else int(pad_id)
        self.device = on(device)
        n = _lib.mok_embed_workspace_size(vocab, hidden, tokens)
        if n == 0:
            raise _lib.MokError(2, "unsupported sizes")
        self.ws = torch.zeros(n, dtype=torch.uint8, device=self.device)

    def _ids(self, ids):
        require(isinstance(ids, torch.Tensor) and ids.numel() <= self.tokens, f"ids: at most {self.tokens} are wanted")
        tensor(ids, "ids", ids.shape, (torch.int32,), self.device)

    def forward(self, table, ids, scale=1.0, out=None, stream=None):
        """[*ids.shape, hidden] of the table's type."""
        self._ids(ids)
        tensor(table, "table", (self.vocab, self.hidden), _TYPES, self.device)
        shape = (*ids.shape, self.hidden)
        if out is None:
            out = torch.empty(shape, dtype=table.dtype, device=self.device)
        tensor(out, "out", shape, (table.dtype,), self.device)
        _lib.mok_embed_forward(table, ids, self.pad_id, float(scale), out, self.ws, stream)
        return out

    def backward(self, dx, ids, scale=1.0, out=None, accumulate=False, stream=None):
        """The table's gradient [vocab, hidden] in ``out`` (bf16 or f32; f32 by
        default): written whole, or with ``accumulate`` added to the rows that
        ``ids`` names."""
        self._ids(ids)
        tensor(dx, "dx", (*ids.shape, self.hidden), _TYPES, self.device)
        require(out is not None or not accumulate, "out: wanted to accumulate into")
        if out is None:
            out = torch.empty((self.vocab, self.hidden), dtype=torch.float32, device=self.device)
        tensor(out, "out", (self.vocab, self.hidden), _TYPES, self.device)
        _lib.mok_embed_backward(dx, ids, self.pad_id, float(scale), out, accumulate, self.ws, stream)
        return out

    def check(self, stream=None):
        """Synchronise and raise if the device recorded an error."""
        st = _lib.mok_check(self.ws, stream)
        if st != 0:
            raise _lib.MokError(st, "embedding: device status")
