"""The dense gated feed-forward block and its gradients (mok_ffn_*; no compute here)."""

from __future__ import annotations

import torch

from . import _lib
from ._check import away, fits, on, require, run_on, tensor, workspace

BF16 = torch.bfloat16


class MoKFeedForward:
    """out = (silu(x W1) * (x W3)) W2 in bf16, for up to ``tokens`` rows a call:
    a shared expert beside the routed ones, or a block without routing.  W1 and
    W3 are [hidden, inner], W2 [inner, hidden]; hidden and inner are multiples
    of 8.

    Owns the workspace and, with ``training``, the context that ``forward`` keeps for
    ``backward`` (of the same x and weights, before the next forward).
    ``infer`` keeps nothing, and streams the weights through every SM for up to
    four tokens.  Calls on one object must not overlap.
    After a timeout the results of all calls since the last ``check`` are void;
    ``check`` raises it and makes the workspace ready again."""

    def __init__(self, hidden, inner, tokens, training=True, device="cuda"):
        self.hidden, self.inner, self.tokens, self.training = hidden, inner, tokens, bool(training)
        self.device = on(device)
        self.ws = workspace(lambda: _lib.mok_ffn_workspace_size(tokens, hidden, inner, self.training), self.device,
                            "unsupported sizes")
        self.ctx = torch.empty(_lib.mok_ffn_ctx_size(tokens, inner), dtype=torch.uint8, device=self.device) \
            if training else None
        self._kept = None  # rows of the last forward
        self._w13, self._w2 = (hidden, inner), (inner, hidden)

    def _begin(self, x, W1, W3, W2):
        d = self.device
        if not (type(x) is torch.Tensor and x.dim() == 2 and x.shape[0] <= self.tokens):
            require(isinstance(x, torch.Tensor) and x.dim() == 2 and x.shape[0] <= self.tokens,
                    f"x: at most {self.tokens} rows of {self.hidden} are wanted")
        rows = (x.shape[0], self.hidden)
        if not (fits(x, rows, BF16, d) and fits(W1, self._w13, BF16, d) and fits(W3, self._w13, BF16, d) and
                fits(W2, self._w2, BF16, d)):
            for name, t, shape in (("x", x, rows), ("W1", W1, self._w13), ("W3", W3, self._w13), ("W2", W2, self._w2)):
                tensor(t, name, shape, (BF16,), d)
        return rows

    def _out(self, out, rows):
        if out is None:
            return torch.empty(rows, dtype=BF16, device=self.device)
        if not fits(out, rows, BF16, self.device):
            tensor(out, "out", rows, (BF16,), self.device)
        return out

    def infer(self, x, W1, W3, W2, out=None, stream=None):
        """out [T, hidden], nothing kept."""
        if away(self.device, stream):
            return run_on(self, stream, self.infer, x, W1, W3, W2, out)
        out = self._out(out, self._begin(x, W1, W3, W2))
        _lib.mok_ffn_infer(self.ws, x, W1, W3, W2, out, stream)
        return out

    def forward(self, x, W1, W3, W2, out=None, stream=None):
        """out [T, hidden]; keeps what ``backward`` reads."""
        if away(self.device, stream):
            return run_on(self, stream, self.forward, x, W1, W3, W2, out)
        require(self.training, "forward: made without training (infer keeps nothing)")
        rows = self._begin(x, W1, W3, W2)
        out = self._out(out, rows)
        _lib.mok_ffn_forward(self.ws, x, W1, W3, W2, out, self.ctx, stream)
        self._kept = rows[0]
        return out

    def alloc_grads(self, T):
        d = dict(dtype=BF16, device=self.device)
        return dict(dX=torch.empty((T, self.hidden), **d), dW1=torch.empty(self._w13, **d),
                    dW3=torch.empty(self._w13, **d), dW2=torch.empty(self._w2, **d))

    def backward(self, x, W1, W3, W2, dout, grads=None, stream=None):
        """dict of dX, dW1, dW3 and dW2, bf16 (``grads``: tensors to write them to)."""
        if away(self.device, stream):
            return run_on(self, stream, self.backward, x, W1, W3, W2, dout, grads)
        rows = self._begin(x, W1, W3, W2)
        require(self._kept == rows[0], f"x: {rows[0]} rows, the last forward had {self._kept}")
        if not fits(dout, rows, BF16, self.device):
            tensor(dout, "dout", rows, (BF16,), self.device)
        if grads is None:
            grads = self.alloc_grads(rows[0])
        else:
            require(isinstance(grads, dict) and {"dX", "dW1", "dW3", "dW2"} <= set(grads),
                    "grads: a dict of dX, dW1, dW3 and dW2 is wanted")
            for name, shape in (("dX", rows), ("dW1", self._w13), ("dW3", self._w13), ("dW2", self._w2)):
                if not fits(grads[name], shape, BF16, self.device):
                    tensor(grads[name], name, shape, (BF16,), self.device)
        _lib.mok_ffn_backward(self.ws, self.ctx, x, W1, W3, W2, dout, grads["dX"], grads["dW1"], grads["dW3"],
                              grads["dW2"], stream)
        return grads

    def check(self, stream=None):
        """Synchronise and raise if the device recorded an error."""
        if away(self.device, stream):
            return run_on(self, stream, self.check)
        st = _lib.mok_check(self.ws, stream)
        if st == _lib.MOK_ERR_TIMEOUT:
            # a call that gave up leaves the abort word behind
            self.ws.zero_()
            if self.device.type == "cuda":
                torch.cuda.current_stream(self.device).synchronize()
        if st != 0:
            raise _lib.MokError(st, "feed-forward block: device status")
