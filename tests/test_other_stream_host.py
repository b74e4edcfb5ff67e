"""Calls on another stream than the current one, on stand-ins for streams (no
GPU needed): what is handed back is told of the caller's stream where it is a
tensor, and a dict of the caller's own may hold anything beside them."""

import contextlib
from types import SimpleNamespace

import pytest
import torch

from mixture_experts_layer_side_gb300 import _check


class Tensor(torch.Tensor):
    def record_stream(self, stream):
        self.told = stream


@pytest.mark.parametrize("kind", ["dict", "tuple", "one", "none"])
def test_results_are_told_of_the_callers_stream(monkeypatch, kind):
    device = torch.device("cuda", 0)
    mine, other = SimpleNamespace(device=device, name="mine"), SimpleNamespace(device=device, name="other")
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: mine)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: other)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    a, b = (torch.zeros(2).as_subclass(Tensor) for _ in range(2))
    result = {"dict": {"dX": a, "dW1": b, "step": 7, "note": "kept", "none": None}, "tuple": (a, None, b), "one": a,
              "none": None}[kind]
    got = _check.run_on(SimpleNamespace(device=device, ws=None), 5, lambda: result)
    assert got is result
    for t in {"dict": (a, b), "tuple": (a, b), "one": (a,), "none": ()}[kind]:
        assert t.told is mine
