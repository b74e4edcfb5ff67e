"""Workspace recovery, argument checks and devices of the few-token layer, the
distillation loss and the embedding that need no GPU."""

import ctypes
import os

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_side_gb300 import build
    if not os.path.exists(build.LIB_PATH):
        build.build()
    from mixture_experts_layer_side_gb300 import _lib
    return _lib


OK, INVALID, UNSUPPORTED, TIMEOUT = 0, 1, 2, 6
A = ctypes.c_void_p(256)      # a 16-byte aligned fake pointer
BIG = 1 << 40


def small_decoder(precision="bf16"):
    from mixture_experts_layer_side_gb300.decode import MoKDecoder
    from mixture_experts_layer_side_gb300.inputs import Shape
    return MoKDecoder(Shape(4, 256, 128, 4, 2), precision=precision, device="cpu")


@pytest.mark.parametrize("status,zeroed", [(TIMEOUT, True), (5, False)])
def test_decoder_is_ready_again_after_a_timeout(lib, monkeypatch, status, zeroed):
    dec = small_decoder()
    dec.ws.fill_(7)
    monkeypatch.setattr(lib, "mok_check", lambda ws, stream=None: status)
    with pytest.raises(lib.MokError) as err:
        dec.check()
    assert err.value.status == status
    assert bool((dec.ws == 0).all()) == zeroed
