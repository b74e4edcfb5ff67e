"""Refusals of the dense feed-forward block: the C ABI's host checks (fake
pointers, nothing is enqueued) and the wrapper's checks.  No GPU needed."""

import ctypes
import os

import pytest
import torch

OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_side_gb300 import build
    if not os.path.exists(build.LIB_PATH):
        build.build()
    from mixture_experts_layer_side_gb300 import _lib
    return _lib


def at(n):
    """A fake pointer: tensors 64 MiB apart."""
    return ctypes.c_void_p(n << 26)


ODD = ctypes.c_void_p((90 << 26) + 8)


def test_ffn_host_checks(lib):
    L = lib.LIB
    size = lib.mok_ffn_workspace_size
    assert size(8, 256, 128, True) > size(8, 256, 128, False) > 0 and size(0, 256, 128, True) > 0
    assert size(300, 8, 8, True) > 0 and lib.mok_ffn_ctx_size(300, 8) >= 3 * 300 * 8 * 2
    for bad in ((-1, 256, 128), (8, 0, 128), (8, 256, 0), (8, 260, 128), (8, 256, 124), (8, lib.MOK_FFN_MAX_SIZE + 8, 128),
                (8, 256, lib.MOK_FFN_MAX_SIZE + 8), ((1 << 22) + 1, 8, 8)):
        assert size(*bad, True) == size(*bad, False) == 0, bad
    assert lib.mok_ffn_ctx_size(-1, 8) == lib.mok_ffn_ctx_size(8, 12) == 0
    # a workspace for more tokens serves fewer
    for H, I in ((256, 128), (1144, 680), (7168, 2048)):
        for training in (False, True):
            need = [size(t, H, I, training) for t in range(0, 400)]
            assert need == sorted(need)

    def infer(T=8, H=256, I=128, ws=at(1), n=BIG, x=at(2), W1=at(3), W3=at(4), W2=at(5), out=at(6)):
        return L.mok_ffn_infer(T, H, I, ws, n, x, W1, W3, W2, out, None)

    def forward(T=8, H=256, I=128, ws=at(1), n=BIG, x=at(2), W1=at(3), W3=at(4), W2=at(5), out=at(6), ctx=at(7)):
        return L.mok_ffn_forward(T, H, I, ws, n, x, W1, W3, W2, out, ctx, None)

    def backward(T=8, H=256, I=128, ws=at(1), n=BIG, ctx=at(7), x=at(2), W1=at(3), W3=at(4), W2=at(5), dout=at(8),
                 dX=at(9), dW1=at(10), dW3=at(11), dW2=at(12)):
        return L.mok_ffn_backward(T, H, I, ws, n, ctx, x, W1, W3, W2, dout, dX, dW1, dW3, dW2, None)

    for name in ("ws", "x", "W1", "W3", "W2"):
        for bad in (None, ODD):
            assert infer(**{name: bad}) == forward(**{name: bad}) == backward(**{name: bad}) == INVALID, name
    for name in ("out", "ctx"):
        for bad in (None, ODD):
            assert forward(**{name: bad}) == INVALID
    assert infer(out=None) == infer(out=ODD) == INVALID
    for name in ("ctx", "dout", "dX", "dW1", "dW3", "dW2"):
        for bad in (None, ODD):
            assert backward(**{name: bad}) == INVALID, name
    for bad in (dict(T=-1), dict(H=0), dict(I=-8)):
        assert infer(**bad) == forward(**bad) == backward(**bad) == INVALID
    for bad in (dict(H=252), dict(I=100), dict(T=(1 << 22) + 1)):
        assert infer(**bad) == forward(**bad) == backward(**bad) == UNSUPPORTED
    assert infer(n=1000) == forward(n=1000) == backward(n=1000) == SMALL
    # an output over an input, another output, the context or the workspace
    last = ctypes.c_void_p((2 << 26) + 8 * 256 * 2 - 16)
    for bad in (at(2), at(3), at(5), last, at(1)):
        assert infer(out=bad) == forward(out=bad) == INVALID
    assert forward(ctx=at(6)) == forward(ctx=at(1)) == forward(ctx=at(4)) == INVALID
    for bad in (dict(dX=at(8)), dict(dX=at(2)), dict(dW1=at(11)), dict(dW2=at(5)), dict(dW3=at(7)), dict(dX=at(1))):
        assert backward(**bad) == INVALID, bad
    assert infer(T=0, x=None, out=None) == forward(T=0, x=None, out=None, ctx=None) == OK
    assert backward(T=0, dW1=None) == backward(T=0, dW2=at(10)) == INVALID


def refused(lib, fn, *a, **kw):
    with pytest.raises(ValueError) as err:
        fn(*a, **kw)
    assert isinstance(err.value, lib.MokError) and err.value.status == INVALID


def test_wrapper_refuses(lib):
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    for bad in ((100, 64, 8), (64, 100, 8), (64, 64, -1), (0, 64, 8), (64, 64, (1 << 22) + 1)):
        with pytest.raises(lib.MokError):
            MoKFeedForward(*bad, device="cpu")
    bf16 = torch.bfloat16
    ffn = MoKFeedForward(64, 32, 8, device="cpu")
    x, W1, W3, W2 = (torch.zeros(s, dtype=bf16) for s in ((4, 64), (64, 32), (64, 32), (32, 64)))
    good = [x, W1, W3, W2]
    for i, bad in [(0, x.float()), (0, torch.zeros((9, 64), dtype=bf16)), (0, x[:, :32]), (0, x[0]), (0, [1.0]), (0, None),
                   (0, torch.zeros((64, 4), dtype=bf16).t()), (1, W2), (1, W1.float()), (2, W3.unsqueeze(0)), (2, None),
                   (2, W2.t()), (3, W1), (3, W2[:16])]:
        args = good[:i] + [bad] + good[i + 1:]
        refused(lib, ffn.infer, *args)
        refused(lib, ffn.forward, *args)
        refused(lib, ffn.backward, *args, x)
    for out in (x.float(), x[:2], torch.zeros((64, 4), dtype=bf16).t()):
        refused(lib, ffn.infer, *good, out=out)
        refused(lib, ffn.forward, *good, out=out)
    refused(lib, ffn.backward, *good, x)  # no forward before it
    ffn._kept = 4
    refused(lib, ffn.backward, *good, x[:2])
    refused(lib, ffn.backward, *good, x.float())
    refused(lib, ffn.backward, x[:2].clone(), W1, W3, W2, x[:2].clone())
    grads = ffn.alloc_grads(4)
    for bad in (dict(dX=x.float()), dict(dW1=W2), dict(dW3=W3.float()), dict(dW2=None)):
        refused(lib, ffn.backward, *good, x, grads=dict(grads, **bad))
    refused(lib, ffn.backward, *good, x, grads={"dX": x})
    refused(lib, MoKFeedForward(64, 32, 8, training=False, device="cpu").forward, *good)
