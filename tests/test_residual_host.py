"""Refusals of the residual join and dropout: the C ABI's host checks (fake
pointers, nothing is enqueued) and the wrappers' checks.  No GPU needed."""

import ctypes
import os

import pytest
import torch

OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_side_gb300 import build
    if not os.path.exists(build.LIB_PATH):
        build.build()
    from mixture_experts_layer_side_gb300 import _lib
    return _lib


def at(n):
    """A fake pointer: matrices a MiB apart."""
    return ctypes.c_void_p(n << 20) if n else None


def test_dropout_host_checks(lib):
    def call(rows=4, cols=64, type=0, x=at(1), ldx=64, p=0.5, call_dev=0, out=at(2), ldo=64, drop=True):
        d = lib.MokDrop(p, 1, 2, call_dev)
        return lib.LIB.mok_dropout(rows, cols, type, x, ldx, d if drop else None, out, ldo, None)

    for bad in (dict(rows=-1), dict(cols=-1), dict(type=2), dict(x=None), dict(out=None), dict(ldx=63), dict(ldo=63),
                dict(p=-0.1), dict(p=1.1), dict(p=float("nan")), dict(call_dev=260), dict(drop=False),
                dict(x=ctypes.c_void_p((1 << 20) + 1)), dict(type=1, x=ctypes.c_void_p((1 << 20) + 2)),
                # rows that meet: shifted, other strides, the end of one in the start of the other
                dict(out=ctypes.c_void_p((1 << 20) + 2)), dict(out=at(1), ldo=65),
                dict(out=ctypes.c_void_p((1 << 20) + 2 * (3 * 64 + 63)))):
        assert call(**bad) == INVALID, bad
    assert call(rows=1 << 31, cols=1 << 31) == UNSUPPORTED
    assert call(rows=0, x=None, out=None) == OK and call(cols=0, x=None, out=None) == OK
    # (a mistake in p is one with no elements too)
    assert call(rows=0, p=2.0) == INVALID


def test_residual_host_checks(lib):
    assert lib.mok_residual_workspace_size(8, 256) > 0
    for bad in ((-1, 64), (8, 0), (8, lib.MOK_RESIDUAL_MAX_HIDDEN + 1), ((1 << 30) + 1, 64)):
        assert lib.mok_residual_workspace_size(*bad) == 0
    need = [lib.mok_residual_workspace_size(t, 1024) for t in range(0, 5000, 7)]
    assert need == sorted(need)

    def spec(T=8, H=64, S=0, B=0, eps=1e-6, scale=1.0, w_out=at(20), gate=at(21), G=1, w_next=at(22), p=0.0):
        val = [v.value if v is not None else None for v in (w_out, gate, w_next)]
        return lib.MokResidual(T, H, S, B, G, eps, scale, *val, lib.MokDrop(p, 0, 0, None))

    def forward(x=at(1), ldx=64, y=at(2), ldy=64, xo=at(3), ldxo=64, n=at(4), ldn=64, r=None, **kw):
        r = spec(**kw) if r is None else r
        return lib.LIB.mok_residual_forward(r, x, ldx, y, ldy, xo, ldxo, n, ldn, None)

    def backward(x=at(1), ldx=64, y=at(2), ldy=64, dxo=at(3), lddxo=64, dn=at(4), lddn=64, dx=at(5), lddx=64, dy=at(6),
                 lddy=64, dw_out=at(7), dgate=at(8), dw_next=at(9), ws=at(30), n=BIG, **kw):
        return lib.LIB.mok_residual_backward(spec(**kw), x, ldx, y, ldy, dxo, lddxo, dn, lddn, dx, lddx, dy, lddy, dw_out,
                                             dgate, dw_next, ws, n, None)

    odd = ctypes.c_void_p((40 << 20) + 1)
    both = (dict(T=-1), dict(H=0), dict(S=2), dict(B=7), dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")),
            dict(scale=float("inf")), dict(G=0), dict(G=3), dict(G=-1), dict(gate=None, G=1), dict(w_out=odd),
            dict(gate=odd), dict(w_next=odd), dict(p=1.5))
    for bad in both:
        assert forward(**bad) == backward(**bad) == INVALID, bad
    assert forward(S=0, B=1) == backward(S=0, B=1) == UNSUPPORTED
    assert forward(H=lib.MOK_RESIDUAL_MAX_HIDDEN + 1) == UNSUPPORTED
    for bad in (dict(x=None), dict(xo=None), dict(n=None), dict(w_next=None), dict(ldx=63), dict(ldy=1), dict(ldxo=0),
                dict(ldn=63), dict(x=odd), dict(xo=odd), dict(n=odd), dict(y=None), dict(y=None, xo=None),
                dict(xo=at(2)), dict(n=at(3)), dict(n=at(1)), dict(xo=ctypes.c_void_p((1 << 20) + 2)),
                dict(xo=at(1), ldxo=72), dict(n=ctypes.c_void_p((2 << 20) + 64))):
        assert forward(**bad) == INVALID, bad
    assert forward(T=0, x=None, y=None, xo=None, n=None) == OK
    for bad in (dict(x=None), dict(y=None), dict(dn=None), dict(dw_next=None), dict(dw_out=None), dict(dgate=None),
                dict(dx=None, dy=None), dict(dxo=None, dn=None, dw_next=None), dict(ws=None), dict(ws=odd),
                dict(lddx=63), dict(lddn=10), dict(dx=odd), dict(dgate=odd), dict(dw_out=ctypes.c_void_p((7 << 20) + 2)),
                dict(w_next=None), dict(w_out=None), dict(gate=None, G=0), dict(dy=None), dict(dx=at(4)), dict(dx=at(1)),
                dict(dy=at(3)), dict(dy=at(5)), dict(dx=at(2)), dict(dy=at(1)), dict(dx=ctypes.c_void_p((3 << 20) + 2))):
        assert backward(**bad) == INVALID, bad
    assert backward(n=100) == SMALL


def refused(lib, fn, *a, **kw):
    with pytest.raises(ValueError) as err:
        fn(*a, **kw)
    assert isinstance(err.value, lib.MokError) and err.value.status == INVALID


def test_wrappers_refuse(lib):
    from mixture_experts_layer_side_gb300.dropout import MoKDropout
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    bf16, f32 = torch.bfloat16, torch.float32
    for p in (-0.1, 1.5, float("nan"), "0.5"):
        refused(lib, MoKDropout, p, device="cpu")
    for seed in (-1, 2**64, 0.5):
        refused(lib, MoKDropout, 0.5, seed=seed, device="cpu")
    drop = MoKDropout(0.5, device="cpu")
    x = torch.zeros((8, 64), dtype=bf16)
    for bad in (x.half(), [1.0], x.t(), x.view(2, 4, 64)[:, :, :32]):
        refused(lib, drop.forward, bad)
    for call in (-1, 2**63, 0.5, torch.zeros(2, dtype=torch.int64), torch.zeros(1, dtype=torch.int32)):
        refused(lib, drop.forward, x, call=call)
    for out in (x.float(), x[:4], x.t()):
        refused(lib, drop.forward, x, out=out)
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        refused(lib, MoKResidual, 64, 8, eps=eps, device="cpu")
    with pytest.raises(lib.MokError):
        MoKResidual(lib.MOK_RESIDUAL_MAX_HIDDEN + 1, 8, device="cpu")
    res = MoKResidual(64, 8, device="cpu")
    w, y = torch.ones(64, dtype=bf16), x.clone()
    good = dict(w_out=w, gate=w, w_next=w)
    for bad in (dict(w_out=w.float()), dict(w_next=w[:32]), dict(gate=w.float()), dict(gate=torch.ones((3, 64), dtype=bf16)),
                dict(gate=torch.ones((16, 64), dtype=bf16)), dict(gate=torch.ones((0, 64), dtype=bf16)), dict(gate=0.5),
                dict(scale=float("nan")), dict(dropout=0.5), dict(dropout=drop, call=-1),
                dict(gate=torch.ones((64, 2), dtype=bf16).t())):
        refused(lib, res.forward, x, y, **dict(good, **bad))
        refused(lib, res.backward, x, x, x, y, **dict(good, **bad))
    for a, b in ((x, y.float()), (x.half(), y), (x, y.half()), (x, y[:4]), (x, y.t()), (x, None), (x[0], y[0]),
                 (torch.zeros((9, 64), dtype=bf16),) * 2, (x.float(), y.float())):
        refused(lib, res.forward, a, b, **good)
    refused(lib, res.forward, x, y, w_out=w, out_next=y)
    refused(lib, res.forward, x, y, out=x.float(), **good)
    refused(lib, res.backward, None, None, x, y, **good)
    refused(lib, res.backward, x, x, x, y, w_out=w)
    refused(lib, res.backward, x.float(), x, x, y, **good)
    refused(lib, res.backward, x, x.float(), x, y, **good)
    refused(lib, res.backward, x, x, x, y, **good, dx=x.float())
    refused(lib, res.norm, x, None)
    refused(lib, res.norm, x, w.float())
    refused(lib, res.norm_backward, x[:3], x, w)
