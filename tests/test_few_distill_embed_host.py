"""Refusals of the few-token layer, the distillation loss and the embedding:
the C ABI's host checks (fake pointers, nothing is enqueued) and the Python
wrappers' checks of their tensors.  No GPU needed."""

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


OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 3
A = ctypes.c_void_p(256)      # a 16-byte aligned fake pointer
ODD = ctypes.c_void_p(257)
BIG = 1 << 40


def test_few_host_checks(lib):
    L, shape = lib.LIB, lib.shape_of
    good = shape(8, 256, 128, 8, 2)
    assert lib.mok_few_workspace_size(good) > 0
    assert lib.mok_few_workspace_size(good, lib.MOK_MXFP8) > 0
    assert lib.mok_few_workspace_size(shape(128, 256, 128, 8, 2)) > 0
    for bad in (shape(129, 256, 128, 8, 2), shape(0, 256, 128, 8, 2), shape(8, 200, 128, 8, 2),
                shape(8, 256, 100, 8, 2), shape(8, 256, 128, 1025, 2), shape(8, 256, 128, 8, 33), shape(8, 32896, 128, 8, 2),
                shape(8, 256, 32896, 8, 2)):
        assert lib.mok_few_workspace_size(bad) == 0
    assert L.mok_few_workspace_size(ctypes.byref(good), 7) == 0
    # a workspace for more tokens serves fewer
    for prec in (lib.MOK_BF16, lib.MOK_MXFP8):
        for sizes in ((128, 128, 1024, 1), (256, 128, 8, 2), (7168, 2048, 256, 8)):
            need = [lib.mok_few_workspace_size(shape(t, *sizes), prec) for t in range(1, 129)]
            assert need == sorted(need) and need[0] > 0
    assert L.mok_few_workspace_size(None, 0) == 0

    def forward(s=good, prec=0, ws=A, n=BIG, idx=A, x=A, sc=A, W1=A, W3=A, W2=A, out=A):
        return L.mok_few_forward(ctypes.byref(s), prec, ws, n, idx, x, sc, W1, W3, W2, out, None)

    def layer(s=good, prec=0, ws=A, n=BIG, x=A, Wr=A, W1=A, W3=A, W2=A, idx=A, sc=A, out=A):
        return L.mok_few_layer(ctypes.byref(s), prec, ws, n, x, Wr, None, W1, W3, W2, idx, sc, out, None)

    for name in ("ws", "idx", "x", "sc", "W1", "W3", "W2", "out"):
        assert forward(**{name: None}) == INVALID, name
        assert layer(**{name: None}) == INVALID, name
    assert layer(Wr=None) == INVALID
    for name in ("ws", "x", "W1", "W3", "W2", "out"):
        assert forward(**{name: ODD}) == INVALID, name
    assert forward(n=256) == SMALL
    assert forward(prec=5) == INVALID
    assert forward(s=shape(129, 256, 128, 8, 2)) == UNSUPPORTED
    assert layer(s=shape(8, 256, 128, 4, 5)) == INVALID  # more choices than experts
    null = lib.MokMx()
    px = ctypes.cast(ctypes.pointer(null), ctypes.c_void_p)
    assert forward(prec=1, W1=px, W3=px, W2=px) == INVALID
    odd = lib.MokMx(256, 257)
    po = ctypes.cast(ctypes.pointer(odd), ctypes.c_void_p)
    assert forward(prec=1, W1=po, W3=po, W2=po) == INVALID


def test_distill_host_checks(lib):
    L = lib.LIB
    assert lib.mok_distill_workspace_size(4, 100, 8) > 0
    for bad in ((-1, 100, 8), (4, 0, 8), (4, 100, 0), (4, 100, lib.MOK_DISTILL_MAX_TOP + 1)):
        assert lib.mok_distill_workspace_size(*bad) == 0

    def step(T=4, V=100, K=8, type=0, z=A, ldz=100, ids=A, vals=A, tau=1.0, dloss=A, loss=A, lse=A, dz=A, lddz=100,
             ws=A, n=BIG):
        return L.mok_distill_step(T, V, K, type, z, ldz, ids, vals, tau, dloss, loss, lse, dz, lddz, ws, n, None)

    def forward(z=A, loss=A, lse=A, ldz=100):
        return L.mok_distill_forward(4, 100, 8, 0, z, ldz, A, A, 1.0, loss, lse, A, BIG, None)

    def backward(lse=A, dloss=A, dz=A, lddz=100):
        return L.mok_distill_backward(4, 100, 8, 0, A, 100, A, A, 1.0, lse, dloss, dz, lddz, A, BIG, None)

    for name in ("z", "ids", "vals", "dloss", "loss", "dz", "ws"):
        assert step(**{name: None}) == INVALID, name
    for bad in (dict(T=-1), dict(V=0), dict(K=0), dict(type=2), dict(ldz=99), dict(lddz=99), dict(tau=0.0),
                dict(tau=-1.0), dict(tau=float("nan")), dict(tau=float("inf")), dict(tau=1e-45), dict(z=ODD),
                dict(dz=ODD), dict(type=1, z=ctypes.c_void_p(258))):
        assert step(**bad) == INVALID, bad
    assert step(K=lib.MOK_DISTILL_MAX_TOP + 1) == UNSUPPORTED
    assert step(n=8) == SMALL
    assert step(T=0, z=None, dz=None) == OK
    assert forward(loss=None) == forward(lse=None) == forward(z=None) == forward(ldz=50) == INVALID
    assert backward(lse=None) == backward(dloss=None) == backward(dz=None) == backward(lddz=1) == INVALID


def test_embed_host_checks(lib):
    L = lib.LIB
    assert lib.mok_embed_workspace_size(100, 64, 10) > 0
    assert lib.mok_embed_workspace_size(100, 64, 0) > 0
    for bad in ((0, 64, 10), (100, 0, 10), (100, 64, -1), ((1 << 30) + 1, 64, 10)):
        assert lib.mok_embed_workspace_size(*bad) == 0

    def forward(V=100, H=64, N=10, type=0, table=A, ids=A, out=A, ws=A, n=BIG):
        return L.mok_embed_forward(V, H, N, type, table, ids, -1, 1.0, out, ws, n, None)

    def backward(V=100, H=64, N=10, dt=0, dx=A, ids=A, gt=1, dtable=A, acc=0, ws=A, n=BIG):
        return L.mok_embed_backward(V, H, N, dt, dx, ids, -1, 1.0, gt, dtable, acc, ws, n, None)

    for name in ("table", "ids", "out", "ws"):
        assert forward(**{name: None}) == INVALID, name
    for name in ("dx", "ids", "dtable", "ws"):
        assert backward(**{name: None}) == INVALID, name
    for bad in (dict(V=0), dict(H=0), dict(N=-1), dict(ws=ODD)):
        assert forward(**bad) == backward(**bad) == INVALID, bad
    assert forward(type=3) == forward(table=ODD) == forward(out=ODD) == INVALID
    assert backward(dt=2) == backward(gt=9) == backward(acc=2) == backward(dx=ODD) == INVALID
    assert backward(gt=1, dtable=ctypes.c_void_p(258)) == INVALID
    assert forward(n=64) == backward(n=64) == SMALL
    assert forward(N=0, table=None, out=None, ids=None) == OK


def refused(lib, call, *a, **kw):
    with pytest.raises(ValueError) as err:
        call(*a, **kw)
    assert isinstance(err.value, lib.MokError) and err.value.status == INVALID


def test_decoder_refuses_tensors(lib):
    from mixture_experts_layer_side_gb300.decode import MoKDecoder
    from mixture_experts_layer_side_gb300.inputs import Shape, make_inputs
    with pytest.raises(lib.MokError):
        MoKDecoder(Shape(129, 256, 128, 4, 2), device="cpu")
    i = make_inputs(Shape(4, 256, 128, 4, 2))
    dec = MoKDecoder(Shape(4, 256, 128, 4, 2), device="cpu")
    good = [i[n] for n in ("x", "idx", "s", "W1", "W3", "W2")]
    for at, bad in [(0, i["x"].float()), (0, torch.cat([i["x"], i["x"]])), (0, i["x"][:, :128]),
                    (0, i["x"].t().contiguous().t()), (0, [1.0]), (1, i["idx"].long()), (1, i["idx"][:3]),
                    (2, i["s"].half()), (2, i["s"].t().contiguous().t()), (3, i["W1"].float()),
                    (3, i["W1"].transpose(1, 2)), (4, i["W3"][:3]), (5, i["W2"].transpose(1, 2).contiguous())]:
        a = list(good)
        a[at] = bad
        refused(lib, dec.forward, *a)
    refused(lib, dec.forward, *good, out=torch.empty(4, 256))
    Wr = torch.zeros((256, 4), dtype=torch.bfloat16)
    refused(lib, dec.layer, i["x"], Wr.float(), *good[3:])
    refused(lib, dec.layer, i["x"], Wr.t().contiguous().t(), *good[3:])
    refused(lib, dec.layer, i["x"], Wr, *good[3:], bias=torch.zeros(5))
    mx = MoKDecoder(Shape(4, 256, 128, 4, 2), precision="mxfp8", device="cpu")
    refused(lib, mx.forward, *good)


def test_distill_refuses_tensors(lib):
    from mixture_experts_layer_side_gb300.distill import DistillLoss
    with pytest.raises(lib.MokError):
        DistillLoss(4, 10, 513, device="cpu")
    d = DistillLoss(4, 10, 3, device="cpu")
    z, ids, vals, w = torch.zeros(4, 10), torch.zeros((4, 3), dtype=torch.int32), torch.zeros(4, 3), torch.zeros(4)
    for a in [(z.double(), ids, vals, w), (z.half(), ids, vals, w), (torch.zeros(5, 10), ids, vals, w),
              (torch.zeros(4, 11), ids, vals, w), (torch.zeros(10, 4).t(), ids, vals, w), (z[0], ids, vals, w),
              (z, ids.long(), vals, w), (z, ids[:3], vals, w), (z, torch.zeros((4, 4), dtype=torch.int32), vals, w),
              (z, ids[:, :0], vals[:, :0], w), (z, ids, vals.bfloat16(), w), (z, ids, vals[:, :2], w),
              (z, ids, vals, w.double()), (z, ids, vals, w[:2]), (z, ids, vals, torch.zeros(4, 1))]:
        refused(lib, d.forward_backward, *a)
    refused(lib, d.forward_backward, z, ids, vals, w, out=z.bfloat16())
    refused(lib, d.forward_backward, z, ids, vals, w, out=torch.zeros(10, 4).t())
    for tau in (0.0, -1.0, float("nan"), float("inf")):
        refused(lib, d.forward, z, ids, vals, temperature=tau)


def test_embedding_refuses_tensors(lib):
    from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
    with pytest.raises(lib.MokError):
        MoKEmbedding(0, 8, 4, device="cpu")
    e = MoKEmbedding(10, 8, 4, device="cpu")
    t, ids = torch.zeros(10, 8), torch.zeros(4, dtype=torch.int32)
    for a in [(t.double(), ids), (t[:9], ids), (torch.zeros(8, 10).t(), ids), (t, ids.long()),
              (t, torch.zeros(5, dtype=torch.int32)), (t, torch.zeros(8, dtype=torch.int32)[::2])]:
        refused(lib, e.forward, *a)
    refused(lib, e.forward, t, ids, out=torch.zeros(4, 8).bfloat16())
    dx = torch.zeros(4, 8)
    refused(lib, e.backward, dx[:3], ids)
    refused(lib, e.backward, dx.half(), ids)
    refused(lib, e.backward, dx, ids, out=torch.zeros(9, 8))
    refused(lib, e.backward, dx, ids, out=torch.zeros(10, 8, dtype=torch.float64))
    refused(lib, e.backward, dx, ids, accumulate=True)
