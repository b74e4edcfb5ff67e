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


def test_decoder_refuses_mxfp8_descriptors_of_other_tensors(lib, monkeypatch):
    """Codes and scales of another shape, orientation or type, which would be read out of range or as other
    values.  (The call itself is taken away: what passes the checks is not enqueued.)"""
    called = []
    monkeypatch.setattr(lib, "mok_few_forward", lambda *a: called.append(a))
    monkeypatch.setattr(lib, "mok_few_layer", lambda *a: called.append(a))
    T, H, I, E, k = 4, 256, 128, 4, 2
    dec = small_decoder("mxfp8")

    def mx(*shape, scales=None, dtype=torch.uint8):
        scales = scales or (shape[0], shape[1] // 32, shape[2])
        return lib.mx(torch.zeros(shape, dtype=dtype), torch.zeros(scales, dtype=torch.uint8))

    x, idx, s = torch.zeros((T, H)).bfloat16(), torch.zeros((T, k), dtype=torch.int32), torch.zeros((T, k))
    Wr = torch.zeros((H, E)).bfloat16()
    w13, w2 = mx(E, H, I), mx(E, I, H)
    raw = lib.MokMx(256, 256)
    flat = lib.mx(torch.zeros(E * H * I, dtype=torch.uint8), torch.zeros((E * H // 32, I), dtype=torch.uint8))
    for W in ((w13, w13, w2), (mx(E, H, I, dtype=torch.float8_e4m3fn), w13, w2), (raw, raw, raw), (flat, w13, w2)):
        called.clear()
        dec.forward(x, idx, s, *W)
        dec.layer(x, Wr, *W)
        assert len(called) == 2
    called.clear()
    for W in ((w2, w13, w2), (w13, w2, w2), (w13, w13, w13), (mx(E - 1, H, I), w13, w2), (w13, mx(E, H, I // 2), w2),
              (w13, w13, mx(E, I, H, scales=(E, I, H // 32))), (mx(E, H, I, scales=(E, H // 32 - 1, I)), w13, w2),
              (mx(E, H, I, dtype=torch.int16), w13, w2), (lib.mx(torch.zeros(9, dtype=torch.uint8), w13.tensors[1]), w13, w2),
              (lib.mx(w13.tensors[0][..., ::2], w13.tensors[1]), w13, w2), (torch.zeros((E, H, I)).bfloat16(), w13, w2)):
        for call in (lambda: dec.forward(x, idx, s, *W), lambda: dec.layer(x, Wr, *W)):
            with pytest.raises(ValueError):
                call()
    assert not called


def distill_calls(lib):
    """The step and the backward on 4 rows of 100 bf16 logits at `z`, rows `ldz` apart, in a workspace that is too
    small for them, so that what passes the other checks is still not enqueued."""
    L = lib.LIB

    def step(z, ldz, dz, lddz, T=4, V=100):
        return L.mok_distill_step(T, V, 8, 0, z, ldz, A, A, 1.0, A, A, A, dz, lddz, A, 8, None)

    def backward(z, ldz, dz, lddz, T=4, V=100):
        return L.mok_distill_backward(T, V, 8, 0, z, ldz, A, A, 1.0, A, A, dz, lddz, A, 8, None)

    return step, backward


def test_distill_refuses_a_gradient_that_overlaps_the_logits_in_part(lib):
    SMALL = 3
    Z = 1 << 20
    for call in distill_calls(lib):
        # in place, apart, and rows that lie between one another
        assert call(Z, 100, Z, 100) == SMALL
        assert call(Z, 100, Z, 200, T=1) == SMALL
        assert call(Z, 100, Z + 800, 100) == call(Z + 800, 100, Z, 100) == SMALL
        assert call(Z, 200, Z + 200, 200) == call(Z + 200, 200, Z, 200) == SMALL
        assert call(Z, 300, Z + 200, 300) == call(Z, 300, Z + 400, 300) == SMALL
        assert call(Z, 300, Z + 200 - 1200, 300) == SMALL
        # (z in columns 0-99 of rows of 400, the gradient's at 100 and 300 of each)
        assert call(Z, 400, Z + 200, 200) == SMALL
        # a row over itself with another stride, shifted, or over another row
        assert call(Z, 100, Z, 200) == call(Z, 200, Z, 100) == INVALID
        assert call(Z, 100, Z + 2, 100) == call(Z, 100, Z - 2, 100) == INVALID
        assert call(Z, 100, Z + 200, 100) == call(Z, 100, Z - 200, 100) == INVALID
        assert call(Z, 300, Z + 198, 300) == call(Z, 300, Z + 402, 300) == INVALID
        assert call(Z, 300, Z + 198 - 600, 300) == INVALID
        assert call(Z, 400, Z + 200, 201) == INVALID
        assert call(Z, 100, Z + 2, 300, T=1) == INVALID
    # every pair of small strides and offsets against the bytes themselves
    step, _ = distill_calls(lib)
    for lz in (3, 4, 7):
        for ld in (3, 5, 7):
            rows = [set(range(2 * lz * i, 2 * lz * i + 6)) for i in range(3)]
            for off in range(-60, 60, 2):
                grad = [set(range(off + 2 * ld * i, off + 2 * ld * i + 6)) for i in range(3)]
                meet = any(a & b for a in rows for b in grad) and not (off == 0 and lz == ld)
                assert step(Z, lz, Z + off, ld, T=3, V=3) == (INVALID if meet else SMALL), (lz, ld, off)


def test_distill_refuses_rows_past_32_bit_columns(lib):
    assert lib.mok_distill_workspace_size(1, 1 << 30, 8) > 0
    for V in ((1 << 30) + 1, 2 ** 31 - 9, 2 ** 31 - 1):
        assert lib.mok_distill_workspace_size(1, V, 8) == 0
        for call in distill_calls(lib):
            assert call(1 << 20, V, 1 << 40, V, T=1, V=V) == UNSUPPORTED
        assert lib.LIB.mok_distill_forward(1, V, 8, 0, A, V, A, A, 1.0, A, A, A, BIG, None) == UNSUPPORTED


def test_distill_refuses_a_temperature_whose_factor_is_infinite(lib):
    def forward(tau):
        return lib.LIB.mok_distill_forward(4, 100, 8, 0, A, 100, A, A, tau, A, A, A, 8, None)

    assert forward(4.3e-39) == forward(1e-30) == 3  # (the workspace is too small)
    for tau in (4.2e-39, 3.5e-39, 2.9e-39, 1e-45):
        assert forward(tau) == INVALID


def test_embedding_refuses_a_pad_id_that_is_no_int32(lib):
    from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
    for pad in (None, 0, -1, 9, 10, 2 ** 31 - 1, -2 ** 31 + 1):
        assert MoKEmbedding(10, 8, 4, pad_id=pad, device="cpu").pad_id == (lib.MOK_EMBED_NO_PAD if pad is None else pad)
    for pad in (2 ** 32 + 5, 2 ** 31, -2 ** 31, -2 ** 32 + 3):
        with pytest.raises(ValueError):
            MoKEmbedding(10, 8, 4, pad_id=pad, device="cpu")


def test_calls_are_made_on_the_device_of_their_tensors(lib, monkeypatch):
    """With another device current than the object's: the workspace's size is asked for, and every call made, with
    the object's own.  (Devices of a fake; "meta" tensors, and checks that take them for the device's.)"""
    from mixture_experts_layer_side_gb300 import _check, decode, distill, embedding
    from mixture_experts_layer_side_gb300.inputs import Shape
    now, real_zeros, real_empty = [0], torch.zeros, torch.empty

    class Device:
        def __init__(self, device):
            self.index = torch.device(device).index

        def __enter__(self):
            self.was, now[0] = now[0], self.index

        def __exit__(self, *a):
            now[0] = self.was

    monkeypatch.setattr(_check, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **kw: real_zeros(*a, device="meta", **kw))
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: real_empty(*a, device="meta", **kw))
    for m in (_check, decode, distill, embedding):
        for n in ("fits", "rows_fit"):
            if hasattr(m, n):
                monkeypatch.setattr(m, n, lambda *a: True)
    seen, asked = [], []
    for n in ("mok_few_forward", "mok_few_layer", "mok_distill_forward", "mok_distill_backward", "mok_distill_step",
              "mok_embed_forward", "mok_embed_backward"):
        monkeypatch.setattr(lib, n, lambda *a, n=n: seen.append((n, now[0])))
    monkeypatch.setattr(lib, "mok_check", lambda *a: seen.append(("mok_check", now[0])) or 0)
    for n in ("mok_few_workspace_size", "mok_distill_workspace_size", "mok_embed_workspace_size"):
        monkeypatch.setattr(lib, n, lambda *a: asked.append(now[0]) or 256)
    t = real_empty((4, 2), device="meta")
    dec = decode.MoKDecoder(Shape(4, 256, 128, 4, 2), device="cuda:1")
    loss = distill.DistillLoss(4, 2, 2, device="cuda:1")
    emb = embedding.MoKEmbedding(10, 8, 8, device="cuda:1")
    assert asked == [1, 1, 1] and now == [0]
    dec.forward(t, t, t, t, t, t)
    dec.layer(t, t, t, t, t)
    loss.forward(t, t, t)
    loss.backward(t, t, t, t, t)
    loss.forward_backward(t, t, t, t)
    emb.forward(t, t)
    emb.backward(t, t)
    for part in (dec, loss, emb):
        part.check()
    assert len(seen) == 10 and all(dev == 1 for _, dev in seen) and now == [0], seen
