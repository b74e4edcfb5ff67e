"""Waits of the few-token layer that run out: the call ends, says so, and a
zeroed workspace serves the next one.  The workspace is prepared on the host:
with the launch-wide abort word set (what a call that timed out leaves
behind) every wait that is not satisfied at once gives up; with counts of
arrivals that no tile can have, joined tiles are never finished, and the waits
for them run out after their limit."""

import pytest
import torch

from _helpers import assert_bf16_close, assert_mxfp8_close, np64, require_gpu

pytestmark = pytest.mark.gpu

ABORT = 3       # header word
HEADER = 256    # bytes; the counts of arrivals follow

# one token (weights of a few units), odd numbers of blocks, many rows on few experts, more phases than one
SHAPES = [(1, 256, 128, 8, 2), (6, 7168, 256, 12, 3), (33, 384, 640, 64, 8), (128, 2048, 768, 16, 8)]


def setup(shape, prec):
    from mixture_experts_layer_side_gb300.decode import MoKDecoder
    from mixture_experts_layer_side_gb300.inputs import Shape, make_inputs
    from mixture_experts_layer_side_gb300.layer import quantize_weights
    inp = {k: v.cuda() for k, v in make_inputs(Shape(*shape), "uniform", seed=9).items()}
    W = [inp[n] for n in ("W1", "W3", "W2")]
    keep = quantize_weights(*W) if prec == "mxfp8" else None
    dec = MoKDecoder(Shape(*shape), precision=prec)
    Wr = torch.randn((shape[1], shape[3]), device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    return inp, W if keep is None else keep["fwd"], keep, dec, Wr


def run(dec, inp, W, Wr, router):
    if router:
        return dec.layer(inp["x"], Wr, *W)
    return (dec.forward(inp["x"], inp["idx"], inp["s"], *W),)


def timed_out(dec):
    from mixture_experts_layer_side_gb300 import _lib
    status = _lib.mok_check(dec.ws)
    dec.ws.zero_()
    return status == 6  # MOK_ERR_TIMEOUT


@pytest.mark.parametrize("router", [False, True])
@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
@pytest.mark.parametrize("shape", SHAPES)
def test_few_unwinds_after_an_abort(shape, prec, router):
    require_gpu()
    inp, W, _keep, dec, Wr = setup(shape, prec)
    first = run(dec, inp, W, Wr, router)
    dec.check()
    for _ in range(20):
        dec.ws.view(torch.int32)[ABORT] = 1
        run(dec, inp, W, Wr, router)
        assert timed_out(dec)
        again = run(dec, inp, W, Wr, router)
        dec.check()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
@pytest.mark.parametrize("shape", SHAPES[1:])
def test_few_waits_run_out(shape, prec):
    require_gpu()
    inp, W, _keep, dec, Wr = setup(shape, prec)
    first = run(dec, inp, W, Wr, False)
    dec.check()
    _, _, I, E, k = shape
    tiles = min(E + 128 * k // 16, 128 * k) * (I // 128)  # of the most units that a call can have
    dec.ws.view(torch.int32)[HEADER // 4:HEADER // 4 + tiles] = 1 << 20
    run(dec, inp, W, Wr, False)
    # (a call after it, without a look at the first's status, says the same)
    run(dec, inp, W, Wr, False)
    assert timed_out(dec)
    again = run(dec, inp, W, Wr, False)
    dec.check()
    assert torch.equal(first[0], again[0])
    ref = np64(first[0])
    (assert_bf16_close if prec == "bf16" else assert_mxfp8_close)(np64(again[0]), ref, "after a timeout")
