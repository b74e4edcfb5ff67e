"""The feed-forward block on a workspace that a timeout left behind: with the
launch-wide abort word set by the host, a wait gives up where it is not
satisfied within a few tenths of a millisecond.  Every call ends and says so,
and a zeroed workspace serves the next one with the same bits."""

import pytest
import torch

import test_ffn_gpu as cases
from _helpers import require_gpu

pytestmark = pytest.mark.gpu

ABORT = 3  # header word
TIMEOUT = 6  # MOK_ERR_TIMEOUT
BF16 = torch.bfloat16


def step(ffn, s):
    w = s["W1"], s["W3"], s["W2"]
    out = ffn.forward(s["x"], *w)
    return [out, *ffn.backward(s["x"], *w, s["dout"]).values(), ffn.infer(s["x"], *w)]


# K cut over 2, 4 and 8 pairs, fewer steps than stages and several times as many, whole tiles with and without a last wave
@pytest.mark.parametrize("T,H,I", [(1, 256, 128), (7, 2048, 768), (100, 2048, 768), (300, 4096, 2048), (1000, 1144, 680),
                                   (3000, 1024, 1024)])
def test_unwinds_after_an_abort(T, H, I):
    require_gpu()
    from mixture_experts_layer_side_gb300 import _lib
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    s = cases.make(T, H, I)
    ffn = MoKFeedForward(H, I, T)
    first = step(ffn, s)
    ffn.check()
    for _ in range(5):
        ffn.ws.view(torch.int32)[ABORT] = 1
        step(ffn, s)
        assert _lib.mok_check(ffn.ws) == TIMEOUT
        ffn.ws.zero_()
        assert all(torch.equal(a, b) for a, b in zip(step(ffn, s), first))
        ffn.check()


def test_check_makes_the_workspace_ready():
    require_gpu()
    from mixture_experts_layer_side_gb300 import _lib
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    s = cases.make(70, 520, 264)
    ffn = MoKFeedForward(520, 264, 70)
    first = step(ffn, s)
    ffn.ws.view(torch.int32)[ABORT] = 1
    step(ffn, s)
    with pytest.raises(_lib.MokError) as err:
        ffn.check()
    assert err.value.status == TIMEOUT and not ffn.ws[:256].any()
    assert all(torch.equal(a, b) for a, b in zip(step(ffn, s), first))
    ffn.check()


def long_tensors(T, H, I):
    g = torch.Generator(device="cuda").manual_seed(1)
    return [0.05 * torch.randn(s, generator=g, device="cuda", dtype=BF16) for s in ((T, H), (H, I), (H, I), (I, H))]


def test_long_sums_give_up():
    """Tiles whose sums take longer than an aborted wait's patience: epilogues give up first, and with three tiles a pair
    the matrix instructions' warp and the copies' after them."""
    require_gpu()
    from mixture_experts_layer_side_gb300 import _lib
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    T, H, I = 60000, 131072, 8
    x, *w = long_tensors(T, H, I)
    ffn = MoKFeedForward(H, I, T, training=False)
    first, out = ffn.infer(x, *w), torch.empty_like(x)
    for _ in range(3):
        ffn.ws.view(torch.int32)[ABORT] = 1
        ffn.infer(x, *w, out=out)
        assert _lib.mok_check(ffn.ws) == TIMEOUT
        ffn.ws.zero_()
        assert torch.equal(ffn.infer(x, *w, out=out), first)
        ffn.check()


def test_long_sums_of_parts_give_up():
    """The same where pairs share a tile: the wait for all of a part's sums gives up while they run."""
    require_gpu()
    from mixture_experts_layer_side_gb300 import _lib
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    T, H, I = 7680, 8, 131072
    x, *w = long_tensors(T, H, I)
    ffn = MoKFeedForward(H, I, T)

    def both():
        out = ffn.forward(x, *w)
        return [out, *ffn.backward(x, *w, x).values()]

    first = both()
    ffn.check()
    for _ in range(3):
        ffn.ws.view(torch.int32)[ABORT] = 1
        both()
        assert _lib.mok_check(ffn.ws) == TIMEOUT
        ffn.ws[:256].zero_()
        assert all(torch.equal(a, b) for a, b in zip(both(), first))
        ffn.check()
