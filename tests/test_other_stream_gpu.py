"""A caller's own dict of gradients with more in it than the four, on another
stream."""

import pytest
import torch

import test_ffn_gpu as cases
from _helpers import require_gpu

pytestmark = pytest.mark.gpu


def test_gradients_into_a_dict_of_the_callers():
    require_gpu()
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    T, H, I = 40, 256, 128
    s = cases.make(T, H, I)
    w = s["W1"], s["W3"], s["W2"]
    ffn = MoKFeedForward(H, I, T)
    ffn.forward(s["x"], *w)
    want = ffn.backward(s["x"], *w, s["dout"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    grads = dict(ffn.alloc_grads(T), step=7, note="kept")
    torch.cuda.synchronize()
    assert ffn.backward(s["x"], *w, s["dout"], grads=grads, stream=side) is grads
    side.synchronize()
    assert all(torch.equal(grads[k], want[k]) for k in want) and grads["step"] == 7
    ffn.check()
