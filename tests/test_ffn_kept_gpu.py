"""Gradients of the dense feed-forward block with h and u kept in f32 from the
forward pass: bounds with no rounding of theirs, and values far out, where silu
has run out on either side.

What the arithmetic adds to the roundings of a, dh, du and the results: the
sums of h, u and da (K 2^-23 of their terms' magnitudes), and that of the
sigmoid s = 1 / (1 + e), e = exp(-h), with e off by (2 + |h|) 2^-23 of itself
(its argument's rounding and its own) and s by s (1 - s) of that.  In silu, h s,
that is |h| s (1 - s) (2 + |h|) 2^-23 < 0.9 2^-23 (most near |h| = 2), in its
derivative s (1 + h (1 - s)) it is s (1 - s) (1 + |h|) (2 + |h|) 2^-23 < 1.4
2^-23 (most near 1.6), and some 4 roundings of 2^-24 of terms of at most 1.3: below 2^-21 of
the factor beside them, of which 2^-20 are allowed."""

import pytest
import torch

import test_ffn_gpu as cases
from _helpers import require_gpu

pytestmark = pytest.mark.gpu

HALF, F32 = cases.HALF, cases.F32
OWN = 2.0 ** -20
# roundings on the way to each result: dh and du (dX), one of them, and the result's own
ROUNDINGS = dict(dX=3, dW1=2, dW3=2)


def reference(s):
    """Gradients of x, W1 and W3 and element bounds, in 64 bits."""
    x, W1, W3, W2, do = (s[k].double() for k in ("x", "W1", "W3", "W2", "dout"))
    T, H, I = x.shape[0], x.shape[1], W2.shape[0]
    h, u = x @ W1, x @ W3
    eh, eu = H * F32 * (x.abs() @ W1.abs()), H * F32 * (x.abs() @ W3.abs())
    sg = torch.sigmoid(h)
    sl, dsl = h * sg, sg * (1 + h * (1 - sg))
    da = do @ W2.t()
    eda = H * F32 * (do.abs() @ W2.abs().t())
    ada = da.abs() + eda
    dh, du = da * u * dsl, da * sl
    # |silu'| <= 1.1, |silu''| <= 0.5
    edh = eda * u.abs() * 1.1 + ada * (eu * 1.1 + (u.abs() + eu) * (0.5 * eh + OWN)) + (HALF + OWN) * dh.abs()
    edu = eda * sl.abs() + ada * (1.1 * eh + OWN) + (HALF + OWN) * du.abs()
    r = dict(dX=dh @ W1.t() + du @ W3.t(), dW1=x.t() @ dh, dW3=x.t() @ du)
    xa = x.abs().t()
    e = dict(dX=edh @ W1.abs().t() + edu @ W3.abs().t() +
             2 * I * F32 * (dh.abs() @ W1.abs().t() + du.abs() @ W3.abs().t()),
             dW1=xa @ edh + T * F32 * (xa @ dh.abs()), dW3=xa @ edu + T * F32 * (xa @ du.abs()))
    return r, e


def compare(got, r, e, name, whole):
    err = (got.double() - r[name]).abs()
    # (a rounding in bf16 of a value that is itself off)
    bound = HALF * r[name].abs() + 1.02 * e[name] + 1e-30
    assert bool((err <= bound).all()), (name, float((err / bound).max()))
    if whole:
        fro = float(err.norm() / r[name].norm())
        assert fro <= 1.8e-3 * ROUNDINGS[name] ** 0.5, (name, fro)


@pytest.mark.parametrize("T,H,I", [(256, 256, 256), (1000, 1144, 680), (513, 2048, 768), (2100, 520, 1032), (129, 128, 128),
                                   (64, 4096, 2056)])
@pytest.mark.parametrize("far", [1, 60])
def test_gradients_without_a_rounding_of_what_is_kept(T, H, I, far):
    require_gpu()
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    s = cases.make(T, H, I, seed=30)
    s["x"] *= far
    w = s["W1"], s["W3"], s["W2"]
    ffn = MoKFeedForward(H, I, T)
    ffn.forward(s["x"], *w)
    got = ffn.backward(s["x"], *w, s["dout"])
    ffn.check()
    r, e = reference(s)
    for name in r:
        compare(got[name], r, e, name, far == 1)
