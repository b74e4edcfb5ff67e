"""The dense gated feed-forward block against its formulas in 64 bits.

Each element's error is held to a bound that follows from the arithmetic: bf16
rounds by at most half a step (2^-8 of the value), 32-bit sums of K terms lose
at most K 2^-23 of the terms' magnitudes.  The whole's relative error is held
to what independent roundings of 1.8e-3 (the root mean square of a bf16
rounding over normal values is 1.7e-3) add up to."""

import numpy as np
import pytest
import torch

from _helpers import require_gpu

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
HALF = torch.finfo(BF16).eps / 2
F32 = 2.0 ** -23


def make(T, H, I, seed=0, std=0.05):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0):
        return (std * torch.randn(shape, generator=g, device="cuda")).to(BF16)

    return dict(x=randn(T, H), W1=randn(H, I, std=std), W3=randn(H, I, std=std), W2=randn(I, H, std=std),
                dout=randn(T, H))


def reference(s):
    """Values and element bounds, in 64 bits."""
    x, W1, W3, W2, do = (s[k].double() for k in ("x", "W1", "W3", "W2", "dout"))
    T, H, I = x.shape[0], x.shape[1], W2.shape[0]
    h, u = x @ W1, x @ W3
    eh, eu = H * F32 * (x.abs() @ W1.abs()), H * F32 * (x.abs() @ W3.abs())
    sg = torch.sigmoid(h)
    sl, dsl = h * sg, sg * (1 + h * (1 - sg))
    a = sl * u
    # |silu'| <= 1.1, |silu''| <= 0.5; a's own arithmetic is some 2^-20 of it
    ea = 1.1 * eh * (u.abs() + eu) + sl.abs() * eu + (HALF + 2.0 ** -20) * a.abs()
    r, e = {}, {}
    r["out"] = a @ W2
    e["out"] = ea @ W2.abs() + I * F32 * (a.abs() @ W2.abs())
    da = do @ W2.t()
    eda = H * F32 * (do.abs() @ W2.abs().t())
    rh, ru = HALF * h.abs() + eh, HALF * u.abs() + eu  # h and u as they are kept
    dh, du = da * u * dsl, da * sl
    edh = eda * u.abs() * 1.1 + (da.abs() + eda) * (ru * 1.1 + (u.abs() + ru) * 0.5 * rh) + (HALF + 2.0 ** -20) * dh.abs()
    edu = eda * sl.abs() + (da.abs() + eda) * 1.1 * rh + (HALF + 2.0 ** -20) * du.abs()
    r["dX"] = dh @ W1.t() + du @ W3.t()
    e["dX"] = edh @ W1.abs().t() + edu @ W3.abs().t() + 2 * I * F32 * (dh.abs() @ W1.abs().t() + du.abs() @ W3.abs().t())
    xa = x.abs().t()
    r["dW1"], e["dW1"] = x.t() @ dh, xa @ edh + T * F32 * (xa @ dh.abs())
    r["dW3"], e["dW3"] = x.t() @ du, xa @ edu + T * F32 * (xa @ du.abs())
    r["dW2"], e["dW2"] = a.t() @ do, ea.t() @ do.abs() + T * F32 * (a.abs().t() @ do.abs())
    return r, e


# roundings on the way to each result: a and its own; h, u, dh or du (two of them in dX) and its own
ROUNDINGS = dict(out=2, dX=5, dW1=4, dW3=3, dW2=2)


def compare(got, r, e, name):
    assert got.dtype == BF16 and got.shape == r[name].shape
    err = (got.double() - r[name]).abs()
    bound = HALF * r[name].abs() + 1.02 * e[name] + 1e-30
    assert bool((err <= bound).all()), (name, float((err / bound).max()))
    if r[name].numel() >= 4096:
        fro = float(err.norm() / r[name].norm())
        assert fro <= 1.8e-3 * ROUNDINGS[name] ** 0.5, (name, fro)


SIZES = [(1, 8, 8), (3, 64, 72), (129, 128, 128), (255, 264, 136), (256, 256, 256), (1000, 1144, 680), (513, 2048, 768),
         (2100, 520, 1032), (64, 4096, 2056), (1537, 776, 8)]


@pytest.mark.parametrize("T,H,I", SIZES)
def test_step_against_formulas(T, H, I):
    require_gpu()
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    s = make(T, H, I)
    w = s["W1"], s["W3"], s["W2"]
    ffn = MoKFeedForward(H, I, T + 5)
    r, e = reference(s)
    nan = {k: torch.full_like(v, float("nan"), dtype=BF16) for k, v in r.items()}
    out = ffn.forward(s["x"], *w, out=nan["out"])
    got = ffn.backward(s["x"], *w, s["dout"], grads={k: nan[k] for k in ("dX", "dW1", "dW3", "dW2")})
    ffn.check()
    for name, t in dict(got, out=out).items():
        compare(t, r, e, name)
    again = ffn.forward(s["x"], *w)
    grads = ffn.backward(s["x"], *w, s["dout"])
    assert torch.equal(again, out) and all(torch.equal(grads[k], got[k]) for k in got)
    ffn.check()


@pytest.mark.parametrize("T,H,I", [(1, 256, 128), (5, 128, 128), (33, 2048, 768), (128, 768, 384), (129, 256, 128),
                                   (1, 7168, 2048), (16, 1144, 680), (100, 2048, 768), (300, 8, 16)])
def test_infer_against_formulas(T, H, I):
    require_gpu()
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    s = make(T, H, I, seed=1)
    ffn = MoKFeedForward(H, I, max(T, 200), training=False)
    r, e = reference(s)
    out = ffn.infer(s["x"], s["W1"], s["W3"], s["W2"], out=torch.full_like(s["x"], float("nan")))
    ffn.check()
    compare(out, r, e, "out")
    for _ in range(3):
        assert torch.equal(ffn.infer(s["x"], s["W1"], s["W3"], s["W2"]), out)


def test_calls_of_every_size_share_a_workspace():
    """Few tokens and many in turn, training and inference, on one object."""
    require_gpu()
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    H, I, most = 512, 256, 700
    s = make(most, H, I, seed=2)
    ffn = MoKFeedForward(H, I, most)
    w = s["W1"], s["W3"], s["W2"]
    r, e = reference(s)
    for T in (700, 1, 128, 129, 64, 700, 17, 300):
        x = s["x"][:T].contiguous()
        for out in (ffn.infer(x, *w), ffn.forward(x, *w)):
            compare(out, {"out": r["out"][:T]}, {"out": e["out"][:T]}, "out")
        part = {k: v[:T].contiguous() if k in ("x", "dout") else v for k, v in s.items()}
        rr, ee = reference(part)
        got = ffn.backward(x, *w, part["dout"])
        for k in got:
            compare(got[k], rr, ee, k)
    ffn.check()


def test_no_rows():
    require_gpu()
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    s = make(0, 128, 128)
    ffn = MoKFeedForward(128, 128, 16)
    w = s["W1"], s["W3"], s["W2"]
    assert ffn.infer(s["x"], *w).shape == ffn.forward(s["x"], *w).shape == (0, 128)
    grads = dict(dX=s["x"].clone(), **{k: torch.full_like(s[k[1:]], float("nan")) for k in ("dW1", "dW3", "dW2")})
    got = ffn.backward(s["x"], *w, s["dout"], grads=grads)
    assert not any(got[k].any() for k in ("dW1", "dW3", "dW2"))
    ffn.check()


def test_large_values_stay_in_range():
    """silu of large negative and positive h: no NaN from exp or from 0 times infinity."""
    require_gpu()
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    T, H, I = 260, 136, 264
    s = make(T, H, I, seed=3)
    s["x"] *= 60
    ffn = MoKFeedForward(H, I, T)
    w = s["W1"], s["W3"], s["W2"]
    r, e = reference(s)
    out = ffn.forward(s["x"], *w)
    got = ffn.backward(s["x"], *w, s["dout"])
    for name, t in dict(got, out=out).items():
        assert torch.isfinite(t).all(), name
    compare(out, r, e, "out")


def test_gradients_against_differences():
    """Central differences of the 64-bit block along random directions."""
    require_gpu()
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    T, H, I = 130, 72, 136
    s = make(T, H, I, seed=4)
    ffn = MoKFeedForward(H, I, T)
    ffn.forward(s["x"], s["W1"], s["W3"], s["W2"])
    got = ffn.backward(s["x"], s["W1"], s["W3"], s["W2"], s["dout"])
    g = torch.Generator(device="cuda").manual_seed(5)
    v = {k: s[k].double() for k in ("x", "W1", "W3", "W2")}

    def loss(x, W1, W3, W2):
        h = x @ W1
        return ((h * torch.sigmoid(h) * (x @ W3) @ W2) * s["dout"].double()).sum()

    for k, grad in (("x", "dX"), ("W1", "dW1"), ("W3", "dW3"), ("W2", "dW2")):
        d = torch.randn(v[k].shape, generator=g, device="cuda", dtype=torch.float64)
        eps = 1e-5
        diff = (loss(**dict(v, **{k: v[k] + eps * d})) - loss(**dict(v, **{k: v[k] - eps * d}))) / (2 * eps)
        # each gradient element is off by at most a few roundings, independent along d
        size = float((got[grad].double().square()).sum().sqrt())
        assert abs(float(diff - (got[grad].double() * d).sum())) <= 6 * 1.8e-3 * ROUNDINGS[grad] ** 0.5 * size, k


def test_same_as_one_expert():
    """The layer with one expert, whose score is 1, is the same block."""
    require_gpu()
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    from mixture_experts_layer_side_gb300.inputs import Shape
    from mixture_experts_layer_side_gb300.layer import MoKLayer
    T, H, I = 384, 256, 128
    s = make(T, H, I, seed=6)
    layer = MoKLayer(Shape(T, H, I, 1, 1))
    layer.build_schedule(torch.zeros((T, 1), dtype=torch.int32, device="cuda"))
    one = torch.ones((T, 1), device="cuda")
    W = [s[k].unsqueeze(0).contiguous() for k in ("W1", "W3", "W2")]
    out = layer.forward(s["x"], one, *W)
    g = layer.backward(s["x"], one, *W, s["dout"])
    ffn = MoKFeedForward(H, I, T)
    mine = ffn.forward(s["x"], s["W1"], s["W3"], s["W2"])
    grads = ffn.backward(s["x"], s["W1"], s["W3"], s["W2"], s["dout"])
    for a, b in ((out, mine), (g["dX"], grads["dX"]), (g["dW1"][0], grads["dW1"]), (g["dW2"][0], grads["dW2"])):
        assert float((a.double() - b.double()).norm() / b.double().norm()) <= 8e-3


def test_graph_and_stream():
    require_gpu()
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    T, H, I = 200, 256, 384
    s = make(T, H, I, seed=7)
    w = s["W1"], s["W3"], s["W2"]
    ffn = MoKFeedForward(H, I, T)
    few = s["x"][:7].contiguous()

    def step():
        return ffn.forward(s["x"], *w), ffn.backward(s["x"], *w, s["dout"]), ffn.infer(few, *w)

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = ffn.forward(s["x"], *w, stream=side)
    got = ffn.backward(s["x"], *w, s["dout"], stream=side)
    one = ffn.infer(few, *w, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(one, want[2]) and all(torch.equal(got[k], want[1][k]) for k in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(2):
        for t in (held[0], held[2], *held[1].values()):
            t.zero_()
        graph.replay()
        assert torch.equal(held[0], want[0]) and torch.equal(held[2], want[2])
        assert all(torch.equal(held[1][k], want[1][k]) for k in got)
    ffn.check()
