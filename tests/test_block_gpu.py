"""Two blocks of a model as they are trained: the norm of the first, a dense
feed-forward block, its join with the residual stream (norms on both sides,
gate, dropout), the routed layer and its join, forward and backward, against
the same in 64 bits, eager, on another stream and captured.

Every tensor between two calls is rounded to bf16 once, which is off by
1.7e-3 of the whole (root mean square; 1.8e-3 is used), and the roundings on
the way to a result are independent.  Norms and joins pass a relative error on
with a factor of about 1, products and gates too; 2 is allowed."""

import pytest
import torch

from _helpers import require_gpu

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
EPS = 1e-6
T, H, I, E, K = 384, 256, 128, 4, 2
ROUNDING = 1.8e-3


def make(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0, mean=0.0):
        return (mean + std * torch.randn(shape, generator=g, device="cuda")).to(BF16)

    s = dict(x=randn(T, H, std=2.0), dx2=randn(T, H), dn2=randn(T, H), gate=randn(8, H, std=0.5, mean=1.0))
    for name in ("w0", "w_out", "w1", "w2"):
        s[name] = randn(H, std=0.2, mean=1.0)
    for name, e in (("d", ()), ("e", (E,))):
        s.update({f"{name}1": randn(*e, H, I, std=0.1), f"{name}3": randn(*e, H, I, std=0.1),
                  f"{name}2": randn(*e, I, H, std=0.1)})
    s["idx"] = torch.stack([torch.randperm(E, generator=g, device="cuda")[:K] for _ in range(T)]).int()
    s["scores"] = torch.rand((T, K), generator=g, device="cuda") * 0.5 + 0.25
    return s


class Blocks:
    def __init__(self, s):
        from mixture_experts_layer_side_gb300.dropout import MoKDropout
        from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
        from mixture_experts_layer_side_gb300.inputs import Shape
        from mixture_experts_layer_side_gb300.layer import MoKLayer
        from mixture_experts_layer_side_gb300.residual import MoKResidual
        self.s = s
        self.res, self.drop, self.ffn = MoKResidual(H, T, eps=EPS), MoKDropout(0.25, seed=5), MoKFeedForward(H, I, T)
        self.layer = MoKLayer(Shape(T, H, I, E, K))
        self.layer.build_schedule(s["idx"])

    def step(self, call=0):
        """Gradients by name, and the last join's outputs."""
        s = self.s
        dense, experts = [s[k] for k in ("d1", "d3", "d2")], [s[k] for k in ("e1", "e3", "e2")]
        n0 = self.res.norm(s["x"], s["w0"])
        y0 = self.ffn.forward(n0, *dense)
        join0 = dict(w_out=s["w_out"], gate=s["gate"], w_next=s["w1"], dropout=self.drop, call=call)
        x1, n1 = self.res.forward(s["x"], y0, **join0)
        y1 = self.layer.forward(n1, s["scores"], *experts)
        join1 = dict(w_next=s["w2"], scale=0.5)
        x2, n2 = self.res.forward(x1, y1, **join1)
        g1 = self.res.backward(s["dx2"], s["dn2"], x2, y1, **join1)
        e = self.layer.backward(n1, s["scores"], *experts, g1["dy"])
        g0 = self.res.backward(g1["dx"], e["dX"], x1, y0, **join0)
        d = self.ffn.backward(n0, *dense, g0["dy"])
        dx, dw0 = self.res.norm_backward(d["dX"], s["x"], s["w0"], dx_new=g0["dx"])
        return dict(x2=x2, n2=n2, x=dx, w0=dw0, d1=d["dW1"], d3=d["dW3"], d2=d["dW2"], w_out=g0["dw_out"],
                    gate=g0["dgate"], w1=g0["dw_next"], e1=e["dW1"], e3=e["dW3"], e2=e["dW2"], w2=g1["dw_next"])

    def mask(self, call):
        return self.drop.forward(torch.ones((T, H), device="cuda"), call=call).double()


def reference(s, mask):
    v = {k: s[k].double().requires_grad_() for k in s if k not in ("idx", "dx2", "dn2", "scores")}

    def norm(x, w):
        return x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * w

    def ffn(x, w1, w3, w2):
        h = x @ w1
        return (h * torch.sigmoid(h) * (x @ w3)) @ w2

    y0 = ffn(norm(v["x"], v["w0"]), v["d1"], v["d3"], v["d2"])
    x1 = v["x"] + v["gate"].repeat_interleave(T // 8, 0) * mask * norm(y0, v["w_out"])
    n1 = norm(x1, v["w1"])
    y1 = 0
    for e in range(E):
        score = (s["scores"].double() * (s["idx"] == e)).sum(1, keepdim=True)
        y1 = y1 + score * ffn(n1, v["e1"][e], v["e3"][e], v["e2"][e])
    x2 = x1 + 0.5 * y1
    n2 = norm(x2, v["w2"])
    ((x2 * s["dx2"].double()).sum() + (n2 * s["dn2"].double()).sum()).backward()
    return dict({k: t.grad for k, t in v.items()}, x2=x2.detach(), n2=n2.detach())


# Roundings of bf16 on the way to each: n0, a, y0, x1, n1, then the layer's (h, u, a, their gradients, a row's sums)
FORWARD, LAYER, JOIN, DENSE = 5, 8, 3, 4


def tolerance(name):
    n = FORWARD + LAYER + (0 if name in ("x2", "n2") else JOIN + LAYER + JOIN + DENSE)
    return 2 * ROUNDING * n ** 0.5


def test_blocks_against_64_bits():
    require_gpu()
    s = make()
    blocks = Blocks(s)
    for call in (0, 3):
        got, want = blocks.step(call), reference(s, blocks.mask(call))
        for name in got:
            err = float((got[name].double() - want[name]).norm() / want[name].norm())
            assert got[name].shape == want[name].shape and err <= tolerance(name), (name, err, tolerance(name))
    blocks.ffn.check()


def test_blocks_on_a_stream_and_in_a_graph():
    require_gpu()
    s = make(seed=1)
    blocks = Blocks(s)
    want = [blocks.step(i) for i in range(3)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = blocks.step(1)
    side.synchronize()
    assert all(torch.equal(got[k], want[1][k]) for k in got)
    number = torch.zeros(1, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = blocks.step(number)
        number += 1
    for i in range(3):
        for t in held.values():
            t.zero_()
        graph.replay()
        assert all(torch.equal(held[k], want[i][k]) for k in held), i
    blocks.ffn.check()
