"""The residual join, dropout and the dense feed-forward block where calls
differ from the usual ones: rows apart in other ways for each tensor, NaN
between and beside rows, outputs among other data, very many rows, offsets past
32 bits, the longest rows, calls between a forward pass and its backward pass.
Bounds are those of the formulas' tests."""

import os
import subprocess
import sys

import pytest
import torch

import test_ffn_gpu as ffn_cases
import test_residual_gpu as join_cases
from _helpers import require_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = join_cases.EPS
NAMES = ("dx", "dy", "dw_out", "dgate", "dw_next")


def among_nan(t, lead, pad):
    """The same matrix with its rows `pad` elements apart and `lead` from the start of the memory, NaN all around."""
    T, H = t.shape
    full = torch.full((lead + (T + 1) * (H + pad),), float("nan"), dtype=t.dtype, device="cuda")
    view = full[lead:lead + T * (H + pad)].view(T, H + pad)[:, :H]
    view.copy_(t)
    return view, full


def around(view, full):
    """What lies outside the matrix."""
    mask = torch.ones(full.numel(), dtype=torch.bool, device="cuda")
    offset = (view.data_ptr() - full.data_ptr()) // full.element_size()
    mask.as_strided(view.shape, view.stride(), offset).fill_(False)
    return full[mask]


@pytest.mark.parametrize("types", ["bf16", "mixed", "f32"])
@pytest.mark.parametrize("T,H,groups,p", [(37, 512, 1, 0.25), (37, 515, 37, 0.25), (400, 7, 4, 0.0), (700, 96, 700, 0.25),
                                          (41, 4104, 41, 0.0), (23, 9001, 1, 0.25)])
def test_every_tensor_apart_in_its_own_way(types, T, H, groups, p):
    require_gpu()
    from mixture_experts_layer_side_gb300.dropout import MoKDropout
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    s = join_cases.inputs(T, H, types, True, groups, True)
    drop = MoKDropout(p, seed=11) if p else None
    r, e = join_cases.reference(s, T, H, 0.5, drop)
    S, B = join_cases.TYPES[types]
    res = MoKResidual(H, T, eps=EPS)
    kw = dict(w_out=s["w_out"], gate=s["gate"], w_next=s["w_next"], scale=0.5, dropout=drop, call=5)
    x, y, dx, dn = (among_nan(s[k], lead, pad)[0] for k, lead, pad in (("x", 1, 3), ("y", 8, 0), ("dx", 0, 8), ("dn", 5, 1)))
    out, out_all = among_nan(torch.empty((T, H), dtype=S, device="cuda"), 3, 5)
    nxt, nxt_all = among_nan(torch.empty((T, H), dtype=B, device="cuda"), 2, 16)
    res.forward(x, y, **kw, out=out, out_next=nxt)
    join_cases.compare((out, nxt), r, e, ("x", "n"))
    gx, gx_all = among_nan(torch.empty((T, H), dtype=S, device="cuda"), 7, 1)
    gy, gy_all = among_nan(torch.empty((T, H), dtype=B, device="cuda"), 0, 2)
    got = res.backward(dx, dn, x, y, **kw, dx=gx, dy=gy)
    join_cases.compare([got[k] for k in NAMES], r, e, NAMES)
    for view, full in ((out, out_all), (nxt, nxt_all), (gx, gx_all), (gy, gy_all)):
        assert torch.isnan(around(view, full)).all()
    # dx and dy in the place of what they come from
    got = res.backward(dx, dn, x, y, **kw, dx=dx, dy=y)
    join_cases.compare([got[k] for k in NAMES], r, e, NAMES)


@pytest.mark.parametrize("H", [256, 259, 2048])
def test_a_bad_row_stays_alone(H):
    """NaN and infinities in one row reach no other row."""
    require_gpu()
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    T = 33
    s = join_cases.inputs(T, H, "bf16", True, 0, True)
    res = MoKResidual(H, T, eps=EPS)
    kw = dict(w_out=s["w_out"], w_next=s["w_next"])
    good = res.forward(s["x"], s["y"], **kw), res.backward(s["dx"], s["dn"], s["x"], s["y"], **kw)
    bad = {k: s[k].clone() for k in ("x", "y", "dx", "dn")}
    bad["x"][7] = float("nan")
    bad["y"][7, ::2] = float("inf")
    bad["y"][20] = -torch.finfo(BF16).max
    bad["dx"][20, 0] = float("inf")
    bad["dn"][7, -1] = float("nan")
    rest = [i for i in range(T) if i not in (7, 20)]
    got = res.forward(bad["x"], bad["y"], **kw), res.backward(bad["dx"], bad["dn"], bad["x"], bad["y"], **kw)
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip(good[0], got[0]))
    assert all(torch.equal(good[1][k][rest], got[1][k][rest]) for k in ("dx", "dy"))


@pytest.mark.parametrize("T,H", [(200000, 8), (100001, 3)])
def test_very_many_rows(T, H):
    """Sums of many rows: 3,648 workers at least take T / 3,648 of them one after the other, more than the 32 that U_COL
    counts: the bounds are widened by T / 1,216 roundings."""
    require_gpu()
    from mixture_experts_layer_side_gb300.dropout import MoKDropout
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    s = join_cases.inputs(T, H, "f32", True, 1, True)
    drop, res = MoKDropout(0.25, seed=3), MoKResidual(H, T, eps=EPS)
    r, e = join_cases.reference(s, T, H, 0.5, drop)
    for k in ("dw_out", "dgate", "dw_next"):
        e[k] = e[k] * (1 + (T / 1216) * 2.0 ** -24 / join_cases.U_COL)
    kw = dict(w_out=s["w_out"], gate=s["gate"], w_next=s["w_next"], scale=0.5, dropout=drop, call=5)
    join_cases.compare(res.forward(s["x"], s["y"], **kw), r, e, ("x", "n"))
    got = res.backward(s["dx"], s["dn"], s["x"], s["y"], **kw)
    join_cases.compare([got[k] for k in NAMES], r, e, NAMES)


def test_join_past_32_bits():
    """More than 2^31 elements, all but the last rows' zero."""
    require_gpu()
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    H, last = 16384, 50
    T = 2**31 // H + 100
    x = torch.zeros((T, H), dtype=BF16, device="cuda")
    y = torch.zeros_like(x)
    s = join_cases.inputs(last, H, "bf16", True, 0, True)
    x[-last:], y[-last:] = s["x"], s["y"]
    kw = dict(w_out=s["w_out"], w_next=s["w_next"])
    res = MoKResidual(H, T, eps=EPS)
    r, e = join_cases.reference(s, last, H, 1.0, None)
    got = res.forward(x, y, **kw)
    join_cases.compare([t[-last:] for t in got], r, e, ("x", "n"))
    assert not got[0][:-last].any() and not got[1][:-last].any()
    dx, dn = got
    dx.zero_(), dn.zero_()
    dx[-last:], dn[-last:] = s["dx"], s["dn"]
    got = res.backward(dx, dn, x, y, **kw, dx=dx, dy=dn)
    join_cases.compare([got["dx"][-last:], got["dy"][-last:], got["dw_out"], got["dw_next"]], r, e,
                       ("dx", "dy", "dw_out", "dw_next"))


@pytest.mark.parametrize("rows,cols,lead,pad,dtype", [(1, 100003, 0, 0, BF16), (1, 100001, 3, 0, F32), (50, 333, 1, 2, BF16),
                                                      (9, 264, 0, 5, F32), (300, 1, 0, 4, BF16), (70, 7, 2, 0, F32)])
def test_dropout_among_nan(rows, cols, lead, pad, dtype):
    """The same elements are kept wherever they lie; what lies around them stays, in place too."""
    require_gpu()
    from mixture_experts_layer_side_gb300.dropout import MoKDropout
    x = torch.randn((rows, cols), generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    drop = MoKDropout(0.3, seed=21)
    keep = torch.from_numpy(join_cases.kept(rows, cols, 0.3, 21, 9)).cuda()
    ref = torch.where(keep, x.double() / (1 - round(0.3 * 65536) / 65536), 0.0)
    apart, full = among_nan(x, lead, pad)
    out, out_all = among_nan(torch.empty_like(x), 8 - lead, pad + 1)
    drop.forward(apart, call=9, out=out)
    bound = (join_cases.half_step(dtype) + 2.0 ** -23) * ref.abs() * 1.001
    assert bool(((out.double() - ref).abs() <= bound).all()) and torch.isnan(around(out, out_all)).all()
    want = out.clone()
    drop.forward(apart, call=9, out=apart)
    assert torch.equal(apart, want) and torch.isnan(around(apart, full)).all()


def compare_elements(got, r, e, name):
    """The elements' bounds alone.  (The whole's error is that of independent roundings only where there are many of
    them: with one token and eight hidden values, one value's rounding of up to 2^-8 = 3.9e-3 can be that of the whole
    gradient of W2, where two independent ones of many make 1.8e-3 sqrt 2 = 2.5e-3.)"""
    err = (got.double() - r[name]).abs()
    bound = ffn_cases.HALF * r[name].abs() + 1.02 * e[name] + 1e-30
    assert got.dtype == BF16 and bool((err <= bound).all()), (name, float((err / bound).max()))


@pytest.mark.parametrize("H,I", [(72, 40), (8, 264), (520, 8)])
def test_ffn_of_every_few_tokens(H, I):
    require_gpu()
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    most = 129
    s = ffn_cases.make(most, H, I, seed=8)
    w = s["W1"], s["W3"], s["W2"]
    ffn = MoKFeedForward(H, I, most)
    for T in (1, 2, 3, 4, 5, 7, 8, 9, 16, 17, 31, 32, 33, 63, 65, 127, 128, 129):
        part = {k: v[:T].contiguous() if k in ("x", "dout") else v for k, v in s.items()}
        r, e = ffn_cases.reference(part)
        out = ffn.forward(part["x"], *w)
        one = ffn.infer(part["x"], *w)  # (between a forward pass and its backward pass)
        got = ffn.backward(part["x"], *w, part["dout"])
        for name, t in dict(got, out=out, one=one).items():
            compare_elements(t, r, e, "out" if name == "one" else name)
    ffn.check()


@pytest.mark.parametrize("T", [1, 3, 200])
@pytest.mark.parametrize("H,I", [(131072, 8), (8, 131072)])
def test_ffn_longest_rows(T, H, I):
    require_gpu()
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    s = ffn_cases.make(T, H, I, seed=9, std=0.01)
    w = s["W1"], s["W3"], s["W2"]
    r, e = ffn_cases.reference(s)
    ffn = MoKFeedForward(H, I, T)
    out = ffn.forward(s["x"], *w)
    got = ffn.backward(s["x"], *w, s["dout"])
    for name, t in dict(got, out=out).items():
        compare_elements(t, r, e, name)
    compare_elements(ffn.infer(s["x"], *w), r, e, "out")
    ffn.check()


@pytest.mark.parametrize("T", [3, 40, 300])
def test_ffn_bad_row_stays_alone(T):
    require_gpu()
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    H, I = 264, 136
    s = ffn_cases.make(T, H, I, seed=10)
    w = s["W1"], s["W3"], s["W2"]
    ffn = MoKFeedForward(H, I, T)
    bad = s["x"].clone()
    bad[1] = float("nan")
    rest = [i for i in range(T) if i != 1]

    def step(x):
        return ffn.forward(x, *w), ffn.infer(x, *w), ffn.backward(x, *w, s["dout"])["dX"]

    for a, b in zip(step(s["x"]), step(bad)):
        assert torch.equal(a[rest], b[rest]) and torch.isnan(b[1]).all()


def test_ffn_past_32_bits():
    """More than 2^31 hidden values: the last tokens' results, and gradients that sum over all tokens."""
    require_gpu()
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    H, I, last = 16, 8200, 300
    T = 2**31 // I + 1000
    s = ffn_cases.make(T, H, I, seed=11, std=0.2)
    w = s["W1"], s["W3"], s["W2"]
    ffn = MoKFeedForward(H, I, T)
    out = ffn.forward(s["x"], *w)
    got = ffn.backward(s["x"], *w, s["dout"])
    ffn.check()
    part = dict(s, x=s["x"][-last:], dout=s["dout"][-last:])
    r, e = ffn_cases.reference(part)
    ffn_cases.compare(out[-last:], r, e, "out")
    ffn_cases.compare(got["dX"][-last:], r, e, "dX")
    # the last columns of I by themselves, over all tokens
    cols = dict(s, W1=s["W1"][:, -32:], W3=s["W3"][:, -32:], W2=s["W2"][-32:])
    r, e = ffn_cases.reference(cols)
    for name, t in (("dW1", got["dW1"][:, -32:]), ("dW3", got["dW3"][:, -32:]), ("dW2", got["dW2"][-32:])):
        ffn_cases.compare(t, r, e, name)


def test_two_graphs_with_objects_of_their_own():
    require_gpu()
    from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    T, H, I = 150, 256, 128
    sets, graphs, held, want = [], [], [], []
    for i in range(2):
        s = dict(ffn_cases.make(T, H, I, seed=20 + i), w=torch.ones(H, dtype=BF16, device="cuda"))
        ffn, res = MoKFeedForward(H, I, T), MoKResidual(H, T)

        def step(s=s, ffn=ffn, res=res):
            w = s["W1"], s["W3"], s["W2"]
            y = ffn.forward(s["x"], *w)
            x, n = res.forward(s["x"], y, w_next=s["w"])
            g = res.backward(s["dout"], n, x, y, w_next=s["w"])
            return [y, x, n, *ffn.backward(s["x"], *w, g["dy"]).values(), g["dx"], g["dw_next"]]

        want.append(step())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(step())
        graphs.append(graph)
        sets.append((s, ffn, res))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, held):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


FIRST_CALLS = """
import torch
from mixture_experts_layer_side_gb300.dropout import MoKDropout
from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
from mixture_experts_layer_side_gb300.residual import MoKResidual
bf16, cuda = torch.bfloat16, "cuda"
for T, H, I in ((2, 256, 128), (70, 520, 264), (3000, 1024, 1024)):
    g = torch.Generator(device=cuda).manual_seed(T)
    x, dout = ((torch.randn((T, H), generator=g, device=cuda)).to(bf16) for _ in range(2))
    W1, W3, W2 = ((0.05 * torch.randn(s, generator=g, device=cuda)).to(bf16) for s in ((H, I), (H, I), (I, H)))
    w = torch.ones(H, dtype=bf16, device=cuda)
    ffn, res, drop = MoKFeedForward(H, I, T), MoKResidual(H, T), MoKDropout(0.25)

    def step():
        y = ffn.forward(x, W1, W3, W2)
        x2, n = res.forward(x, y, w_out=w, w_next=w, dropout=drop)
        b = res.backward(dout, n, x2, y, w_out=w, w_next=w, dropout=drop)
        d = ffn.backward(x, W1, W3, W2, b["dy"])
        return [y, x2, n, b["dx"], b["dw_out"], *d.values(), ffn.infer(n, W1, W3, W2), drop.forward(y)]

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in held]
    assert all(torch.equal(a, b) for a, b in zip(got, step())), (T, H, I)
    ffn.check()
print("captured")
"""


def test_first_calls_of_a_process_are_captured():
    """Nothing of a kernel's first launch (its shared memory, how many clusters fit) hinders a capture."""
    require_gpu()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "captured" in done.stdout, done.stderr[-3000:]
