"""The residual join and dropout against their formulas in 64 bits, with error
bounds that follow from the arithmetic: outputs in bf16 are off by at most half
a step, 2^-9 of the value at its larger end (2^-8 counting the step below a power
of two), 32-bit sums and products by a few 2^-24 of the terms' magnitudes."""

import numpy as np
import pytest
import torch

from _helpers import require_gpu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": (BF16, BF16), "mixed": (F32, BF16), "f32": (F32, F32)}
EPS = 1e-6
# A row's sum: at most 16 terms a thread one after the other, then 10 levels, the
# product and the root: under 32 roundings, and as many in what is made of it.
U = 64 * 2.0 ** -24
# Column sums go on over a worker's rows (T / 152 at most 32 here, or 4) and 16
# parts of at most 304, and each term has U by itself.
U_COL = U + (32 + 19 + 16 + 4) * 2.0 ** -24


def half_step(t):
    return torch.finfo(t).eps / 2


def philox_np(blocks, call, seed):
    """Philox-4x32-10 on numpy words: uint32 [blocks, 4]."""
    m0, m1, w0, w1 = (np.uint64(v) for v in (0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85))
    low, s32 = np.uint64(0xFFFFFFFF), np.uint64(32)
    b = np.asarray(blocks, dtype=np.uint64)
    c = [b & low, b >> s32, np.full_like(b, call & 0xFFFFFFFF), np.full_like(b, call >> 32)]
    k0, k1 = np.uint64(seed & 0xFFFFFFFF), np.uint64(seed >> 32)
    for _ in range(10):
        p0, p1 = c[0] * m0, c[2] * m1
        c = [(p1 >> s32) ^ c[1] ^ k0, p1 & low, (p0 >> s32) ^ c[3] ^ k1, p0 & low]
        k0, k1 = (k0 + w0) & low, (k1 + w1) & low
    return np.stack(c, 1).astype(np.uint32)


def kept(T, H, p, seed, call, first=0):
    i = np.arange(first, first + T * H, dtype=np.uint64)
    b0 = int(i[0]) >> 3
    words = philox_np(np.arange(b0, (int(i[-1]) >> 3) + 1), call, seed)
    bits = np.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)
    return (bits[(i - np.uint64(8 * b0)).astype(np.int64)] >= round(p * 65536)).reshape(T, H)


def test_generator_known_answers():
    # the published vectors of Philox-4x32-10: all zeros, all ones, digits of pi
    assert philox_np([0], 0, 0)[0].tolist() == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    ones = 2**64 - 1
    assert philox_np([ones], ones, ones)[0].tolist() == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def rows(g, T, H, dtype, pad, std=1.0):
    full = (std * torch.randn((T, H + pad), generator=g)).to(dtype).cuda()
    return full[:, :H]


def inputs(T, H, types, post, groups, nxt, pad=0, seed=0):
    S, B = TYPES[types]
    g = torch.Generator().manual_seed(seed)
    s = dict(x=rows(g, T, H, S, pad, 2.0), y=rows(g, T, H, B, pad), dx=rows(g, T, H, S, pad),
             dn=rows(g, T, H, B, pad) if nxt else None)
    s["w_out"] = (1 + 0.3 * torch.randn(H, generator=g)).to(B).cuda() if post else None
    s["w_next"] = (1 + 0.3 * torch.randn(H, generator=g)).to(B).cuda() if nxt else None
    s["gate"] = torch.randn((groups, H), generator=g).to(B).cuda() if groups else None
    return s


def n64(t):
    return None if t is None else t.double().cpu().numpy()


def reference(s, T, H, scale, drop):
    """Outputs in 64 bits and, by the same names, bounds on what 32-bit arithmetic adds to their rounding."""
    x, y, dxo, dn = n64(s["x"]), n64(s["y"]), n64(s["dx"]), n64(s["dn"])
    w_out, w_next, gate = n64(s["w_out"]), n64(s["w_next"]), n64(s["gate"])
    G = 0 if gate is None else gate.shape[0]
    mask = np.ones((T, H))
    if drop:
        p = round(drop.p * 65536) / 65536
        mask = kept(T, H, drop.p, drop.seed, 5) / (1 - p) if p < 1 else np.zeros((T, H))
    f = scale * (np.repeat(gate, T // G, 0) if G else np.ones((T, H)))
    z, yh = y, None
    if w_out is not None:
        ry = 1 / np.sqrt((y * y).mean(1, keepdims=True) + EPS)
        yh = y * ry
        z = yh * w_out
    r, e = {}, {}
    d = np.where(mask > 0, mask * z, 0)
    r["x"] = x + f * d
    e["x"] = U * (np.abs(x) + np.abs(f * d))
    if w_next is not None:
        rn = 1 / np.sqrt((r["x"] ** 2).mean(1, keepdims=True) + EPS)
        r["n"] = r["x"] * rn * w_next
        e["n"] = 2 * U * (np.abs(x) + np.abs(f * d)) * rn * np.abs(w_next) + 2 * U * np.abs(r["n"])
    # backward, with x as x'
    g, eg = dxo, U * np.abs(dxo)
    if dn is not None:
        rn = 1 / np.sqrt((x ** 2).mean(1, keepdims=True) + EPS)
        xh, t = x * rn, dn * w_next
        g = dxo + rn * (t - xh * (t * xh).mean(1, keepdims=True))
        eg = U * (np.abs(dxo) + rn * (np.abs(t) + 2 * np.abs(xh) * np.abs(t * xh).mean(1, keepdims=True)))
        r["dw_next"], e["dw_next"] = (dn * xh).sum(0), U_COL * np.abs(dn * xh).sum(0)
    r["dx"], e["dx"] = g, eg
    if G:
        both = scale * g * d
        r["dgate"] = both.reshape(G, -1, H).sum(1)
        e["dgate"] = (np.abs(scale * d) * eg + U_COL * np.abs(both)).reshape(G, -1, H).sum(1)
    dz = np.where(mask > 0, g * f * mask, 0)
    ez = np.abs(f * mask) * eg + U * np.abs(dz)
    r["dy"], e["dy"] = dz, ez
    if w_out is not None:
        t = dz * w_out
        et = ez * np.abs(w_out) + U * np.abs(t)
        r["dw_out"], e["dw_out"] = (dz * yh).sum(0), (ez * np.abs(yh) + U_COL * np.abs(dz * yh)).sum(0)
        r["dy"] = ry * (t - yh * (t * yh).mean(1, keepdims=True))
        e["dy"] = ry * (et + np.abs(yh) * (et * np.abs(yh)).mean(1, keepdims=True) +
                        U * (np.abs(t) + 2 * np.abs(yh) * np.abs(t * yh).mean(1, keepdims=True)))
    return r, e


def compare(got, r, e, names):
    for name, t in zip(names, got):
        if name not in r:
            assert t is None, name
            continue
        assert t.dtype in (BF16, F32)
        err = np.abs(n64(t).reshape(r[name].shape) - r[name])
        # (the bf16 below an f32 value that is itself off)
        bound = half_step(t.dtype) * np.abs(r[name]) + 1.01 * e[name] + 1e-37
        assert (err <= bound).all(), (name, float((err / bound).max()))


CASES = [  # T, H, types, post, groups, next, p, pad
    (1, 2048, "mixed", True, 0, True, 0.0, 0),
    (7, 8, "bf16", True, 1, True, 0.0, 0),
    (3, 1, "f32", True, 1, True, 0.0, 0),
    (64, 256, "bf16", True, 64, True, 0.125, 0),
    (65, 264, "mixed", False, 5, True, 0.5, 8),
    (33, 1003, "f32", True, 11, True, 0.3, 5),
    (50, 77, "bf16", True, 10, True, 0.3, 0),
    (1000, 2048, "bf16", True, 8, True, 0.125, 0),
    (300, 7168, "bf16", True, 1, True, 0.0, 0),
    (301, 7168, "mixed", True, 7, True, 0.1, 8),
    (19, 8192, "f32", True, 0, True, 0.1, 0),
    (20, 8200, "bf16", True, 4, True, 0.1, 0),
    (9, 16384, "f32", True, 3, True, 0.1, 0),
    (9, 16383, "mixed", True, 3, True, 0.1, 0),
    (128, 512, "bf16", False, 0, True, 0.0, 0),
    (128, 512, "bf16", True, 0, False, 0.0, 0),
    (128, 512, "f32", False, 1, False, 0.25, 3),
    (128, 512, "mixed", False, 0, False, 0.25, 3),
    (4000, 320, "mixed", True, 1, True, 1.0, 0),
    (2, 4096, "bf16", True, 2, True, 0.99999, 0),
]


@pytest.mark.parametrize("T,H,types,post,groups,nxt,p,pad", CASES)
def test_against_formulas(T, H, types, post, groups, nxt, p, pad):
    require_gpu()
    from mixture_experts_layer_side_gb300.dropout import MoKDropout
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    s = inputs(T, H, types, post, groups, nxt, pad)
    drop = MoKDropout(p, seed=(3 << 40) + 77) if p else None
    res = MoKResidual(H, T + 3, eps=EPS)
    kw = dict(w_out=s["w_out"], gate=s["gate"], w_next=s["w_next"], scale=0.5, dropout=drop, call=5)
    r, e = reference(s, T, H, 0.5, drop)
    forward = res.forward(s["x"], s["y"], **kw)
    compare(forward, r, e, ("x", "n"))
    got = res.backward(s["dx"], s["dn"], s["x"], s["y"], **kw)
    names = ("dx", "dy", "dw_out", "dgate", "dw_next")
    compare([got[k] for k in names], r, e, names)
    # the same bits again, and in place
    again = res.backward(s["dx"], s["dn"], s["x"], s["y"], **kw)
    S, B = TYPES[types]
    x, y = s["x"].clone(), s["y"].clone()
    place = res.forward(x, y, **kw, out=x, out_next=y if nxt else None)
    assert place[0] is x
    for a, b in zip(forward, place):
        assert (a is None and b is None) or torch.equal(a, b)
    dx, dn = s["dx"].clone(), None if s["dn"] is None else s["dn"].clone()
    inplace = res.backward(dx, dn, s["x"], s["y"], **kw, dx=dx, dy=dn)
    for k in names:
        assert (got[k] is None and inplace[k] is None and again[k] is None) or \
            (torch.equal(got[k], inplace[k]) and torch.equal(got[k], again[k])), k


def test_forward_then_differences():
    """Gradients against central differences of the forward pass itself, in f32 on few columns."""
    require_gpu()
    from mixture_experts_layer_side_gb300.dropout import MoKDropout
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    T, H, h = 6, 24, 2.0 ** -6
    s = inputs(T, H, "f32", True, 3, True)
    drop = MoKDropout(0.25, seed=9)
    res = MoKResidual(H, T, eps=EPS)

    def loss(v):
        a, n = res.forward(v["x"], v["y"], v["w_out"], v["gate"], v["w_next"], 0.5, drop, 2)
        return (a.double() * s["dx"].double()).sum() + (n.double() * s["dn"].double()).sum()

    x_new, _ = res.forward(s["x"], s["y"], s["w_out"], s["gate"], s["w_next"], 0.5, drop, 2)
    got = res.backward(s["dx"], s["dn"], x_new, s["y"], s["w_out"], s["gate"], s["w_next"], 0.5, drop, 2)
    for name, grad in (("x", "dx"), ("y", "dy"), ("w_out", "dw_out"), ("gate", "dgate"), ("w_next", "dw_next")):
        flat = got[grad].reshape(-1)
        for i in range(0, flat.numel(), max(1, flat.numel() // 12)):
            f = []
            for sign in (1, -1, 2, -2):
                v = {k: t.clone() if k == name else t for k, t in s.items() if t is not None}
                v[name].reshape(-1)[i] += sign * h
                f.append(float(loss(v)))
            # the fourth-order formula: what is left is h^4 / 30 of the fifth derivative, and the f32 rounding of
            # 2 T H outputs of size ~4 over h
            d = (8 * (f[0] - f[1]) - (f[2] - f[3])) / (12 * h)
            assert abs(d - float(flat[i])) <= 1e-3 * (1 + abs(d)), (name, i, d, float(flat[i]))


def test_norm_alone():
    require_gpu()
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    for T, H, types in ((5, 7168, "mixed"), (40, 100, "f32"), (17, 16384, "bf16")):
        s = inputs(T, H, types, False, 0, True)
        res = MoKResidual(H, T, eps=EPS)
        r, e = reference(dict(s, y=s["y"] * 0, gate=None), T, H, 1.0, None)
        compare([res.norm(s["x"], s["w_next"])], r, e, ("n",))
        dx, dw = res.norm_backward(s["dn"], s["x"], s["w_next"], dx_new=s["dx"])
        compare([dx, dw], r, e, ("dx", "dw_next"))
        r, e = reference(dict(s, y=s["y"] * 0, dx=s["dx"] * 0), T, H, 1.0, None)
        compare(res.norm_backward(s["dn"], s["x"], s["w_next"]), r, e, ("dx", "dw_next"))


def test_missing_gradients():
    require_gpu()
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    T, H = 30, 640
    s = inputs(T, H, "bf16", True, 1, True)
    res = MoKResidual(H, T)
    w = dict(w_out=s["w_out"], gate=s["gate"], w_next=s["w_next"])
    zero = torch.zeros_like(s["dx"])
    a, b = res.backward(None, s["dn"], s["x"], s["y"], **w), res.backward(zero, s["dn"], s["x"], s["y"], **w)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    a, b = res.backward(s["dx"], None, s["x"], s["y"], **w), res.backward(s["dx"], zero, s["x"], s["y"], **w)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    assert not a["dw_next"].any()


def test_no_rows():
    require_gpu()
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    res = MoKResidual(64, 4)
    s = inputs(0, 64, "bf16", True, 1, True)
    x, n = res.forward(s["x"], s["y"], s["w_out"], s["gate"], s["w_next"])
    assert x.shape == n.shape == (0, 64)
    torch.cuda.synchronize()
    junk = [torch.full((64,), float("nan"), device="cuda") for _ in range(8)]
    del junk
    got = res.backward(s["dx"], s["dn"], s["x"], s["y"], s["w_out"], s["gate"], s["w_next"])
    for k in ("dw_out", "dgate", "dw_next"):
        assert not got[k].any(), k


def test_dropped_infinities_stay_out():
    """An infinity or NaN at a dropped element changes nothing, forward or backward."""
    require_gpu()
    from mixture_experts_layer_side_gb300.dropout import MoKDropout
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    for T, H in ((40, 96), (40, 97)):
        s = inputs(T, H, "f32", False, 4, False)
        drop = MoKDropout(0.5, seed=4)
        res = MoKResidual(H, T)
        off = torch.from_numpy(~kept(T, H, 0.5, 4, 0)).cuda()
        bad = torch.where(off, torch.tensor([float("inf"), float("nan"), -float("inf")], device="cuda").repeat(T * H)[:T * H]
                          .reshape(T, H), s["y"])
        kw = dict(gate=s["gate"], dropout=drop)
        assert torch.equal(res.forward(s["x"], s["y"], **kw)[0], res.forward(s["x"], bad, **kw)[0])
        a, b = (res.backward(s["dx"], None, s["x"], v, **kw) for v in (s["y"], bad))
        for k in ("dx", "dy", "dgate"):
            assert torch.equal(a[k], b[k]) and torch.isfinite(a[k]).all(), k
        assert torch.equal(drop.forward(bad), drop.forward(s["y"])) and not drop.forward(bad)[off].any()


def test_zero_rows_and_lowest_values():
    require_gpu()
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    T, H = 4, 256
    s = inputs(T, H, "bf16", True, 0, True)
    s["x"][1], s["y"][1], s["y"][2] = 0, 0, 0
    s["y"][3] = 2.0 ** -100
    res = MoKResidual(H, T, eps=EPS)
    kw = dict(w_out=s["w_out"], w_next=s["w_next"])
    r, e = reference(s, T, H, 1.0, None)
    compare(res.forward(s["x"], s["y"], **kw), r, e, ("x", "n"))
    got = res.backward(s["dx"], s["dn"], s["x"], s["y"], **kw)
    compare([got[k] for k in ("dx", "dy", "dw_out", "dw_next")], r, e, ("dx", "dy", "dw_out", "dw_next"))


def test_weights_of_other_alignment():
    """Vectors and single elements give the same values (a weight, a stream, a gradient off by one element)."""
    require_gpu()
    from mixture_experts_layer_side_gb300.dropout import MoKDropout
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    T, H = 37, 512
    s = inputs(T, H, "bf16", True, 1, True)
    drop, res = MoKDropout(0.25, seed=1), MoKResidual(H, T, eps=EPS)
    off = torch.empty(H + 1, dtype=BF16, device="cuda")[1:]
    off.copy_(s["w_next"])
    r, e = reference(s, T, H, 1.0, drop)
    kw = dict(w_out=s["w_out"], gate=s["gate"], w_next=off, dropout=drop, call=5)
    compare(res.forward(s["x"], s["y"], **kw), r, e, ("x", "n"))
    got = res.backward(s["dx"], s["dn"], s["x"], s["y"], **kw)
    names = ("dx", "dy", "dw_out", "dgate", "dw_next")
    compare([got[k] for k in names], r, e, names)


@pytest.mark.parametrize("shape,pad,dtype,p", [((5, 328), 0, F32, 0.125), ((1,), 0, BF16, 0.5), ((7, 9, 3), 0, BF16, 0.3),
                                               ((100, 77), 3, F32, 0.3), ((64, 256), 8, BF16, 0.1), ((3, 1000), 1, BF16, 0.9),
                                               ((1000, 4096), 0, BF16, 0.1), ((10, 10), 0, F32, 0.0), ((10, 10), 0, F32, 1.0),
                                               ((0, 10), 0, F32, 0.5)])
def test_dropout(shape, pad, dtype, p):
    require_gpu()
    from mixture_experts_layer_side_gb300.dropout import MoKDropout
    g = torch.Generator().manual_seed(0)
    full = torch.randn((*shape[:-1], shape[-1] + pad), generator=g).to(dtype).cuda()
    x = full[..., :shape[-1]]
    drop = MoKDropout(p, seed=2**63 + 12345)
    out = drop.forward(x, call=2**40 + 1)
    n = x.numel()
    if n:
        pp = round(p * 65536) / 65536
        keep = kept(1, n, p, 2**63 + 12345, 2**40 + 1).reshape(shape)
        ref = np.where(keep, n64(x) / (1 - pp) if p < 1 else 0, 0)
        # one rounding of 1 / (1 - p), one of the product, one to the type
        assert (np.abs(n64(out) - ref) <= (half_step(dtype) + 2 * 2.0 ** -24) * np.abs(ref) * 1.001).all()
        assert n < 1000 or abs(keep.mean() - (1 - p)) <= 6 * (p * (1 - p) / n) ** 0.5 + 1e-9
    assert torch.equal(drop.backward(x, call=2**40 + 1), out)
    number = torch.tensor([2**40 + 1], device="cuda")
    assert torch.equal(drop.forward(x, call=number), out)
    if n > 50 and 0 < p < 1:
        assert not torch.equal(drop.forward(x, call=0), out)
    if pad:
        keep_rest = full.clone()
        drop.forward(x, call=2**40 + 1, out=x)
        assert torch.equal(x, out) and torch.equal(full[..., shape[-1]:], keep_rest[..., shape[-1]:])


def test_dropout_far_elements():
    """Elements past 2^32: the counter's upper words, offsets past 32 bits."""
    require_gpu()
    from mixture_experts_layer_side_gb300.dropout import MoKDropout
    n = 2**32 + 4096
    x = torch.ones(n, dtype=BF16, device="cuda")
    drop = MoKDropout(0.5, seed=1)
    out = drop.forward(x, call=3, out=x)
    for first in (0, 2**31 - 512, 2**32 - 512, n - 1000):
        keep = kept(1, 1000, 0.5, 1, 3, first=first)[0]
        assert np.array_equal(n64(out[first:first + 1000]) == 2.0, keep), first


def test_graph_counts_calls():
    """A captured join and its gradient: each replay has the mask of the counter's value."""
    require_gpu()
    from mixture_experts_layer_side_gb300.dropout import MoKDropout
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    T, H = 50, 768
    s = inputs(T, H, "bf16", True, 1, True)
    drop, res = MoKDropout(0.25, seed=8), MoKResidual(H, T)
    number = torch.zeros(1, dtype=torch.int64, device="cuda")
    w = dict(w_out=s["w_out"], gate=s["gate"], w_next=s["w_next"], dropout=drop)

    def step():
        x, n = res.forward(s["x"], s["y"], **w, call=number)
        return x, n, res.backward(s["dx"], s["dn"], x, s["y"], **w, call=number)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x, n, got = step()
        number += 1
    for i in range(3):
        graph.replay()
        rx, rn = res.forward(s["x"], s["y"], **w, call=i)
        want = res.backward(s["dx"], s["dn"], rx, s["y"], **w, call=i)
        assert torch.equal(x, rx) and torch.equal(n, rn)
        for k in want:
            assert torch.equal(got[k], want[k]), (i, k)


def test_other_stream():
    require_gpu()
    from mixture_experts_layer_side_gb300.dropout import MoKDropout
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    T, H = 64, 1024
    s = inputs(T, H, "mixed", True, 1, True)
    drop, res = MoKDropout(0.25, seed=8), MoKResidual(H, T)
    w = dict(w_out=s["w_out"], gate=s["gate"], w_next=s["w_next"], dropout=drop)
    want = res.forward(s["x"], s["y"], **w)
    grads = res.backward(s["dx"], s["dn"], s["x"], s["y"], **w)
    plain = drop.forward(s["x"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = res.forward(s["x"], s["y"], **w, stream=side)
    got_grads = res.backward(s["dx"], s["dn"], s["x"], s["y"], **w, stream=side)
    got_plain = drop.forward(s["x"], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(plain, got_plain)
    assert all(torch.equal(grads[k], got_grads[k]) for k in grads)
