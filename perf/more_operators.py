"""Cases of the operators of a block around the mixture-of-experts layer: the join of a block with its residual
stream (norms, gate, scale and dropout in one pass), dropout by itself, and the dense gated feed-forward block.

``listed()`` and ``draw(rng)`` give cases (dicts of plain values), ``prepare(case, seed)`` the inputs on the GPU,
``run(state)`` one pass, ``work(case)`` the bytes and operations that a pass cannot do without and
``exact(case, seed)`` its results in 64 bits.  With ``own`` false ``run`` computes each operator in elementary torch
operations in 32 bits; with ``own`` true it makes the calls of ``mixture_experts_layer_side_gb300``.

The operators:

  residual  z = y / sqrt(mean y^2 + eps) * w_out (or y itself), d = dropout(z), x' = x + scale * gate * d,
            n = x' / sqrt(mean x'^2 + eps) * w_next; a gate row serves T / G consecutive rows.  Forward, or the
            gradients of x, y, w_out, gate and w_next from those of x' and n
  dropout   out_i = x_i / (1 - p) where kept, else 0: kept where the element's 16 bits of Philox-4x32-10 (key: the
            seed; counter: the block of eight elements and the number of the call) are not below p * 65536, with
            p a multiple of 1 / 65536.  Its gradient is the same call on the output's gradient
  ffn       out = (silu(x W1) * (x W3)) W2; forward alone, or a step that gives the gradients too
"""

import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------- cases
def listed():
    res, drp, ffn = dict(op="residual"), dict(op="dropout"), dict(op="ffn")
    return [
        # one token of one request, 32-bit stream, norms on both sides of the block: latency counts
        dict(res, name="residual: forward, 1 token, f32 stream", mode="forward", T=1, H=2048, pad=0, stream="f32",
             branch="bf16", post=True, groups=0, next=True, p=0.0, scale=1.0),
        # the training forward of the widest layer: a gate a channel, both norms
        dict(res, name="residual: forward, 8192 rows", mode="forward", T=8192, H=7168, pad=0, stream="bf16",
             branch="bf16", post=True, groups=1, next=True, p=0.0, scale=0.5),
        # its backward pass
        dict(res, name="residual: backward, 8192 rows", mode="backward", T=8192, H=7168, pad=0, stream="bf16",
             branch="bf16", post=True, groups=1, next=True, p=0.0, scale=0.5),
        # an odd width (rows not aligned), a gate a sequence, dropout, everything in 32 bits
        dict(res, name="residual: forward, odd width, gate a sequence, dropout", mode="forward", T=1000, H=1003, pad=5,
             stream="f32", branch="f32", post=True, groups=8, next=True, p=0.125, scale=1.0),
        # a regularised training step of a mid-sized layer with 32-bit stream, conditioned by a gate a sequence
        dict(res, name="residual: backward, 4096 rows, gate a sequence, dropout", mode="backward", T=4096, H=2048,
             pad=0, stream="f32", branch="bf16", post=True, groups=16, next=True, p=0.125, scale=1.0),
        # a few rows by themselves
        dict(drp, name="dropout: 5 rows of 328, f32", T=5, H=328, pad=0, dtype="f32", p=0.125),
        # activations of a long training batch
        dict(drp, name="dropout: 16384 rows of 7168, bf16", T=16384, H=7168, pad=0, dtype="bf16", p=0.125),
        # the shared expert for one token of a serving step
        dict(ffn, name="ffn: forward, 1 token", mode="infer", T=1, H=7168, I=2048),
        # and for a batch of requests on a mid-sized layer
        dict(ffn, name="ffn: forward, 100 tokens, mid", mode="infer", T=100, H=2048, I=768),
        # a prefill
        dict(ffn, name="ffn: forward, 8192 tokens", mode="infer", T=8192, H=7168, I=2048),
        # a training step, no size a multiple of a tile
        dict(ffn, name="ffn: step, ragged", mode="step", T=1000, H=1144, I=680),
        # a training step of the widest layer
        dict(ffn, name="ffn: step, 8192 tokens", mode="step", T=8192, H=7168, I=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {op: max(work(c)[unit] for c in listed() if c["op"] == op)
            for op, unit in (("residual", "bytes"), ("dropout", "bytes"), ("ffn", "flops"))}
    while True:
        op = rng.choice(["residual", "residual", "dropout", "ffn", "ffn"])
        if op == "residual":
            T = _log(rng, 1, 16384)
            groups = rng.choice([0, 1, 1, rng.randint(2, 16), T])
            if groups > 1:
                T = max(1, T // groups) * groups
            stream, branch = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
            c = dict(op=op, mode=rng.choice(["forward", "backward"]), T=T,
                     H=rng.choice([1, 8, 8, 8]) * _log(rng, 8, 1024), pad=rng.choice([0, 0, 8, 3]), stream=stream,
                     branch=branch, post=rng.random() < 0.7, groups=groups, next=rng.random() < 0.8,
                     p=rng.choice([0.0, 0.0, 0.125, 0.5]), scale=rng.choice([1.0, 0.5, 0.22]))
        elif op == "dropout":
            c = dict(op=op, T=_log(rng, 1, 16384), H=_log(rng, 1, 8192), pad=rng.choice([0, 0, 0, 8, 3]),
                     dtype=rng.choice(["bf16", "bf16", "f32"]), p=rng.choice([0.0625, 0.125, 0.25, 0.5]))
        else:
            c = dict(op=op, mode=rng.choice(["infer", "step"]), T=_log(rng, 1, 8192), H=8 * _log(rng, 8, 896),
                     I=8 * _log(rng, 8, 512))
        w = work(c)
        if w["bytes" if op != "ffn" else "flops"] <= most[op]:
            return c


def work(case):
    c = case
    if c["op"] == "residual":
        n = c["T"] * c["H"]
        S, B = (2 if c[t] == "bf16" else 4 for t in ("stream", "branch"))
        backward = c["mode"] == "backward"
        # forward: x, y in, x' and n out; backward: the gradients of x' and n, x' and y in, those of x and y out
        # (without the second norm n, its gradient and x' are not there; without the first and a gate y is not read)
        if backward:
            b = n * (2 * S + B + (S + B if c["next"] else 0) + (B if c["post"] or c["groups"] else 0))
        else:
            b = n * (2 * S + B + (B if c["next"] else 0))
        b += c["groups"] * c["H"] * B * (2 if backward else 1)
        return {"bytes": float(b), "flops": n * (25.0 if backward else 12.0)}
    if c["op"] == "dropout":
        n = c["T"] * c["H"]
        return {"bytes": n * 2.0 * (2 if c["dtype"] == "bf16" else 4), "flops": 10.0 * n}
    T, H, I = c["T"], c["H"], c["I"]
    weights = 3.0 * H * I * 2
    if c["mode"] == "infer":
        return {"bytes": weights + T * H * 4.0, "flops": 6.0 * T * H * I}
    return {"bytes": 2 * weights + T * H * 8.0, "flops": 18.0 * T * H * I}


# ---------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32)


def _rows(g, T, H, pad, dtype, std):
    """[T, H] whose rows are H + pad elements apart."""
    full = torch.empty((T, H + pad), device=DEVICE, dtype=dtype)
    for t in range(0, T, 4096):
        n = min(4096, T - t)
        full[t:t + n] = _randn(g, n, H + pad) * std
    return full[:, :H]


def _prepare_residual(c, g):
    T, H, pad = c["T"], c["H"], c["pad"]
    S, B = TYPES[c["stream"]], TYPES[c["branch"]]
    s = {}
    # a stream that grew over the blocks before, a few channels far above the others
    channel = 1.0 + 15.0 * (torch.rand((H,), generator=g, device=DEVICE) < 0.01)
    s["x"] = _rows(g, T, H, pad, S, 2.0)  # x, or x' in the backward pass
    s["x"] *= channel.to(S)
    s["y"] = _rows(g, T, H, pad, B, 0.7)
    s["w_out"] = (1.0 + 0.2 * _randn(g, H)).to(B) if c["post"] else None
    s["w_next"] = (1.0 + 0.2 * _randn(g, H)).to(B) if c["next"] else None
    s["gate"] = (0.5 * _randn(g, c["groups"], H)).to(B) if c["groups"] else None
    if c["mode"] == "backward":
        s["dx"] = _rows(g, T, H, 0, S, 1.0)
        s["dn"] = _rows(g, T, H, 0, B, 1.0) if c["next"] else None
    s["seed"], s["call"] = int(torch.randint(0, 2**62, (1,), generator=g, device=DEVICE)), 7
    if own:
        from mixture_experts_layer_side_gb300.dropout import MoKDropout
        from mixture_experts_layer_side_gb300.residual import MoKResidual
        s["handle"] = MoKResidual(H, T, eps=EPS, device=DEVICE)
        s["dropout"] = MoKDropout(c["p"], seed=s["seed"], device=DEVICE) if c["p"] else None
    return s


def _prepare_dropout(c, g):
    s = dict(x=_rows(g, c["T"], c["H"], c["pad"], TYPES[c["dtype"]], 1.0))
    s["seed"], s["call"] = int(torch.randint(0, 2**62, (1,), generator=g, device=DEVICE)), 3
    if own:
        from mixture_experts_layer_side_gb300.dropout import MoKDropout
        s["handle"] = MoKDropout(c["p"], seed=s["seed"], device=DEVICE)
    return s


def _prepare_ffn(c, g):
    T, H, I = c["T"], c["H"], c["I"]
    s = dict(x=_randn(g, T, H).bfloat16())
    for name, (r, k) in (("W1", (H, I)), ("W3", (H, I)), ("W2", (I, H))):
        s[name] = (0.02 * _randn(g, r, k)).bfloat16()
    if c["mode"] == "step":
        s["dout"] = _randn(g, T, H).bfloat16()
    if own:
        from mixture_experts_layer_side_gb300.feedforward import MoKFeedForward
        s["handle"] = MoKFeedForward(H, I, T, training=c["mode"] == "step", device=DEVICE)
    return s


def prepare(case, seed):
    make = {"residual": _prepare_residual, "dropout": _prepare_dropout, "ffn": _prepare_ffn}[case["op"]]
    return dict(make(case, _gen(seed)), case=dict(case))


# ---------------------------------------------------------------------------------------------------- one pass
_M0, _M1, _W0, _W1, _LOW = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85, 0xFFFFFFFF


def _mul32(a, m):
    """Both 32-bit halves of a * m (64-bit products that wrap around)."""
    w = a * m
    return (w >> 32) & _LOW, w & _LOW


def _kept(T, H, p, seed, call):
    """Truth values [T, H]: which elements dropout keeps."""
    blocks = (T * H + 7) // 8
    i = torch.arange(blocks, device=DEVICE, dtype=torch.int64)
    c0, c1 = i & _LOW, i >> 32
    c2, c3 = torch.full_like(i, call & _LOW), torch.full_like(i, call >> 32)
    k0, k1 = seed & _LOW, seed >> 32
    for _ in range(10):
        h0, l0 = _mul32(c0, _M0)
        h1, l1 = _mul32(c2, _M1)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + _W0) & _LOW, (k1 + _W1) & _LOW
    at = round(p * 65536)
    parts = [half for c in (c0, c1, c2, c3) for half in ((c & 0xFFFF) >= at, (c >> 16) >= at)]
    return torch.stack(parts, 1).reshape(-1)[:T * H].reshape(T, H)


def _plain_drop(v, s):
    c = s["case"]
    if not c["p"]:
        return v
    return torch.where(_kept(*v.shape, c["p"], s["seed"], s["call"]), v * (1.0 / (1.0 - c["p"])), 0.0)


def _rstd(v):
    return 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def _gate_rows(s, T):
    return None if s["gate"] is None else s["gate"].float().repeat_interleave(T // s["gate"].shape[0], 0)


def _plain_residual(s):
    c = s["case"]
    S, B, scale = TYPES[c["stream"]], TYPES[c["branch"]], c["scale"]
    x, y, gate = s["x"].float(), s["y"].float(), _gate_rows(s, c["T"])
    if c["post"]:
        w_out = s["w_out"].float()
        y_hat = y * _rstd(y)
        z = y_hat * w_out
    else:
        z = y
    if c["mode"] == "forward":
        d = _plain_drop(z, s) * scale
        x = x + (d if gate is None else d * gate)
        return x.to(S), ((x * _rstd(x)) * s["w_next"].float()).to(B) if c["next"] else None
    g = s["dx"].float()
    dw_out = dgate = dw_next = None
    if c["next"]:
        r, dn = _rstd(x), s["dn"].float()
        x_hat = x * r
        t = dn * s["w_next"].float()
        g = g + r * (t - x_hat * (t * x_hat).mean(1, keepdim=True))
        dw_next = (dn * x_hat).sum(0)
    db = g * scale
    if gate is not None:
        dgate = (db * _plain_drop(z, s)).reshape(c["groups"], -1, c["H"]).sum(1).to(B)
        db = db * gate
    dz = _plain_drop(db, s)
    if c["post"]:
        t = dz * w_out
        dw_out = (dz * y_hat).sum(0)
        dz = _rstd(y) * (t - y_hat * (t * y_hat).mean(1, keepdim=True))
    return g.to(S), dz.to(B), dw_out, dgate, dw_next


def _plain_ffn(s):
    x, W1, W3, W2 = (s[n].float() for n in ("x", "W1", "W3", "W2"))
    h, u = x @ W1, x @ W3
    sig = 1.0 / (1.0 + torch.exp(-h))
    a = h * sig * u
    out = (a @ W2).bfloat16()
    if s["case"]["mode"] == "infer":
        return out
    dout = s["dout"].float()
    da = dout @ W2.t()
    dW2 = a.t() @ dout
    dh, du = da * u * sig * (1.0 + h * (1.0 - sig)), da * h * sig
    grads = (dh @ W1.t() + du @ W3.t(), x.t() @ dh, x.t() @ du, dW2)
    return (out, *(v.bfloat16() for v in grads))


def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "dropout":
            return _plain_drop(s["x"].float(), s).to(s["x"].dtype)
        return _plain_residual(s) if c["op"] == "residual" else _plain_ffn(s)
    if c["op"] == "dropout":
        return s["handle"].forward(s["x"], call=s["call"])
    if c["op"] == "residual":
        weights = dict(w_out=s["w_out"], gate=s["gate"], w_next=s["w_next"], scale=c["scale"], dropout=s["dropout"],
                       call=s["call"])
        if c["mode"] == "forward":
            return s["handle"].forward(s["x"], s["y"], **weights)
        got = s["handle"].backward(s["dx"], s["dn"], s["x"], s["y"], **weights)
        return got["dx"], got["dy"], got["dw_out"], got["dgate"], got["dw_next"]
    w = s["W1"], s["W3"], s["W2"]
    if c["mode"] == "infer":
        return s["handle"].infer(s["x"], *w)
    out = s["handle"].forward(s["x"], *w)
    got = s["handle"].backward(s["x"], *w, s["dout"])
    return out, got["dX"], got["dW1"], got["dW3"], got["dW2"]


# ---------------------------------------------------------------------------------------------------- 64 bits
def _exact_kept(T, H, p, seed, call):
    """Which elements are kept, with products made of 16-bit digits."""
    def product(a, m):
        a0, a1, m0, m1 = a % 65536, a // 65536, m % 65536, m // 65536
        mid = a0 * m1 + a1 * m0 + a0 * m0 // 65536
        return a1 * m1 + mid // 65536, mid % 65536 * 65536 + a0 * m0 % 65536

    full = 2**32
    index = torch.arange((T * H + 7) // 8, device=DEVICE)
    ctr = [index % full, index // full, torch.zeros_like(index) + call % full, torch.zeros_like(index) + call // full]
    key = [seed % full, seed // full]
    for rnd in range(10):
        hi0, lo0 = product(ctr[0], 0xD2511F53)
        hi1, lo1 = product(ctr[2], 0xCD9E8D57)
        key_now = [(key[0] + rnd * 0x9E3779B9) % full, (key[1] + rnd * 0xBB67AE85) % full]
        ctr = [torch.bitwise_xor(torch.bitwise_xor(hi1, ctr[1]), key_now[0]), lo1,
               torch.bitwise_xor(torch.bitwise_xor(hi0, ctr[3]), key_now[1]), lo0]
    bits = torch.empty((index.numel(), 8), device=DEVICE, dtype=torch.int64)
    for w in range(4):
        bits[:, 2 * w], bits[:, 2 * w + 1] = ctr[w] % 65536, ctr[w] // 65536
    return bits.reshape(-1)[:T * H].reshape(T, H) >= p * 65536


def _exact_residual(c, s):
    x, y = s["x"].double(), s["y"].double()
    n = c["H"]
    factor = torch.full_like(y, c["scale"])
    if c["groups"]:
        each = c["T"] // c["groups"]
        gate = s["gate"].double()[torch.arange(c["T"], device=DEVICE) // each]
        factor *= gate
    drop = torch.ones_like(y)
    if c["p"]:
        drop = _exact_kept(c["T"], n, c["p"], s["seed"], s["call"]).double() / (1.0 - c["p"])
    size_y = torch.sqrt(y.square().sum(1, keepdim=True) / n + EPS)
    z = y / size_y * s["w_out"].double() if c["post"] else y
    if c["mode"] == "forward":
        x = x + factor * drop * z
        out = x / torch.sqrt(x.square().sum(1, keepdim=True) / n + EPS) * s["w_next"].double() if c["next"] else None
        return x, out
    dx = s["dx"].double()
    dw_out = dgate = dw_next = None
    if c["next"]:
        size = torch.sqrt(x.square().sum(1, keepdim=True) / n + EPS)
        dn = s["dn"].double()
        v = dn * s["w_next"].double()
        dx = dx + v / size - x * (v * x).sum(1, keepdim=True) / (n * size**3)
        dw_next = (dn * x / size).sum(0)
    if c["groups"]:
        dgate = (dx * c["scale"] * drop * z).reshape(c["groups"], each, n).sum(1)
    dz = dx * factor * drop
    if c["post"]:
        v = dz * s["w_out"].double()
        dw_out = (dz * y / size_y).sum(0)
        dz = v / size_y - y * (v * y).sum(1, keepdim=True) / (n * size_y**3)
    return dx, dz, dw_out, dgate, dw_next


def _exact_ffn(c, s):
    x, W1, W3, W2 = (s[n].double() for n in ("x", "W1", "W3", "W2"))
    h, u = x @ W1, x @ W3
    gated = torch.sigmoid(h)
    silu = h * gated
    out = (silu * u) @ W2
    if c["mode"] == "infer":
        return out
    dout = s["dout"].double()
    da = dout @ W2.t()
    dh, du = da * u * (gated + silu * (1.0 - gated)), da * silu
    return out, dh @ W1.t() + du @ W3.t(), x.t() @ dh, x.t() @ du, (silu * u).t() @ dout


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "dropout":
        x = s["x"].double()
        return torch.where(_exact_kept(c["T"], c["H"], c["p"], s["seed"], s["call"]), x / (1.0 - c["p"]), 0.0)
    return _exact_residual(c, s) if c["op"] == "residual" else _exact_ffn(c, s)
