"""Cases of the operators around the mixture-of-experts layer: the layer for a few tokens, the distillation loss
from a teacher's top logits, and the token embedding with its gradient.

``listed()`` and ``draw(rng)`` give cases (dicts of plain values), ``prepare(case, seed)`` the inputs on the GPU,
``run(state)`` one pass, ``work(case)`` the bytes and operations that a pass cannot do without and
``exact(case, seed)`` its results in 64 bits.  With ``own`` false ``run`` computes each operator in elementary torch
operations in 32 bits; with ``own`` true it makes the calls of ``mixture_experts_layer_side_gb300``.

The operators:

  few      out_t = sum_j s_tj ((silu(x_t W1_e) * (x_t W3_e)) W2_e), e = idx_tj, for T <= 128 tokens; with ``router``
           the selection and the scores come from the layer's top-k softmax router in the same call
  distill  loss_t = KL(p_t || softmax(z_t / tau)), p_t the softmax of the teacher's listed logits / tau over the list;
           forward (loss and log-sum-exp), backward (gradient of z) or both in one call ("step")
  embed    x_n = scale * table[id_n], and its gradient, each table row's tokens summed in ascending order
"""

import math

import numpy as np
import torch

own = False

DEVICE = "cuda"


# ---------------------------------------------------------------------------------------------------- cases
def listed():
    few, dis, emb = dict(op="few"), dict(op="distill"), dict(op="embed")
    wide = dict(H=7168, I=2048, k=8)
    mid = dict(H=2048, I=768, E=64, k=8)
    return [
        # one token of one request on a mid-sized layer: latency counts
        dict(few, name="few: 1 token, mid", T=1, **mid, prec="bf16", router=False, routing="uniform"),
        # one token on the widest layer: its eight experts' weights, router included
        dict(few, name="few: 1 token, wide, router", T=1, E=256, **wide, prec="bf16", router=True, routing="zipf"),
        # a small batch of requests: most of the read is experts with one or two rows
        dict(few, name="few: 24 tokens, wide", T=24, E=256, **wide, prec="bf16", router=False, routing="zipf"),
        # the most tokens the operator takes, skewed: every expert, some with dozens of rows
        dict(few, name="few: 128 tokens, mid, mxfp8, router", T=128, **mid, prec="mxfp8", router=True, routing="zipf"),
        # eight requests on the widest layer in 8 bits
        dict(few, name="few: 8 tokens, wide, mxfp8", T=8, E=384, **wide, prec="mxfp8", router=False, routing="uniform"),
        # the last, small micro-batch of a run with 32-bit logits
        dict(dis, name="distill: step, 48 rows, f32", mode="step", T=48, V=32000, K=8, pad=0, dtype="f32", tau=1.0,
             masked=0.0),
        # an odd vocabulary (rows not aligned), ragged teacher lists, an evaluation pass
        dict(dis, name="distill: forward, odd vocabulary", mode="forward", T=1000, V=50001, K=20, pad=0, dtype="bf16",
             tau=2.0, masked=0.2),
        # the training step's loss on a long batch
        dict(dis, name="distill: step, 4096 rows", mode="step", T=4096, V=131072, K=64, pad=64, dtype="bf16", tau=1.0,
             masked=0.05),
        # a few tokens of a serving step, odd sizes
        dict(emb, name="embed: lookup, 5 tokens", mode="lookup", N=5, V=1003, H=328, dtype="f32", skew=0.0),
        # the lookup of a training batch
        dict(emb, name="embed: lookup, 16384 tokens", mode="lookup", N=16384, V=131072, H=7168, dtype="bf16", skew=1.0),
        # the whole gradient, zero rows included
        dict(emb, name="embed: gradient, dense", mode="dense", N=8192, V=65536, H=2048, dtype="bf16", skew=1.0),
        # a later micro-batch added to the 32-bit gradient: only the rows of its tokens
        dict(emb, name="embed: gradient, accumulated", mode="accumulate", N=16384, V=32768, H=7168, dtype="bf16",
             skew=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["few", "few", "distill", "embed"])
        if op == "few":
            E = _log(rng, 4, 384)
            c = dict(op=op, T=_log(rng, 1, 128), H=128 * _log(rng, 1, 56), I=128 * _log(rng, 1, 16), E=E,
                     k=rng.randint(1, min(E, 10)), prec=rng.choice(["bf16", "mxfp8"]), router=rng.random() < 0.5,
                     routing=rng.choice(["uniform", "zipf"]))
            held = 3 * E * c["H"] * c["I"] * (2 if c["prec"] == "bf16" else 1)
        elif op == "distill":
            c = dict(op=op, mode=rng.choice(["forward", "backward", "step"]), T=_log(rng, 1, 4096), V=_log(rng, 300, 131072),
                     K=_log(rng, 1, 100), pad=rng.choice([0, 0, 1, 64]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                     tau=rng.choice([0.5, 1.0, 2.0, 4.0]), masked=rng.choice([0.0, 0.1, 0.5]))
            held = 4 * c["T"] * c["V"]
        else:
            c = dict(op=op, mode=rng.choice(["lookup", "dense", "accumulate"]), N=_log(rng, 1, 32768), V=_log(rng, 300, 131072),
                     H=rng.choice([1, 8, 8, 128]) * _log(rng, 1, 56), dtype=rng.choice(["bf16", "bf16", "f32"]),
                     skew=rng.choice([0.0, 1.0, 1.0]))
            held = 4 * c["V"] * c["H"]
        if work(c)["bytes"] <= most and held <= 12e9:
            return c


def _distinct(c):
    """Expected number of distinct experts of a case's routing, from a fixed sample of routings."""
    g = np.random.RandomState(0)
    got = []
    for _ in range(4):
        key = g.randn(c["T"], c["E"]) * (1.7 if c["router"] else 1.0)
        if c["routing"] == "zipf":
            p = np.arange(1, c["E"] + 1) ** -1.2
            key = key + np.log(p / p.sum())
        top = np.argpartition(-key, c["k"] - 1, axis=1)[:, :c["k"]]
        got.append(len(np.unique(top)))
    return sum(got) / len(got)


def work(case):
    c = case
    if c["op"] == "few":
        T, H, I, E, k = (c[n] for n in ("T", "H", "I", "E", "k"))
        weights = _distinct(c) * 3 * H * I * (2 if c["prec"] == "bf16" else 33 / 32)
        b = weights + T * H * 4 + (H * E * 2 + T * k * 8 if c["router"] else T * k * 8)
        f = T * k * 6.0 * H * I + (2.0 * T * H * E if c["router"] else 0)
    elif c["op"] == "distill":
        z = c["T"] * c["V"] * (2 if c["dtype"] == "bf16" else 4)
        b = z * (1 if c["mode"] == "forward" else 2) + c["T"] * (c["K"] * 8 + 8)
        f = c["T"] * c["V"] * (4.0 if c["mode"] == "forward" else 8.0)
    else:
        n, e = c["N"] * c["H"], 2 if c["dtype"] == "bf16" else 4
        if c["mode"] == "lookup":
            b, f = 2 * n * e, n
        else:
            # dense: the whole gradient in the type of the table; accumulate: the touched rows of a 32-bit one, both ways
            rows = c["V"] * e if c["mode"] == "dense" else _touched(c) * 8
            b, f = n * e + rows * c["H"], 2.0 * n
        b += c["N"] * 4
    return {"bytes": float(b), "flops": float(f)}


def _id_probs(c):
    p = 1.0 / (np.arange(c["V"]) + 2.7) ** c["skew"]
    return p / p.sum()


def _touched(c):
    return float((1.0 - np.exp(c["N"] * np.log1p(-np.minimum(_id_probs(c), 1 - 1e-12)))).sum())


# ---------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32)


def _pow2(e):
    """2^e of whole numbers in [-126, 127], exactly."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _mx_quantize(v, dim):
    """E4M3 codes (u8, the shape of v) and E8M0 scales of 32-element blocks along ``dim``: exponent
    floor(log2 amax) - 8, codes rounded to nearest even, saturating."""
    shape = list(v.shape)
    b = v.reshape(shape[:dim] + [shape[dim] // 32, 32] + shape[dim + 1:])
    amax = b.abs().amax(dim + 1, keepdim=True)
    exp = (torch.frexp(amax)[1] - 9).clamp(-126, 126)  # the values here are far from either end
    exp = torch.where(amax > 0, exp, torch.full_like(exp, -126))
    q = (b * _pow2(-exp)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.reshape(shape).view(torch.uint8), (exp + 127).squeeze(dim + 1).to(torch.uint8)


def _mx_values(q, sf, dim):
    """The 32-bit values of codes and scales."""
    v = q.view(torch.float8_e4m3fn).float()
    return v * _pow2(sf.int() - 127).repeat_interleave(32, dim)


def _weights(g, c, rows, cols):
    """[E, rows, cols] weights of standard deviation 0.02: a bf16 tensor, or (codes, scales) along the rows."""
    E = c["E"]
    if c["prec"] == "bf16":
        W = torch.empty((E, rows, cols), device=DEVICE, dtype=torch.bfloat16)
        for e in range(0, E, 8):
            n = min(8, E - e)
            W[e:e + n] = _randn(g, n, rows, cols) * 0.02
        return W
    q = torch.empty((E, rows, cols), device=DEVICE, dtype=torch.uint8)
    sf = torch.empty((E, rows // 32, cols), device=DEVICE, dtype=torch.uint8)
    for e in range(0, E, 8):
        n = min(8, E - e)
        q[e:e + n], sf[e:e + n] = _mx_quantize((_randn(g, n, rows, cols) * 0.02).bfloat16().float(), 1)
    return q, sf


def _prepare_few(c, g):
    T, H, I, E, k = (c[n] for n in ("T", "H", "I", "E", "k"))
    s = {}
    bias = None
    if c["routing"] == "zipf":
        p = torch.arange(1, E + 1, device=DEVICE, dtype=torch.float64).pow(-1.2)
        bias = torch.log(p / p.sum())[torch.randperm(E, generator=g, device=DEVICE)].float()
    if c["router"]:
        # activations and router weights on a grid coarse enough that a 32-bit sum of their products is exact in
        # any order: the selection then does not hang on the order of the sum
        s["x"] = ((_randn(g, T, H) * 32).round().clamp(-127, 127) / 32).bfloat16()
        s["Wr"] = ((_randn(g, H, E) * 0.02 * 2048).round().clamp(-127, 127) / 2048).bfloat16()
        s["bias"] = bias
    else:
        s["x"] = _randn(g, T, H).bfloat16()
        logits = _randn(g, T, E)
        key = logits if bias is None else logits + bias
        idx = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :k]
        s["scores"] = torch.softmax(torch.gather(logits, 1, idx), dim=1).contiguous()
        s["idx"] = idx.int().contiguous()
    s["W1"], s["W3"], s["W2"] = _weights(g, c, H, I), _weights(g, c, H, I), _weights(g, c, I, H)
    if own:
        from mixture_experts_layer_side_gb300 import _lib
        from mixture_experts_layer_side_gb300.decode import MoKDecoder
        from mixture_experts_layer_side_gb300.inputs import Shape
        s["layer"] = MoKDecoder(Shape(T, H, I, E, k), precision=c["prec"], device=DEVICE)
        s["W"] = tuple(s[n] if c["prec"] == "bf16" else _lib.mx(*s[n]) for n in ("W1", "W3", "W2"))
    return s


def _prepare_distill(c, g):
    T, V, K = c["T"], c["V"], c["K"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    full = torch.empty((T, V + c["pad"]), device=DEVICE, dtype=dt)  # rows of a padded vocabulary
    for t in range(0, T, 512):
        n = min(512, T - t)
        full[t:t + n] = _randn(g, n, V + c["pad"]) * 2.5
    s = dict(z=full[:, :V], tau=c["tau"])
    if V > 1000:
        s["z"][:, V - 7:V - 2] = -math.inf  # tokens that the student never gives
    # distinct ids a row, none of those: one of each of K equal ranges
    width = max(1, (V - 8 if V > 1000 else V) // K)
    ids = torch.arange(K, device=DEVICE) * width + (torch.rand((T, K), generator=g, device=DEVICE) * width).long().clamp(max=width - 1)
    vals = 6.0 + 2.0 * _randn(g, T, K)
    off = torch.rand((T, K), generator=g, device=DEVICE) < c["masked"]  # lists of fewer entries, some of none
    off |= torch.rand((T, 1), generator=g, device=DEVICE) < 0.1 * (c["masked"] > 0)
    s["ids"] = torch.where(off, -1, ids).int().contiguous()
    s["vals"] = vals.sort(dim=1, descending=True)[0].contiguous()
    s["dloss"] = torch.rand((T,), generator=g, device=DEVICE) / T  # weights of the rows in the mean
    if c["mode"] == "backward":
        s["lse"] = torch.cat([torch.logsumexp(p.double() / c["tau"], 1) for p in s["z"].split(512)]).float()
    if own:
        from mixture_experts_layer_side_gb300.distill import DistillLoss
        s["handle"] = DistillLoss(T, V, K, device=DEVICE)
    return s


def _prepare_embed(c, g):
    N, V, H = c["N"], c["V"], c["H"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    s = dict(scale=math.sqrt(H) if c["mode"] == "lookup" else 0.5, pad=V - 1)
    cdf = torch.from_numpy(np.cumsum(_id_probs(c))).to(DEVICE)
    u = torch.rand((N,), generator=g, device=DEVICE, dtype=torch.float64)
    ids = torch.searchsorted(cdf, u).clamp(max=V - 1)
    ids[N - N // 16:] = V - 1  # the end of the batch is padding
    s["ids"] = ids.int()
    if c["mode"] == "lookup":
        s["table"] = torch.empty((V, H), device=DEVICE, dtype=dt)
        for v in range(0, V, 16384):
            n = min(16384, V - v)
            s["table"][v:v + n] = _randn(g, n, H) * 0.02
    else:
        s["dx"] = _randn(g, N, H).to(dt)
        if c["mode"] == "accumulate":
            s["dtable"] = torch.zeros((V, H), device=DEVICE)
    if own:
        from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
        s["handle"] = MoKEmbedding(V, H, N, pad_id=s["pad"], device=DEVICE)
        if c["mode"] == "dense":
            s["out"] = torch.empty((V, H), device=DEVICE, dtype=dt)
    return s


def prepare(case, seed):
    g = _gen(seed)
    s = {"few": _prepare_few, "distill": _prepare_distill, "embed": _prepare_embed}[case["op"]](case, g)
    return dict(s, case=dict(case))


# ---------------------------------------------------------------------------------------------------- one pass
def _plain_few(s):
    c = s["case"]
    T, k, mx = c["T"], c["k"], c["prec"] == "mxfp8"
    x = s["x"].float()
    if c["router"]:
        logits = x @ s["Wr"].float()
        key = logits if s["bias"] is None else logits + s["bias"]
        idx = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :k]
        chosen = torch.gather(logits, 1, idx)
        e = torch.exp(chosen - chosen.amax(1, keepdim=True))
        scores = e / e.sum(1, keepdim=True)
    else:
        idx, scores = s["idx"].long(), s["scores"]
    # the rows of each expert that was chosen, side by side
    experts, row_of = torch.unique(idx.reshape(-1), return_inverse=True)
    member = row_of[:, None] == torch.arange(experts.numel(), device=x.device)
    place = torch.gather(member.long().cumsum(0), 1, row_of[:, None])[:, 0] - 1
    widest = int(place.max()) + 1
    token = torch.arange(T * k, device=x.device) // k

    def weights(name):
        if mx:
            return _mx_values(s[name][0][experts], s[name][1][experts], 1)
        return s[name][experts].float()

    if mx:
        x = _mx_values(*_mx_quantize(x, 1), 1)
    rows = x.new_zeros((experts.numel(), widest, c["H"]))
    rows[row_of, place] = x[token]
    h, u = torch.bmm(rows, weights("W1")), torch.bmm(rows, weights("W3"))
    a = h / (1.0 + torch.exp(-h)) * u
    if mx:
        a = _mx_values(*_mx_quantize(a, 2), 2)
    y = torch.bmm(a, weights("W2"))[row_of, place].reshape(T, k, c["H"])
    out = (scores[:, :, None] * y).sum(1).bfloat16()
    return (out, idx.int(), scores) if c["router"] else out


def _teacher(ids, vals, tau):
    """Probabilities of the listed tokens (zero where the id is -1) and their logarithms."""
    v = torch.where(ids >= 0, vals / tau, -math.inf)
    top = v.amax(1, keepdim=True)
    e = torch.exp(v - torch.where(torch.isfinite(top), top, 0.0))
    total = e.sum(1, keepdim=True)
    p = torch.where(total > 0, e / total, 0.0)
    return p, torch.where(p > 0, torch.log(p), 0.0)


def _plain_distill(s):
    mode, tau = s["case"]["mode"], s["tau"]
    z = s["z"].float() / tau
    p, log_p = _teacher(s["ids"], s["vals"], tau)
    at = s["ids"].long().clamp(min=0)
    if mode == "backward":
        lse = s["lse"]
    else:
        top = z.amax(1)
        lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    loss = (p * torch.where(p > 0, log_p - (torch.gather(z, 1, at) - lse[:, None]), 0.0)).sum(1)
    if mode == "forward":
        return loss, lse
    g = torch.exp(z - lse[:, None]) * p.sum(1, keepdim=True)
    g.scatter_add_(1, at, -p)
    dz = (g * (s["dloss"] / tau)[:, None]).to(s["z"].dtype)
    return dz if mode == "backward" else (loss, dz)


def _plain_embed(s):
    mode = s["case"]["mode"]
    if mode == "lookup":
        return (s["table"][s["ids"].long()].float() * s["scale"]).to(s["table"].dtype)
    rows = s["dx"].float() * (s["scale"] * (s["ids"] != s["pad"]))[:, None]
    if mode == "accumulate":
        return s["dtable"].index_add_(0, s["ids"].long(), rows)
    full = rows.new_zeros((s["case"]["V"], s["case"]["H"]))
    return full.index_add_(0, s["ids"].long(), rows).to(s["dx"].dtype)


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"few": _plain_few, "distill": _plain_distill, "embed": _plain_embed}[c["op"]](s)
    if c["op"] == "few":
        if c["router"]:
            return s["layer"].layer(s["x"], s["Wr"], *s["W"], bias=s["bias"])
        return s["layer"].forward(s["x"], s["idx"], s["scores"], *s["W"])
    if c["op"] == "distill":
        if c["mode"] == "forward":
            return s["handle"].forward(s["z"], s["ids"], s["vals"], temperature=s["tau"])
        if c["mode"] == "backward":
            return s["handle"].backward(s["z"], s["ids"], s["vals"], s["lse"], s["dloss"], temperature=s["tau"])
        return s["handle"].forward_backward(s["z"], s["ids"], s["vals"], s["dloss"], temperature=s["tau"])
    if c["mode"] == "lookup":
        return s["handle"].forward(s["table"], s["ids"], scale=s["scale"])
    if c["mode"] == "dense":
        return s["handle"].backward(s["dx"], s["ids"], scale=s["scale"], out=s["out"])
    return s["handle"].backward(s["dx"], s["ids"], scale=s["scale"], out=s["dtable"], accumulate=True)


# ---------------------------------------------------------------------------------------------------- 64 bits
def _exact_mx(v):
    """Values after block quantisation along the last dimension, in 64 bits: the E4M3 grid from its definition."""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    X = torch.where(amax > 0, (torch.frexp(amax)[1] - 9).clamp(-127, 127), -127).double()
    w = b / torch.exp2(X)
    step = torch.exp2((torch.frexp(w.abs())[1] - 1).clamp(min=-6).double() - 3)
    r = (w.abs() / step).round() * step
    return (torch.sign(w) * r.clamp(max=448.0) * torch.exp2(X)).reshape(v.shape)


def _exact_few(c, s):
    mx = c["prec"] == "mxfp8"
    x = s["x"].double()
    if c["router"]:
        logits = x @ s["Wr"].double()
        key = logits.float() if s["bias"] is None else logits.float() + s["bias"]
        idx = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :c["k"]]
        scores = torch.softmax(torch.gather(logits, 1, idx), 1)
    else:
        idx, scores = s["idx"].long(), s["scores"].double()
    if mx:
        x = _exact_mx(x)

    def matrix(name, e):
        if not mx:
            return s[name][e].double()
        q, sf = s[name][0][e].long(), s[name][1][e].double()
        ex, man = ((q >> 3) & 15).double(), (q & 7).double()
        v = torch.where(ex == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * torch.exp2(ex - 7))
        return torch.where(q >= 128, -v, v) * torch.exp2(sf - 127).repeat_interleave(32, 0)

    out = torch.zeros_like(x)
    for e in idx.unique().tolist():
        t, j = (idx == e).nonzero(as_tuple=True)
        h, u = x[t] @ matrix("W1", e), x[t] @ matrix("W3", e)
        a = h * torch.sigmoid(h) * u
        out.index_add_(0, t, scores[t, j][:, None] * ((_exact_mx(a) if mx else a) @ matrix("W2", e)))
    return (out, None, scores) if c["router"] else out


def _exact_distill(c, s):
    losses, sums, grads = [], [], []
    for at in torch.arange(c["T"], device=DEVICE).split(256):
        z = s["z"][at].double() / c["tau"]
        ids, v = s["ids"][at].long(), s["vals"][at].double() / c["tau"]
        has = (ids >= 0).any(1)
        log_p = torch.log_softmax(torch.where(ids >= 0, v, -math.inf), 1)
        p = torch.where(has[:, None] & (ids >= 0), torch.exp(log_p), 0.0)
        # the backward pass alone is given the forward's 32-bit log-sum-exp
        lse = s["lse"][at].double() if c["mode"] == "backward" else torch.logsumexp(z, 1)
        log_q = torch.gather(z, 1, ids.clamp(min=0)) - lse[:, None]
        losses.append(torch.where(p > 0, p * (log_p - log_q), 0.0).sum(1))
        sums.append(lse)
        if c["mode"] != "forward":
            g = torch.exp(z - lse[:, None]) * has[:, None]
            grads.append((g.scatter_add(1, ids.clamp(min=0), -p) * (s["dloss"][at].double() / c["tau"])[:, None]).float())
    if c["mode"] == "forward":
        return torch.cat(losses), torch.cat(sums)
    return torch.cat(grads) if c["mode"] == "backward" else (torch.cat(losses), torch.cat(grads))


def _exact_embed(c, s):
    ids = s["ids"].long()
    if c["mode"] == "lookup":
        return s["table"][ids].double() * s["scale"]
    keep = ids != s["pad"]
    full = torch.zeros((c["V"], c["H"]), device=DEVICE, dtype=torch.float64)
    return full.index_add_(0, ids[keep], s["dx"][keep].double() * s["scale"])


def exact(case, seed):
    s = prepare(case, seed)
    return {"few": _exact_few, "distill": _exact_distill, "embed": _exact_embed}[case["op"]](case, s)
