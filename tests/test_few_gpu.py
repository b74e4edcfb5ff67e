"""The layer for a few tokens through the C ABI against the float64 oracle:
every precision, routings that crowd, repeat, skip or break experts, the
router in the same call, reruns, graph replay and other streams."""

import numpy as np
import pytest
import torch

from _helpers import assert_bf16_close, assert_mxfp8_close, np64, require_gpu
from oracle import moe, router

pytestmark = pytest.mark.gpu


def make(T, H, I, E, k, kind, seed):
    from mixture_experts_layer_side_gb300.inputs import Shape, make_inputs
    inp = make_inputs(Shape(T, H, I, E, k), "zipf" if kind == "zipf" else "uniform", seed=seed)
    if kind == "one":       # every row on one expert
        inp["idx"][:] = E // 2
    elif kind == "repeat":  # a token lists an expert more than once
        inp["idx"][:, k // 2:] = inp["idx"][:, :k - k // 2]
    return inp


def decoder(T, H, I, E, k, prec):
    from mixture_experts_layer_side_gb300.decode import MoKDecoder
    from mixture_experts_layer_side_gb300.inputs import Shape
    return MoKDecoder(Shape(T, H, I, E, k), precision=prec)


def weights(inp, prec):
    from mixture_experts_layer_side_gb300.layer import quantize_weights
    W = [inp[n].cuda() for n in ("W1", "W3", "W2")]
    if prec == "bf16":
        return W, None
    q = quantize_weights(*W)
    return q["fwd"], q


def oracle_out(inp, prec, idx=None, s=None):
    a = {n: np64(v) for n, v in inp.items()}
    idx = inp["idx"].numpy() if idx is None else idx
    s = a["s"] if s is None else s
    return moe.forward(a["x"], idx, s, a["W1"], a["W3"], a["W2"], quant="mxfp8" if prec == "mxfp8" else None)[0]


def assert_close(got, ref, prec, name):
    (assert_bf16_close if prec == "bf16" else assert_mxfp8_close)(np64(got), ref, name)


# sizes: one column block, odd numbers of 128-blocks, k = 1, k = E, rows beyond
# every tile of tokens that a kernel may take at once
SHAPES = [(1, 128, 128, 4, 2), (1, 256, 128, 8, 2), (2, 384, 256, 5, 5), (7, 640, 384, 16, 3), (16, 256, 128, 8, 2),
          (17, 1024, 128, 3, 1), (33, 256, 640, 64, 8), (64, 512, 256, 12, 4), (128, 384, 384, 24, 6),
          (128, 256, 256, 300, 8)]


@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
@pytest.mark.parametrize("shape", SHAPES)
def test_few_matches_oracle(shape, prec):
    require_gpu()
    inp = make(*shape, "zipf", sum(shape))
    dec = decoder(*shape, prec)
    W, _keep = weights(inp, prec)
    out = torch.full((shape[0], shape[1]), float("nan"), dtype=torch.bfloat16, device="cuda")
    dec.forward(inp["x"].cuda(), inp["idx"].cuda(), inp["s"].cuda(), *W, out=out)
    dec.check()
    assert_close(out, oracle_out(inp, prec), prec, f"few {shape}")


@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
@pytest.mark.parametrize("kind", ["one", "repeat"])
@pytest.mark.parametrize("T", [1, 9, 100, 128])
def test_few_crowded_and_repeated_experts(T, kind, prec):
    """All rows on one expert (more rows than one tile holds: T * k of them),
    and tokens that list an expert twice."""
    require_gpu()
    shape = (T, 256, 256, 9, 4)
    inp = make(*shape, kind, T)
    dec = decoder(*shape, prec)
    W, _keep = weights(inp, prec)
    out = dec.forward(inp["x"].cuda(), inp["idx"].cuda(), inp["s"].cuda(), *W)
    dec.check()
    assert_close(out, oracle_out(inp, prec), prec, f"{kind} T={T}")


@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_few_wide_top32(prec):
    require_gpu()
    shape = (5, 2048, 768, 64, 32)
    inp = make(*shape, "uniform", 3)
    dec = decoder(*shape, prec)
    W, _keep = weights(inp, prec)
    out = dec.forward(inp["x"].cuda(), inp["idx"].cuda(), inp["s"].cuda(), *W)
    dec.check()
    assert_close(out, oracle_out(inp, prec), prec, "top-32")


@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_few_bad_index_is_recorded_and_adds_nothing(prec):
    require_gpu()
    from mixture_experts_layer_side_gb300 import _lib
    shape = (6, 256, 128, 8, 3)
    inp = make(*shape, "uniform", 1)
    idx, s = inp["idx"].clone(), inp["s"].clone()
    idx[1, 0], idx[3, 2], idx[4, :] = -1, 8, 10 ** 9
    dec = decoder(*shape, prec)
    W, _keep = weights(inp, prec)
    out = dec.forward(inp["x"].cuda(), idx.cuda(), inp["s"].cuda(), *W)
    with pytest.raises(_lib.MokError) as err:
        dec.check()
    assert err.value.status == 5
    bad = (idx < 0) | (idx >= 8)
    s[bad] = 0
    ref = oracle_out(inp, prec, idx=torch.where(bad, 0, idx).numpy(), s=np64(s))
    assert_close(out, ref, prec, "rows with ids left out")
    assert (out[4] == 0).all()
    # the error is forgotten, the workspace serves the next call
    out = dec.forward(inp["x"].cuda(), inp["idx"].cuda(), inp["s"].cuda(), *W)
    dec.check()
    assert_close(out, oracle_out(inp, prec), prec, "after a bad call")


def test_few_nan_and_inf_stay_in_their_token():
    require_gpu()
    shape = (5, 256, 128, 4, 2)
    inp = make(*shape, "one", 1)
    dec = decoder(*shape, "bf16")
    W, _keep = weights(inp, "bf16")
    x = inp["x"].clone()
    x[1, 3], x[3, 200] = float("nan"), float("inf")
    clean = dec.forward(inp["x"].cuda(), inp["idx"].cuda(), inp["s"].cuda(), *W)
    out = dec.forward(x.cuda(), inp["idx"].cuda(), inp["s"].cuda(), *W)
    dec.check()
    assert torch.isnan(out[1]).all()
    for t in (0, 2, 4):
        assert torch.equal(out[t], clean[t])


@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_few_takes_fewer_tokens_than_its_workspace(prec):
    require_gpu()
    T, H, I, E, k = 40, 384, 256, 10, 3
    inp = make(T, H, I, E, k, "zipf", 2)
    dec = decoder(T, H, I, E, k, prec)
    W, _keep = weights(inp, prec)
    ref = oracle_out(inp, prec)
    for n in (40, 1, 13, 0, 27, 40):
        out = dec.forward(inp["x"][:n].cuda(), inp["idx"][:n].cuda(), inp["s"][:n].cuda(), *W)
        assert out.shape == (n, H)
        if n:
            assert_close(out, ref[:n], prec, f"{n} tokens")
    dec.check()


def router_inputs(T, H, E, seed, biased):
    """x and Wr on a grid on which any order of the f32 sum is exact."""
    g = torch.Generator().manual_seed(seed)
    x = ((torch.randn((T, H), generator=g) * 32).round().clamp(-127, 127) / 32).to(torch.bfloat16)
    Wr = ((torch.randn((H, E), generator=g) * 40).round().clamp(-127, 127) / 2048).to(torch.bfloat16)
    bias = torch.randn(E, generator=g) if biased else None
    return x, Wr, bias


@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
@pytest.mark.parametrize("shape,biased", [((1, 256, 128, 8, 2), False), ((5, 384, 128, 5, 5), True),
                                          ((128, 256, 256, 65, 8), True), ((3, 7168, 128, 256, 8), True),
                                          ((20, 128, 128, 1024, 32), False), ((9, 1152, 128, 130, 1), True)])
def test_few_layer_with_router(shape, biased, prec):
    """Selection exact (the logits are exact in f32), scores to f32 rounding,
    the output against the oracle on that routing."""
    require_gpu()
    T, H, I, E, k = shape
    inp = make(*shape, "uniform", 7)
    x, Wr, bias = router_inputs(T, H, E, T + E, biased)
    inp["x"] = x
    dec = decoder(*shape, prec)
    W, _keep = weights(inp, prec)
    out, idx, s = dec.layer(x.cuda(), Wr.cuda(), *W, bias=bias.cuda() if biased else None)
    dec.check()
    logits = np64(x) @ np64(Wr)
    key = logits.astype(np.float32)
    assert (key == logits).all()
    if biased:
        key = key + bias.numpy()
    idx_ref, _ = router.topk_softmax(key.astype(np.float64), None, k)
    np.testing.assert_array_equal(idx.cpu().numpy(), idx_ref)
    ch = np.take_along_axis(logits, idx_ref, axis=1)
    ez = np.exp(ch - ch.max(axis=1, keepdims=True))
    s_ref = ez / ez.sum(axis=1, keepdims=True)
    np.testing.assert_allclose(s.cpu().numpy(), s_ref, rtol=2e-6, atol=1e-7)
    assert_close(out, oracle_out(inp, prec, idx=idx_ref, s=s_ref), prec, "layer")


def test_few_router_of_the_longest_rows():
    """128 tokens of the longest rows: what the logits' sums take of shared
    memory is longer than the stages beside them."""
    require_gpu()
    T, H, I, E, k = 128, 32768, 128, 16, 16
    inp = make(T, H, I, E, k, "uniform", 9)
    x, Wr, _ = router_inputs(T, H, E, 3, False)
    inp["x"] = x
    dec = decoder(T, H, I, E, k, "mxfp8")
    W, _keep = weights(inp, "mxfp8")
    out, idx, s = dec.layer(x.cuda(), Wr.cuda(), *W)
    dec.check()
    logits = np64(x) @ np64(Wr)
    assert (logits.astype(np.float32) == logits).all()
    idx_ref, _ = router.topk_softmax(logits, None, k)
    np.testing.assert_array_equal(idx.cpu().numpy(), idx_ref)
    ch = np.take_along_axis(logits, idx_ref, axis=1)
    ez = np.exp(ch - ch.max(axis=1, keepdims=True))
    s_ref = ez / ez.sum(axis=1, keepdims=True)
    np.testing.assert_allclose(s.cpu().numpy(), s_ref, rtol=2e-6, atol=1e-7)
    assert_close(out, oracle_out(inp, "mxfp8", idx=idx_ref, s=s_ref), "mxfp8", "longest rows")


def test_few_router_ties_and_nan():
    """Equal logits go to the lower expert; a NaN logit ranks last."""
    require_gpu()
    T, H, I, E, k = 4, 128, 128, 70, 6
    inp = make(T, H, I, E, k, "uniform", 1)
    x = torch.ones((T, H), dtype=torch.bfloat16)
    Wr = torch.zeros((H, E), dtype=torch.bfloat16)
    Wr[0, 40:50] = 1.0
    Wr[1, 41] = float("nan")
    dec = decoder(T, H, I, E, k, "bf16")
    W, _keep = weights(inp, "bf16")
    _, idx, s = dec.layer(x.cuda(), Wr.cuda(), *W)
    assert idx.cpu().tolist() == [[40, 42, 43, 44, 45, 46]] * T
    np.testing.assert_allclose(s.cpu().numpy(), 1 / 6, rtol=1e-6)


@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_few_agrees_with_the_training_forward(prec):
    """The same routing through MoKRouter / MoKLayer and in one call."""
    require_gpu()
    from mixture_experts_layer_side_gb300.inputs import Shape
    from mixture_experts_layer_side_gb300.layer import MoKLayer, MoKRouter
    shape = (24, 512, 256, 16, 4)
    inp = make(*shape, "uniform", 9)
    x, Wr, _ = router_inputs(24, 512, 16, 1, False)
    x, Wr = x.cuda(), Wr.cuda()
    W, _keep = weights(inp, prec)
    out, idx, s = decoder(*shape, prec).layer(x, Wr, *W)
    r, layer = MoKRouter(Shape(*shape)), MoKLayer(Shape(*shape), precision=prec)
    idx2, s2 = r.forward(x, Wr)
    assert torch.equal(idx, idx2)
    torch.testing.assert_close(s, s2, rtol=2e-6, atol=1e-7)
    layer.build_schedule(idx2)
    ref = layer.forward(x, s2, *W)
    assert_close(out, np64(ref), prec, "against mok_forward")


@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_few_reruns_are_bitwise_identical_also_in_a_graph_and_on_a_side_stream(prec):
    require_gpu()
    shape = (12, 512, 384, 20, 4)
    T, H, I, E, k = shape
    inp = make(*shape, "zipf", 4)
    x, Wr, bias = router_inputs(T, H, E, 5, True)
    x, Wr, bias = x.cuda(), Wr.cuda(), bias.cuda()
    dec = decoder(*shape, prec)
    W, _keep = weights(inp, prec)
    first = dec.layer(x, Wr, *W, bias=bias)
    for _ in range(20):
        again = dec.layer(x, Wr, *W, bias=bias)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again = dec.layer(x, Wr, *W, bias=bias)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dec.layer(x, Wr, *W, bias=bias)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    dec.check()


@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_few_wide_layer_on_sampled_columns(prec):
    """H = 7168, I = 2048: more work than one wave of tiles, against f64
    products on the GPU's own inputs."""
    require_gpu()
    shape = (6, 7168, 2048, 12, 3)
    inp = make(*shape, "uniform", 6)
    dec = decoder(*shape, prec)
    W, _keep = weights(inp, prec)
    out = dec.forward(inp["x"].cuda(), inp["idx"].cuda(), inp["s"].cuda(), *W)
    dec.check()
    assert_close(out, oracle_out(inp, prec), prec, "wide")
