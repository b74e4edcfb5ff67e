"""Infinities, extreme values, second parts and streams of the few-token
layer, the distillation loss and the embedding."""

import numpy as np
import pytest
import torch

from _helpers import np64, require_gpu

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- few tokens
def small_layer(shape, prec="bf16", seed=3):
    from mixture_experts_layer_side_gb300.decode import MoKDecoder
    from mixture_experts_layer_side_gb300.inputs import Shape, make_inputs
    return MoKDecoder(Shape(*shape), precision=prec), make_inputs(Shape(*shape), "uniform", seed=seed)


# a unit whose tiles are whole, tiles cut along K, experts of more rows than a step of the epilogue, 64 rows side by side
A_SHAPES = [(1, 128, 128, 4, 1), (7, 512, 1024, 4, 2), (33, 384, 640, 9, 3), (128, 1024, 384, 3, 2)]


@pytest.mark.parametrize("shape", A_SHAPES)
def test_few_second_part_of_the_hidden_values(shape):
    """h = h_t and u = h_t (even columns) or h_t (1 + 2^-12) (odd ones), W2 = +w and -w in turn: a's first bf16
    parts are equal but for boundaries between two bf16, so that y is what the second parts say.

    Tolerance.  a as two bf16 is off by 2^-9 of its second part, which is at most 2^-9 of a: 2^-18 |a|.  Its f32
    arithmetic (an exponential, a division, two products) and the sums over K (the tensor core's too, a few units of
    2^-23 of the largest term for each 16 of K) stay under 2^-19 |a| beside it.  y sums I of them; out is rounded
    once, 2^-8 of itself at most.  Without the second parts y would be off by half of I |a| 2^-12, 16 times the bound."""
    require_gpu()
    T, H, I, E, k = shape
    dec, inp = small_layer(shape)
    x = torch.zeros((T, H), dtype=torch.bfloat16)
    x[:, 0] = 1 + torch.arange(T) / 32         # exact in bf16
    x[:, H - 1] = x[:, 0] / 64
    W1, W3 = torch.zeros((E, H, I)), torch.zeros((E, H, I))
    W1[:, 0], W3[:, 0] = 1, 1
    W3[:, H - 1, 1::2] = 1 / 64                # x_0 / 64 / 64 = x_0 2^-12
    w = 1 + (torch.arange(H) % 4) / 4
    W2 = torch.empty((E, I, H))
    W2[:, 0::2], W2[:, 1::2] = w, -w
    s = torch.zeros((T, k))
    s[:, 0] = 1
    idx = (torch.arange(T)[:, None] + torch.arange(k)) % E
    out = dec.forward(x.cuda(), idx.int().cuda(), s.cuda(), *[m.bfloat16().cuda() for m in (W1, W3, W2)])
    dec.check()
    h = np64(x[:, 0])
    a = h / (1 + np.exp(-h)) * h
    ref = -(I / 2) * 2.0 ** -12 * a[:, None] * np64(w)
    bound = I * (2.0 ** -18 + 2.0 ** -19) * a[:, None] * np64(w) + 2.0 ** -8 * np.abs(ref)
    err = np.abs(np64(out) - ref)
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("shape", [(1, 7168, 128, 256, 8), (5, 7168, 128, 256, 8), (3, 1152, 128, 130, 8)])
def test_few_router_with_an_infinite_input(shape):
    """An infinite x makes the token's logits +-inf, wherever in its row it stands: the experts of +inf come first,
    those of -inf last, each in ascending order.  As MoKRouter has it; other tokens are as without it."""
    require_gpu()
    from mixture_experts_layer_side_gb300.inputs import Shape
    from mixture_experts_layer_side_gb300.layer import MoKRouter
    T, H, I, E, k = shape
    dec, inp = small_layer(shape)
    g = torch.Generator().manual_seed(5)
    Wr = (torch.randint(1, 128, (H, E), generator=g) * (torch.randint(0, 2, (H, E), generator=g) * 2 - 1) / 2048).bfloat16()
    x = ((torch.randn((T, H), generator=g) * 32).round().clamp(-127, 127) / 32).bfloat16()
    W = [inp[n].cuda() for n in ("W1", "W3", "W2")]
    clean = dec.layer(x.cuda(), Wr.cuda(), *W)[1].cpu()
    router = MoKRouter(Shape(*shape))
    # the rows at the ends of a part of the logits' sums, and others
    for at in [0, 1, H - 1] + [r for p in (H // 64 + 7 & ~7, (H // 64 + 7 & ~7) * 3) for r in (p - 1, p)]:
        xi = x.clone()
        xi[T - 1, at] = float("inf")
        Wr_at = Wr.clone()
        Wr_at[at] = -1
        Wr_at[at, 3::E // 4] = 1
        _, idx, _ = dec.layer(xi.cuda(), Wr_at.cuda(), *W)
        dec.check()
        up = list(range(3, E, E // 4))
        want = (up + [e for e in range(E) if e not in up])[:k]
        assert idx[T - 1].tolist() == want, at
        assert torch.equal(idx, router.forward(xi.cuda(), Wr_at.cuda())[0])
    assert torch.equal(dec.layer(x.cuda(), Wr.cuda(), *W)[1].cpu(), clean)


@pytest.mark.parametrize("shape", [(1, 128, 128, 4, 2), (6, 512, 1024, 4, 1), (33, 384, 640, 9, 3), (128, 1024, 384, 3, 2)])
def test_few_infinite_weights(shape):
    """An infinite W2 makes y what its one product says, +-inf, whatever a's second part is."""
    require_gpu()
    from oracle import moe
    T, H, I, E, k = shape
    dec, inp = small_layer(shape)
    W2 = inp["W2"].clone()
    for i, n in [(0, 5), (I // 2, 64), (I - 1, H - 1), (17, H // 2)]:
        W2[1, i, n] = float("inf")
        W2[1, i, (n + 9) % H] = -float("inf")
    out = dec.forward(*[inp[n].cuda() for n in ("x", "idx", "s", "W1", "W3")], W2.cuda())
    dec.check()
    a = {n: np64(v) for n, v in inp.items()}
    with np.errstate(invalid="ignore"):
        ref = moe.forward(a["x"], inp["idx"].numpy(), a["s"], a["W1"], a["W3"], np64(W2))[0]
    got = np64(out)
    assert np.isinf(ref).any()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))  # (two of either sign in one sum)
    np.testing.assert_array_equal(np.where(np.isinf(ref), ref, 0), np.where(np.isinf(got), got, 0))
    fin = np.isfinite(ref)
    assert np.abs(got[fin] - ref[fin]).max() <= 2e-2 * np.abs(ref[fin]).max()


# ---------------------------------------------------------------- distillation
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [0.25, 1.0, 4.0])
def test_distill_teacher_values_of_the_types_ends(tau, dtype):
    """Values at f32's lowest and highest: differences first, whatever the temperature."""
    require_gpu()
    from mixture_experts_layer_side_gb300.distill import DistillLoss
    from test_distill_gpu import check, make
    T, V, K = 5, 900, 6
    lo, hi = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    _, z, ids, vals, dloss = make(T, V, K, dtype, 4, masked=0.0)
    vals[0] = lo                                  # all masked alike: uniform
    vals[1] = torch.tensor([lo, lo, lo, 1.0, 2.0, -3.0])
    vals[2] = torch.tensor([hi, 0.0, 1.0, lo, 5.0, 6.0])
    vals[3] = hi
    vals[4] = torch.tensor([lo, -np.inf, lo, -np.inf, 0.0, 0.0])
    ids[4, 4:] = -1
    d = DistillLoss(T, V, K)
    a = [t.cuda() for t in (z, ids, vals, dloss)]
    loss, lse = d.forward(*a[:3], temperature=tau)
    dz = d.backward(*a[:3], lse, a[3], temperature=tau)
    loss2, dz2 = d.forward_backward(*a, temperature=tau)
    d.check()
    check(z, ids, vals, dloss, tau, loss, lse, dz, dtype)
    check(z, ids, vals, dloss, tau, loss2, None, dz2, dtype)


@pytest.mark.parametrize("V,dtype", [(900011, "bf16"), (600011, "f32")])
def test_distill_rows_past_eight_blocks(V, dtype):
    """A row too long for eight blocks' shared memory: the step is two launches."""
    require_gpu()
    from mixture_experts_layer_side_gb300 import _lib
    from mixture_experts_layer_side_gb300.distill import DistillLoss
    from test_distill_gpu import make, run_all
    run_all(2, V, 16, dtype, 1.0, 1)
    _, z, ids, vals, dloss = make(2, V, 16, dtype, 1)
    d = DistillLoss(2, V, 16)
    before = _lib.mok_launch_count()
    d.forward_backward(z.cuda(), ids.cuda(), vals.cuda(), dloss.cuda())
    assert _lib.mok_launch_count() - before == 2


@pytest.mark.parametrize("V", [9000, 900011])
def test_distill_step_on_rows_of_the_lowest_value_at_a_low_temperature(V):
    """The lowest value over the temperature is past f32; the differences are zero all the same."""
    require_gpu()
    from mixture_experts_layer_side_gb300.distill import DistillLoss
    z = torch.full((2, V), torch.finfo(torch.bfloat16).min, dtype=torch.bfloat16)
    z[1, 100:] = -np.inf
    ids = torch.tensor([[0, 5], [7, 9]]).int()
    d = DistillLoss(2, V, 2)
    loss, dz = d.forward_backward(z.cuda(), ids.cuda(), torch.zeros(2, 2).cuda(), torch.ones(2).cuda(), temperature=0.5)
    d.check()
    np.testing.assert_allclose(loss.cpu().numpy(), [np.log(V) + np.log(0.5), np.log(100) + np.log(0.5)], rtol=1e-5)
    q = torch.zeros((2, V), dtype=torch.float64)
    q[0], q[1, :100] = 1 / V, 1 / 100
    q[0, ids[0].long()] -= 0.5
    q[1, ids[1].long()] -= 0.5
    err = (dz.double().cpu() - 2 * q).abs()
    assert (err <= 2.0 ** -8 * (2 * q).abs() + 1e-5 * 2 * q.abs().amax(1, keepdim=True)).all()


# ---------------------------------------------------------------- embedding
@pytest.mark.parametrize("N", [40, 5000])
def test_embedding_the_lowest_id_is_an_error_where_there_is_no_padding(N):
    require_gpu()
    from mixture_experts_layer_side_gb300 import _lib
    from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
    V, H = 50, 16
    ids = (torch.arange(N) % V).int()
    ids[7] = -2 ** 31
    table, dx = torch.randn(V, H), torch.randn(N, H)
    e = MoKEmbedding(V, H, N)
    for call in (lambda: e.forward(table.cuda(), ids.cuda()), lambda: e.backward(dx.cuda(), ids.cuda())):
        call()
        with pytest.raises(_lib.MokError) as err:
            e.check()
        assert err.value.status == 5
        e.check()


# ---------------------------------------------------------------- streams
def stream_calls():
    """(name, call(stream) -> tensors, bytes of the largest of them) of every class's methods, of sizes that the
    allocator serves with a block of their own."""
    from mixture_experts_layer_side_gb300.distill import DistillLoss
    from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
    from test_distill_gpu import make
    dec, inp = small_layer((128, 16384, 128, 4, 2))
    i = {n: v.cuda() for n, v in inp.items()}
    Wr = torch.randn((16384, 4), device="cuda").bfloat16()
    W = [i[n] for n in ("W1", "W3", "W2")]
    yield "few forward", lambda s: dec.forward(i["x"], i["idx"], i["s"], *W, stream=s), 128 * 16384 * 2, dec
    yield "few layer", lambda s: dec.layer(i["x"], Wr, *W, stream=s), 128 * 16384 * 2, dec
    T, V = 512, 8192
    a = [t.cuda() for t in make(T, V, 8, "f32", 1)[1:]]
    d = DistillLoss(T, V, 8)
    lse = d.forward(*a[:3])[1]
    yield "distill backward", lambda s: d.backward(*a[:3], lse, a[3], stream=s), T * V * 4, d
    yield "distill step", lambda s: d.forward_backward(*a, stream=s), T * V * 4, d
    e = MoKEmbedding(4096, 1024, 4096)
    table, ids = torch.randn(4096, 1024, device="cuda"), torch.randint(0, 4096, (4096,), device="cuda").int()
    yield "embed forward", lambda s: e.forward(table, ids, stream=s), 4096 * 1024 * 4, e
    yield "embed backward", lambda s: e.backward(table, ids, stream=s), 4096 * 1024 * 4, e


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_on_another_stream_take_no_memory_in_use(raw):
    """A tensor that the current stream still has to read is dropped, and a call is made on another stream at once:
    its outputs may not take that memory.  And outputs that are dropped while the current stream still reads them
    are not taken by the next call on the other."""
    require_gpu()
    side = torch.cuda.Stream()
    arg = side.cuda_stream if raw else side
    for name, call, size, owner in stream_calls():
        want = call(None)
        want = want if isinstance(want, tuple) else (want,)
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        kept = torch.full((size // 4,), 7, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)  # 50 ms
        copy = kept.clone()
        del kept
        got = call(arg)
        got = got if isinstance(got, tuple) else (got,)
        torch.cuda.synchronize()
        assert (copy == 7).all(), name
        assert all(torch.equal(a, b) for a, b in zip(want, got)), name
        del copy, got
        # outputs read on the current stream, late, and dropped before
        got = call(arg)
        got = got if isinstance(got, tuple) else (got,)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(100_000_000)
        copies = [t.clone() for t in got]
        del got
        with torch.cuda.stream(side):
            over = [torch.zeros_like(t) for t in want]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, copies)), name
        owner.check(stream=arg)
        del over, copies, want


def test_a_workspace_is_ready_for_every_stream():
    """The zeros of a new workspace are there for a first call on another stream."""
    require_gpu()
    from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
    side = torch.cuda.Stream()
    table, ids = torch.randn(64, 64, device="cuda"), torch.arange(64, device="cuda").int()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    e = MoKEmbedding(64, 64, 64)
    assert torch.cuda.current_stream().query()  # nothing of it is still to come
    out = e.forward(table, ids, stream=side)
    e.check(stream=side)
    assert torch.equal(out, table)


def test_a_stream_of_another_device_is_refused():
    require_gpu()
    from mixture_experts_layer_side_gb300 import _check

    class Other:
        device = torch.device("cuda", 7)

    with pytest.raises(ValueError):
        _check.run_on(Other, torch.cuda.Stream(), lambda: None)


# ---------------------------------------------------------------- the longest rows and offsets
@pytest.mark.parametrize("V,launches", [(851968, 1), (851976, 2)])
def test_distill_rows_that_just_fit_eight_blocks(V, launches):
    """The last length of eight blocks' shared memory, with the longest list beside it, and the next."""
    require_gpu()
    from mixture_experts_layer_side_gb300 import _lib
    from mixture_experts_layer_side_gb300.distill import DistillLoss
    from test_distill_gpu import check, make
    _, z, ids, vals, dloss = make(2, V, 512, "bf16", 5)
    d = DistillLoss(2, V, 512)
    before = _lib.mok_launch_count()
    loss, dz = d.forward_backward(z.cuda(), ids.cuda(), vals.cuda(), dloss.cuda())
    assert _lib.mok_launch_count() - before == launches
    d.check()
    check(z, ids, vals, dloss, 1.0, loss, None, dz, "bf16")


def test_distill_offsets_past_32_bits():
    """Rows 2^26 elements apart: the last lies 2.6e9 elements from the first."""
    require_gpu()
    from mixture_experts_layer_side_gb300.distill import DistillLoss
    from test_distill_gpu import check, make
    T, V, K, ld = 40, 5003, 7, 1 << 26
    _, z, ids, vals, dloss = make(T, V, K, "bf16", 6)
    a = [t.cuda() for t in (ids, vals, dloss)]
    far = torch.empty((T - 1) * ld + V, dtype=torch.bfloat16, device="cuda").as_strided((T, V), (ld, 1))
    far.copy_(z)
    d = DistillLoss(T, V, K)
    loss, lse = d.forward(far, *a[:2])
    dz = d.backward(far, *a[:2], lse, a[2])
    check(z, ids, vals, dloss, 1.0, loss, lse, dz, "bf16")
    loss2, dz2 = d.forward_backward(far, *a, out=far)
    d.check()
    check(z, ids, vals, dloss, 1.0, loss2, None, dz2, "bf16")


def test_distill_the_longest_row():
    """2^30 logits of 0 but for a few: sums of terms that are 1 are exact, so that the tolerances are the types'."""
    require_gpu()
    from mixture_experts_layer_side_gb300.distill import DistillLoss
    V = 1 << 30
    z = torch.zeros((1, V), dtype=torch.bfloat16, device="cuda")
    z[0, V - 1], z[0, 1 << 29] = 16.0, -float("inf")
    ids = torch.tensor([[V - 1, 3]], dtype=torch.int32, device="cuda")
    d = DistillLoss(1, V, 2)
    one = torch.ones(1, device="cuda")
    total = V - 2 + np.exp(16.0)
    loss, dz = d.forward_backward(z, ids, torch.zeros((1, 2), device="cuda"), one)
    want = np.log(0.5) - (0.5 * 16.0 - np.log(total))
    assert abs(float(loss) - want) <= 1e-5 * (1 + abs(want))
    fwd, lse = d.forward(z, ids, torch.zeros((1, 2), device="cuda"))
    assert abs(float(lse) - np.log(total)) <= 1e-5 * np.log(total) and abs(float(fwd) - want) <= 1e-5 * (1 + abs(want))
    d.check()
    g = dz[0]
    assert float(g[1 << 29]) == 0.0
    for at, q in ((V - 1, np.exp(16.0) / total - 0.5), (3, 1 / total - 0.5)):
        assert abs(float(g[at]) - q) <= 2.0 ** -8 * abs(q)
    rest = torch.ones(V, dtype=torch.bool, device="cuda")
    rest[[V - 1, 3, 1 << 29]] = False
    lo, hi = g.masked_fill(~rest, float(g[0])).aminmax()
    assert abs(float(lo) * total - 1) <= 2.0 ** -8 + 1e-5 and abs(float(hi) * total - 1) <= 2.0 ** -8 + 1e-5


@pytest.mark.parametrize("V,H,N", [(300000, 8192, 100), (300000, 8192, 5000), (1 << 30, 2, 100), (1 << 30, 2, 5000)])
def test_embedding_offsets_past_32_bits(V, H, N):
    """Rows past 2^31 elements, and the most rows that a table may have: ids near the end, two tokens each."""
    require_gpu()
    from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
    e = MoKEmbedding(V, H, N, pad_id=V - 1)
    g = torch.Generator(device="cuda").manual_seed(N)
    ids = V - 2 - torch.randperm(N, generator=g, device="cuda") // 2
    ids[0] = V - 1
    dx = torch.randn((N, H), generator=g, device="cuda").bfloat16()
    want = torch.zeros((N, H), device="cuda", dtype=torch.float64)      # of the last N rows
    use = ids != V - 1
    want.index_add_(0, (ids - (V - N))[use], dx[use].double())
    out = torch.full((V, H), 3.0, dtype=torch.bfloat16, device="cuda")
    e.backward(dx, ids.int(), out=out)
    assert torch.equal(out[V - N:], want.float().bfloat16())            # (two bf16 terms: exact in f32 but for their span)
    assert not out[:V - N].any()
    e.backward(dx, ids.int(), out=out, accumulate=True)
    assert (out[V - N:].double() - 2 * want).abs().max() <= 2.0 ** -7 * want.abs().max()
    got = e.forward(out, ids.int())
    e.check()
    assert torch.equal(got, out[ids])
