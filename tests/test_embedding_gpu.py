"""The token embedding and its gradient against float64 sums: odd widths and
vocabularies, tokens that are alone, shared by thousands, padding or out of
range, both forms of the gradient, reruns, differences.

Tolerances.  The lookup is one f32 product rounded once: bitwise.  A row's
gradient is an f32 sum of n terms and one product: at most (n + 2) 2^-23 of the
sum of their magnitudes, and 2^-8 of itself more where it is rounded to bf16."""

import numpy as np
import pytest
import torch

from _helpers import np64, require_gpu

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def make_ids(N, V, kind, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        return torch.full((N,), V // 2, dtype=torch.int32)
    if kind == "skew":
        p = 1.0 / (torch.arange(V) + 2.7)
        return torch.multinomial(p, N, replacement=True, generator=g).int()
    return torch.randint(0, V, (N,), generator=g).int()


def plain(dx, ids, V, scale):
    """(gradient, sum of magnitudes, tokens of each row) in float64; ids < 0 left out."""
    dx, ids = np64(dx), ids.numpy()
    use = (ids >= 0) & (ids < V)
    full, size, count = np.zeros((V, dx.shape[1])), np.zeros((V, dx.shape[1])), np.zeros(V)
    np.add.at(full, ids[use], dx[use])
    np.add.at(size, ids[use], np.abs(dx[use]))
    np.add.at(count, ids[use], 1)
    return full * scale, size * abs(scale), count


def assert_gradient(got, dx, ids, V, scale, grad, base=None):
    ref, size, count = plain(dx, ids, V, scale)
    if base is not None:
        ref, size = ref + np64(base), size + np.abs(np64(base))
    got = np64(got)
    bound = (count[:, None] + 2) * 2.0 ** -23 * size + (2.0 ** -8 * np.abs(ref) if grad == "bf16" else 0)
    err = np.abs(got - ref)
    assert (err <= bound).all(), float((err - bound).max())
    untouched = count == 0
    want = np.zeros_like(ref) if base is None else np64(base)
    np.testing.assert_array_equal(got[untouched], want[untouched])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,H", [(1, 1, 1), (5, 3, 7), (64, 1000, 256), (1000, 77, 520), (33, 500, 1003),
                                   (4097, 5000, 128)])
def test_lookup_is_bitwise(N, V, H, dtype):
    require_gpu()
    from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
    g = torch.Generator().manual_seed(N + V)
    table = torch.randn((V, H), generator=g).to(TYPES[dtype])
    ids = make_ids(N, V, "uniform", 1)
    e = MoKEmbedding(V, H, N)
    for scale in (1.0, float(np.float32(np.sqrt(H))), -0.3):
        out = e.forward(table.cuda(), ids.cuda(), scale=scale)
        ref = (table.float() * np.float32(scale)).to(TYPES[dtype])[ids.long()]
        assert torch.equal(out.cpu(), ref)
    e.check()


def test_lookup_shapes_padding_and_bad_ids():
    require_gpu()
    from mixture_experts_layer_side_gb300 import _lib
    from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
    V, H = 50, 264
    table = torch.randn((V, H), generator=torch.Generator().manual_seed(1)).cuda()
    ids = torch.randint(0, V, (3, 11), generator=torch.Generator().manual_seed(2)).int()
    e = MoKEmbedding(V, H, 64, pad_id=-1)
    ids[0, 3] = -1  # padding outside the table: zeros, no error
    out = e.forward(table, ids.cuda())
    e.check()
    assert out.shape == (3, 11, H) and (out[0, 3] == 0).all()
    inside = ids != -1
    assert torch.equal(out.cpu()[inside], table.cpu()[ids[inside].long()])
    assert e.forward(table, ids[:, :0].cuda()).shape == (3, 0, H)
    for bad in (V, -2, 2 ** 31 - 1):
        ids[1, 1] = bad
        out = e.forward(table, ids.cuda())
        assert (out[1, 1] == 0).all()
        with pytest.raises(_lib.MokError) as err:
            e.check()
        assert err.value.status == 5
    # padding inside the table reads its row
    e = MoKEmbedding(V, H, 64, pad_id=7)
    assert torch.equal(e.forward(table, torch.full((2,), 7, dtype=torch.int32, device="cuda")), table[[7, 7]])
    e.check()


CASES = [(1, 1, 1, "uniform"), (1, 1000, 256, "uniform"), (7, 3, 5, "uniform"), (32, 4, 128, "uniform"),
         (33, 9, 130, "one"), (64, 9, 512, "one"), (1000, 100, 264, "skew"), (3000, 50, 1003, "uniform"),
         (5000, 1, 64, "one"), (4096, 5000, 328, "skew"), (9000, 70000, 40, "skew"), (20000, 2000, 96, "one"),
         (2049, 1023, 33, "uniform"), (2049, 1024, 33, "uniform"), (70001, 300, 16, "skew"),
         (300, 1100000, 8, "uniform"), (8192, 524287, 8, "skew"), (8193, 300, 24, "skew"), (4096, 1048575, 4, "uniform"),
         (4096, 1048576, 4, "uniform"), (2000, 2097152, 2, "uniform")]


@pytest.mark.parametrize("dx_type,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("N,V,H,kind", CASES)
def test_gradient_matches_sums(N, V, H, kind, dx_type, grad):
    require_gpu()
    from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
    g = torch.Generator().manual_seed(N + V)
    dx = torch.randn((N, H), generator=g).to(TYPES[dx_type])
    ids = make_ids(N, V, kind, 1)
    e = MoKEmbedding(V, H, N)
    out = torch.full((V, H), float("nan"), dtype=TYPES[grad], device="cuda")
    e.backward(dx.cuda(), ids.cuda(), scale=0.7, out=out)
    assert_gradient(out, dx, ids, V, np.float32(0.7), grad)
    base = torch.randn((V, H), generator=g).to(TYPES[grad])
    acc = base.cuda()
    e.backward(dx.cuda(), ids.cuda(), scale=0.7, out=acc, accumulate=True)
    assert_gradient(acc, dx, ids, V, np.float32(0.7), grad, base=base)
    e.check()


def test_gradient_wide_rows():
    require_gpu()
    from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
    N, V, H = 3000, 400, 7168
    g = torch.Generator(device="cuda").manual_seed(1)
    dx = torch.randn((N, H), generator=g, device="cuda").to(torch.bfloat16)
    ids = make_ids(N, V, "skew", 1)
    e = MoKEmbedding(V, H, N)
    assert_gradient(e.backward(dx, ids.cuda()), dx.cpu(), ids, V, 1.0, "f32")


@pytest.mark.parametrize("grad", ["bf16", "f32"])
def test_gradient_padding_and_bad_ids(grad):
    require_gpu()
    from mixture_experts_layer_side_gb300 import _lib
    from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
    N, V, H = 700, 90, 72
    g = torch.Generator().manual_seed(5)
    dx = torch.randn((N, H), generator=g)
    ids = make_ids(N, V, "skew", 3)
    ids[::7] = 4
    e = MoKEmbedding(V, H, N, pad_id=4)
    kept = torch.where(ids == 4, -1, ids)
    out = e.backward(dx.cuda(), ids.cuda(), out=torch.full((V, H), 9.0, device="cuda", dtype=TYPES[grad]))
    e.check()
    assert_gradient(out, dx, kept, V, 1.0, grad)
    ids[5], ids[6], ids[13] = V, -1, -2 ** 31
    kept = torch.where((ids == 4) | (ids < 0) | (ids >= V), -1, ids)
    out = e.backward(dx.cuda(), ids.cuda(), out=out)
    assert_gradient(out, dx, kept, V, 1.0, grad)
    with pytest.raises(_lib.MokError) as err:
        e.check()
    assert err.value.status == 5
    # nothing but padding, and nothing at all
    base = torch.randn((V, H), generator=g).to(TYPES[grad]).cuda()
    was = base.clone()
    e.backward(dx.cuda(), torch.full((N,), 4, dtype=torch.int32, device="cuda"), out=base, accumulate=True)
    e.backward(dx[:0].cuda(), ids[:0].cuda(), out=base, accumulate=True)
    assert torch.equal(base, was)
    e.backward(dx[:0].cuda(), ids[:0].cuda(), out=base)
    assert (base == 0).all()
    e.check()


def test_gradient_takes_fewer_tokens_and_unaligned_tensors():
    """Views that start one element into their storage."""
    require_gpu()
    from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
    N, V, H = 500, 60, 128
    g = torch.Generator().manual_seed(5)
    e = MoKEmbedding(V, H, N)
    for n in (500, 3, 131):
        for t in ("bf16", "f32"):
            dx = torch.randn(n * H + 1, generator=g).to(TYPES[t])
            ids = make_ids(n + 1, V, "skew", n)
            dxc, idc = dx.cuda()[1:].view(n, H), ids.cuda()[1:]
            out = torch.empty(V * H + 1, dtype=TYPES[t], device="cuda")[1:].view(V, H)
            e.backward(dxc, idc, out=out)
            assert_gradient(out, dx[1:].view(n, H), ids[1:], V, 1.0, t)
            table = torch.randn(V * H + 1, generator=g).to(TYPES[t])
            got = e.forward(table.cuda()[1:].view(V, H), idc)
            assert torch.equal(got.cpu(), table[1:].view(V, H)[ids[1:].long()])
    e.check()


def test_gradient_against_differences():
    """<dtable, U> against the change of <forward(table), dx> along U: both
    are linear, so one step of 1 is exact but for f32 rounding."""
    require_gpu()
    from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
    N, V, H = 400, 37, 96
    g = torch.Generator().manual_seed(6)
    table, U = torch.randn((V, H), generator=g), torch.randn((V, H), generator=g)
    dx = torch.randn((N, H), generator=g)
    ids = make_ids(N, V, "skew", 3)
    e = MoKEmbedding(V, H, N)
    grad = e.backward(dx.cuda(), ids.cuda(), scale=1.5)
    hi = e.forward((table + U).cuda(), ids.cuda(), scale=1.5)
    lo = e.forward(table.cuda(), ids.cuda(), scale=1.5)
    change = ((hi.double() - lo.double()).cpu() * dx.double()).sum()
    along = (grad.double().cpu() * U.double()).sum()
    assert abs(change - along) <= 1e-5 * dx.double().norm() * U.double().norm()


def test_gradient_reruns_graph_and_side_stream():
    require_gpu()
    from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
    N, V, H = 6000, 900, 264
    dx = torch.randn((N, H), generator=torch.Generator().manual_seed(1)).cuda()
    ids = make_ids(N, V, "skew", 3).cuda()
    e = MoKEmbedding(V, H, N)
    first = e.backward(dx, ids)
    for _ in range(20):
        assert torch.equal(first, e.backward(dx, ids))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again = e.backward(dx, ids)
    side.synchronize()
    assert torch.equal(first, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = e.backward(dx, ids)
    got.fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, got)
