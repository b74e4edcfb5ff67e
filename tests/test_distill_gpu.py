"""The distillation loss and its gradient against a plain float64 reading of
the formulas: vocabularies of every alignment, strided and in-place rows,
lists that are ragged, empty or name an id twice, -inf on either side,
differences of the loss, and reruns.

Tolerances.  The kernel's terms are exp(z / tau - lse) in f32: the argument is
rounded at |z| / tau + |lse| <= 64 units, so a term is off by at most about
64 * 2^-23 = 8e-6 of itself, and a few more units of 2^-22 for the
exponential: 1e-5 of the row's largest term bounds an f32 gradient.  A bf16
gradient is rounded once more: 2^-8 of itself.  The loss and lse are sums of
the same kind: 1e-5 * (1 + |lse| + |loss|)."""

import numpy as np
import pytest
import torch

from _helpers import require_gpu

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(T, V, K, dtype, seed, pad=0, offset=0, masked=0.3):
    """z [T, V] (a view with rows V + pad apart, `offset` elements into its
    storage), ids, vals, dloss on the CPU."""
    g = torch.Generator().manual_seed(seed)
    store = (3.0 * torch.randn(T * (V + pad) + offset, generator=g)).to(TYPES[dtype])
    z = store[offset:].view(T, V + pad)[:, :V]
    ids = torch.stack([torch.randperm(V, generator=g)[:K] if V >= K else torch.randint(0, V, (K,), generator=g)
                       for _ in range(T)]).int()
    ids[torch.rand(ids.shape, generator=g) < masked] = -1
    vals = 5.0 * torch.randn((T, K), generator=g)
    dloss = torch.rand(T, generator=g) + 0.1
    return store, z, ids, vals, dloss


def plain(z, ids, vals, dloss, tau):
    """(loss, lse, dz) in float64."""
    z = z.double().numpy() / tau
    ids, vals = ids.numpy().astype(np.int64), vals.double().numpy()
    T, V = z.shape
    with np.errstate(divide="ignore", invalid="ignore"):
        top = z.max(1, keepdims=True)
        lse = (top + np.log(np.exp(z - top).sum(1, keepdims=True)))[:, 0]
    loss, dz = np.zeros(T), np.zeros((T, V))
    for t in range(T):
        use = ids[t] >= 0
        v = vals[t][use] / tau
        if v.size == 0 or v.max() == -np.inf:
            continue
        p = np.exp(v - v.max())
        p /= p.sum()
        at = ids[t][use]
        log_q = z[t][at] - lse[t]
        on = p > 0
        loss[t] = (p[on] * (np.log(p[on]) - log_q[on])).sum()
        g = np.exp(z[t] - lse[t])
        np.add.at(g, at, -p)
        dz[t] = g * float(dloss[t]) / tau
    return loss, lse, dz


def view_like(store, z, device="cuda"):
    s = store.to(device)
    return s.as_strided(z.shape, z.stride(), z.storage_offset())


def check(z, ids, vals, dloss, tau, loss, lse, dz, dtype):
    loss_r, lse_r, dz_r = plain(z, ids, vals, dloss, tau)
    if lse is not None:
        np.testing.assert_allclose(lse.double().cpu().numpy(), lse_r, rtol=1e-5, atol=1e-5)
    if loss is not None:
        got = loss.double().cpu().numpy()
        inf = np.isinf(loss_r)
        np.testing.assert_array_equal(np.isinf(got), inf)
        assert (np.abs(got - loss_r)[~inf] <= 1e-5 * (1 + np.abs(lse_r) + np.abs(loss_r))[~inf]).all()
    if dz is not None:
        got = dz.double().cpu().numpy()
        top = np.abs(dz_r).max(1, keepdims=True)
        scale = np.maximum(top, (dloss.numpy() / tau)[:, None] * (top > 0))
        bound = 1e-5 * scale + (2.0 ** -8 * np.abs(dz_r) if dtype == "bf16" else 0)
        err = np.abs(got - dz_r)
        assert (err <= bound).all(), float((err - bound).max())


def run_all(T, V, K, dtype, tau, seed, **kw):
    from mixture_experts_layer_side_gb300.distill import DistillLoss
    store, z, ids, vals, dloss = make(T, V, K, dtype, seed, **kw)
    d = DistillLoss(T, V, K)
    zc, idc, vc, gc = view_like(store, z), ids.cuda(), vals.cuda(), dloss.cuda()
    loss, lse = d.forward(zc, idc, vc, temperature=tau)
    check(z, ids, vals, dloss, tau, loss, lse, None, dtype)
    out = torch.full((T, V + 3), float("nan"), dtype=TYPES[dtype], device="cuda")
    dz = d.backward(zc, idc, vc, lse, gc, temperature=tau, out=out[:, :V])
    assert torch.isnan(out[:, V:]).all()
    check(z, ids, vals, dloss, tau, None, None, dz, dtype)
    loss2, dz2 = d.forward_backward(zc, idc, vc, gc, temperature=tau)
    check(z, ids, vals, dloss, tau, loss2, None, dz2, dtype)
    # in place, and nothing beside the rows is touched
    inplace = view_like(store, z)
    loss3, dz3 = d.forward_backward(inplace, idc, vc, gc, temperature=tau, out=inplace)
    assert dz3.data_ptr() == inplace.data_ptr()
    assert torch.equal(loss2, loss3) and torch.equal(dz2, dz3)
    inplace2 = view_like(store, z)
    assert torch.equal(d.backward(inplace2, idc, vc, lse, gc, temperature=tau, out=inplace2), dz)
    if z.stride(0) > V and T > 1:
        gap = inplace.as_strided((T - 1, z.stride(0) - V), (z.stride(0), 1), z.storage_offset() + V)
        was = store.as_strided((T - 1, z.stride(0) - V), (z.stride(0), 1), z.storage_offset() + V)
        assert torch.equal(gap.cpu(), was)
    d.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (3, 2, 2), (5, 7, 3), (2, 31, 31), (9, 257, 5), (4, 1000, 512),
                                   (17, 4099, 33), (6, 32000, 64), (3, 50001, 20), (2, 131072, 100), (130, 515, 8), (400, 16385, 12),
                                   (650, 40007, 9)])
def test_distill_matches_formula(T, V, K, dtype):
    require_gpu()
    run_all(T, V, K, dtype, 1.0 if T % 2 else 2.5, T + V)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 1, 3, 8, 13])
@pytest.mark.parametrize("offset", [0, 1, 5])
def test_distill_strides_and_alignments(offset, pad, dtype):
    require_gpu()
    run_all(5, 1003, 12, dtype, 0.5, offset + pad, pad=pad, offset=offset)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distill_longest_rows(dtype):
    """A vocabulary past any on-chip form of the row."""
    require_gpu()
    run_all(2, 600011, 16, dtype, 1.0, 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distill_empty_lists_and_infinities(dtype):
    require_gpu()
    from mixture_experts_layer_side_gb300.distill import DistillLoss
    T, V, K = 8, 700, 6
    _, z, ids, vals, dloss = make(T, V, K, dtype, 3, masked=0.0)
    z = z.clone()
    ids[0] = -1                                    # an empty list
    vals[1] = -np.inf                              # a list of -inf alone
    vals[2, 3] = -np.inf                           # one entry of p = 0 ...
    z[2, int(ids[2, 3])] = -np.inf                 # ... where q = 0 too
    z[3, :] = -np.inf                              # one token left
    z[3, 5] = 1.0
    ids[3] = torch.tensor([5, -1, -1, -1, -1, -1])
    z[4, int(ids[4, 0])] = -np.inf                 # p > 0 where q = 0: the loss is +inf
    z[5] = torch.finfo(TYPES[dtype]).min           # the lowest value everywhere but one place
    z[5, 9] = 0.0
    ids[5] = torch.tensor([9, 9, -1, 9, -1, -1])   # the same id three times
    vals[6, 2] = np.nan                            # a value whose id is left out
    ids[6, 2] = -1
    vals[7] = torch.tensor([80.0, -80.0, 0.0, 1.0, 2.0, 3.0])  # p of all sizes down to zero
    d = DistillLoss(T, V, K)
    a = [t.cuda() for t in (z, ids, vals, dloss)]
    loss, lse = d.forward(a[0], a[1], a[2])
    dz = d.backward(a[0], a[1], a[2], lse, a[3])
    loss2, dz2 = d.forward_backward(*a)
    d.check()
    for lo, g in ((loss, dz), (loss2, dz2)):
        check(z, ids, vals, dloss, 1.0, lo, lse, g, dtype)
        assert lo[0] == 0 and lo[1] == 0 and torch.isinf(lo[4])
        assert (g[0] == 0).all() and (g[1] == 0).all()


def test_distill_nan_rows_stay_alone_and_empty_lists_win():
    require_gpu()
    from mixture_experts_layer_side_gb300.distill import DistillLoss
    T, V, K = 4, 5000, 4
    _, z, ids, vals, dloss = make(T, V, K, "f32", 3, masked=0.0)
    z = z.clone()
    z[1, 4000] = float("nan")
    z[2, 17] = float("nan")
    ids[2] = -1
    d = DistillLoss(T, V, K)
    loss, dz = d.forward_backward(*[t.cuda() for t in (z, ids, vals, dloss)])
    assert torch.isnan(loss[1]) and torch.isnan(dz[1]).all()
    assert loss[2] == 0 and (dz[2] == 0).all()
    keep = [0, 3]
    check(z[keep], ids[keep], vals[keep], dloss[keep], 1.0, loss[keep], None, dz[keep], "f32")


def test_distill_bad_ids_are_recorded_and_left_out():
    require_gpu()
    from mixture_experts_layer_side_gb300 import _lib
    from mixture_experts_layer_side_gb300.distill import DistillLoss
    T, V, K = 3, 100, 5
    _, z, ids, vals, dloss = make(T, V, K, "f32", 3, masked=0.0)
    bad = ids.clone()
    bad[0, 1], bad[1, 0], bad[2, 4] = V, -2, 2 ** 31 - 1
    ids[bad != ids] = -1
    d = DistillLoss(T, V, K)
    loss, dz = d.forward_backward(z.cuda(), bad.cuda(), vals.cuda(), dloss.cuda())
    check(z, ids, vals, dloss, 1.0, loss, None, dz, "f32")
    with pytest.raises(_lib.MokError) as err:
        d.check()
    assert err.value.status == 5
    d.check()


def test_distill_gradient_against_differences():
    """Central differences of the forward's loss along random directions; the
    loss is f32, so a step of 2^-5 leaves an error of about 1e-6 / 2^-5 + h^2."""
    require_gpu()
    from mixture_experts_layer_side_gb300.distill import DistillLoss
    T, V, K, tau, h = 6, 300, 10, 2.0, 2.0 ** -5
    _, z, ids, vals, _ = make(T, V, K, "f32", 8)
    ids[0] = torch.arange(10)
    one = torch.ones(T)
    d = DistillLoss(T, V, K)
    a = [t.cuda() for t in (z, ids, vals)]
    loss, lse = d.forward(*a, temperature=tau)
    dz = d.backward(*a, lse, one.cuda(), temperature=tau).double().cpu()
    g = torch.Generator().manual_seed(2)
    for _ in range(5):
        u = torch.randn((T, V), generator=g)
        hi = d.forward((z + h * u).cuda(), *a[1:], temperature=tau)[0].double().cpu()
        lo = d.forward((z - h * u).cuda(), *a[1:], temperature=tau)[0].double().cpu()
        slope = (dz * u.double()).sum(1)
        assert ((hi - lo) / (2 * h) - slope).abs().max() < 2e-3, ((hi - lo) / (2 * h) - slope).abs().max()


def test_distill_reruns_graph_and_side_stream():
    require_gpu()
    from mixture_experts_layer_side_gb300.distill import DistillLoss
    T, V, K = 40, 9001, 16
    _, z, ids, vals, dloss = make(T, V, K, "bf16", 3)
    d = DistillLoss(T, V, K)
    a = [t.cuda() for t in (z, ids, vals, dloss)]
    first = d.forward_backward(*a)
    for _ in range(10):
        assert all(torch.equal(x, y) for x, y in zip(first, d.forward_backward(*a)))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again = d.forward_backward(*a)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = d.forward_backward(*a)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, got))


def test_distill_no_rows():
    require_gpu()
    from mixture_experts_layer_side_gb300.distill import DistillLoss
    d = DistillLoss(4, 100, 3)
    z, ids, vals = torch.empty((0, 100), device="cuda"), torch.empty((0, 3), dtype=torch.int32, device="cuda"), \
        torch.empty((0, 3), device="cuda")
    loss, lse = d.forward(z, ids, vals)
    assert loss.shape == lse.shape == (0,)
    assert d.forward_backward(z, ids, vals, loss)[1].shape == (0, 100)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distill_rows_of_the_lowest_value(dtype):
    """Every logit at the type's lowest value: the student is uniform."""
    require_gpu()
    from mixture_experts_layer_side_gb300.distill import DistillLoss
    T, V, K = 3, 9000, 2
    z = torch.full((T, V), torch.finfo(TYPES[dtype]).min, dtype=TYPES[dtype])
    z[1, 100:] = -np.inf
    z[2, 3] = 0.0
    ids = torch.tensor([[0, 5], [7, 9], [3, -1]]).int()
    d = DistillLoss(T, V, K)
    loss, dz = d.forward_backward(z.cuda(), ids.cuda(), torch.zeros(T, K).cuda(), torch.ones(T).cuda())
    want = [np.log(V) + np.log(0.5), np.log(100) + np.log(0.5), 0.0]
    np.testing.assert_allclose(loss.cpu().numpy(), want, rtol=1e-5, atol=1e-6)
    q = torch.zeros((T, V), dtype=torch.float64)
    q[0], q[1, :100], q[2, 3] = 1 / V, 1 / 100, 1
    q[0, ids[0].long()] -= 0.5
    q[1, ids[1].long()] -= 0.5
    q[2, 3] -= 1
    assert (dz.double().cpu() - q).abs().max() <= (2.0 ** -8 if dtype == "bf16" else 1e-5) * 0.5
