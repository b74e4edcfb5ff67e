"""The residual join where values are not finite: gradients of no rows beside
weights that are not, and dropped elements of rows whose norm is not."""

import pytest
import torch

import test_residual_gpu as cases
from _helpers import require_gpu

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("types", ["bf16", "mixed", "f32"])
@pytest.mark.parametrize("H", [64, 67, 9000])
def test_no_rows_give_zeros_whatever_the_weights(types, H):
    require_gpu()
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    s = cases.inputs(0, H, types, True, 1, True)
    s["gate"][0, 1], s["gate"][0, 5], s["w_out"][2], s["w_out"][7], s["w_next"][3] = INF, NAN, -INF, NAN, INF
    res = MoKResidual(H, 4)
    # (what the allocator hands out next is not zero)
    junk = [torch.full((H,), NAN, device="cuda") for _ in range(8)]
    del junk
    got = res.backward(s["dx"], s["dn"], s["x"], s["y"], s["w_out"], s["gate"], s["w_next"])
    for k in ("dw_out", "dgate", "dw_next"):
        assert torch.equal(got[k], torch.zeros_like(got[k])), k
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = res.backward(s["dx"], s["dn"], s["x"], s["y"], s["w_out"], s["gate"], s["w_next"])
    for k in ("dw_out", "dgate", "dw_next"):
        held[k].fill_(NAN)
    graph.replay()
    assert not any(held[k].any() for k in ("dw_out", "dgate", "dw_next"))


@pytest.mark.parametrize("types", ["bf16", "mixed", "f32"])
@pytest.mark.parametrize("H", [96, 97, 2048, 9000])
def test_dropped_elements_of_a_bad_row_keep_the_stream(types, H):
    """x' = x + scale gate dropout(z) with a dropped element of z 0 whatever it is: a row whose norm is NaN, and a
    column whose weight is infinite, leave x as it is where z is dropped."""
    require_gpu()
    from mixture_experts_layer_side_gb300.dropout import MoKDropout
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    T = 33
    s = cases.inputs(T, H, types, True, 3, True)
    s["y"][5, 2], s["y"][9, 1], s["w_out"][4] = NAN, INF, INF
    drop, res = MoKDropout(0.5, seed=4), MoKResidual(H, T)
    x = res.forward(s["x"], s["y"], s["w_out"], s["gate"], s["w_next"], dropout=drop)[0]
    off = torch.from_numpy(~cases.kept(T, H, 0.5, 4, 0)).cuda()
    assert torch.equal(x[off], s["x"][off])
    # kept, they are what the formula makes of them: NaN all over a row without a norm, and where infinity meets 0
    assert torch.isnan(x[5][~off[5]]).all() and bool(torch.isfinite(x[9, 2:4]).all())
    assert bool(torch.isfinite(x[:, :4][[i for i in range(T) if i not in (5, 9)]]).all())
