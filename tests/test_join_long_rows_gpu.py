"""The residual join on rows of any alignment that take a CTA each, several
rows one after the other for every team: more than the rows that lie ahead in
shared memory, so that each of their places is filled again."""

import pytest
import torch

import test_residual_gpu as cases
from _helpers import require_gpu

pytestmark = pytest.mark.gpu

NAMES = ("dx", "dy", "dw_out", "dgate", "dw_next")


def roundings(T, H):
    """Of a column's sum: the rows of the least workers that take these sizes (one CTA an SM) one after the other, 16
    threads' parts and the terms' own.  (The bounds of the formulas' tests count 32 such rows.)"""
    return cases.U_COL + max(0, -(-T // 152) - 32) * 2.0 ** -24


@pytest.mark.parametrize("types", ["bf16", "mixed", "f32"])
@pytest.mark.parametrize("T,H,groups,p,pad", [(8000, 515, 1, 0.0, 3), (8000, 515, 8000, 0.125, 0), (6000, 1003, 12, 0.125, 1),
                                              (6000, 1003, 1, 0.125, 6), (6000, 1003, 6000, 0.0, 5), (2000, 4099, 1, 0.0, 0),
                                              (2000, 4099, 500, 0.25, 2), (1000, 9001, 0, 0.125, 3), (1000, 9001, 1000, 0.0, 1),
                                              (1600, 2043, 4, 0.0, 7)])
def test_places_are_filled_again(T, H, groups, p, pad, types):
    require_gpu()
    from mixture_experts_layer_side_gb300.dropout import MoKDropout
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    s = cases.inputs(T, H, types, True, groups, True, pad)
    drop = MoKDropout(p, seed=(3 << 40) + 77) if p else None
    res = MoKResidual(H, T)
    kw = dict(w_out=s["w_out"], gate=s["gate"], w_next=s["w_next"], scale=0.5, dropout=drop, call=5)
    r, e = cases.reference(s, T, H, 0.5, drop)
    for k in ("dw_out", "dgate", "dw_next"):
        if k in e:
            e[k] = e[k] * (roundings(T, H) / cases.U_COL)
    forward = res.forward(s["x"], s["y"], **kw)
    cases.compare(forward, r, e, ("x", "n"))
    got = res.backward(s["dx"], s["dn"], s["x"], s["y"], **kw)
    cases.compare([got[k] for k in NAMES], r, e, NAMES)
    # the same bits again, and in place
    x, y = s["x"].clone(), s["y"].clone()
    for a, b in zip(forward, res.forward(x, y, **kw, out=x, out_next=y)):
        assert torch.equal(a, b)
    dx, dn = s["dx"].clone(), s["dn"].clone()
    place = res.backward(dx, dn, s["x"], s["y"], **kw, dx=dx, dy=dn)
    assert all(torch.equal(got[k], place[k]) for k in NAMES if got[k] is not None)


@pytest.mark.parametrize("types", ["bf16", "f32"])
def test_norm_alone_of_many_long_rows(types):
    require_gpu()
    from mixture_experts_layer_side_gb300.residual import MoKResidual
    for T, H, pad in ((6000, 1003, 1), (2000, 4099, 3)):
        s = cases.inputs(T, H, types, False, 0, True, pad)
        res = MoKResidual(H, T)
        r, e = cases.reference(dict(s, y=s["y"] * 0), T, H, 1.0, None)
        e["dw_next"] = e["dw_next"] * (roundings(T, H) / cases.U_COL)
        cases.compare([res.norm(s["x"], s["w_next"])], r, e, ("n",))
        cases.compare(res.norm_backward(s["dn"], s["x"], s["w_next"], dx_new=s["dx"]), r, e, ("dx", "dw_next"))
