"""The parameters' gradients of norm_block over many rows, held to what their sums can be off by, which is less
than what a row, or a group of a row, brings to many of the columns: one that is left out fails.

A term is a product of the gradient that reaches it and of values of the row: the products, the sigmoid and the
row's norm are 64 roundings of the term, the gradient through the second norm 128 of its two terms
(`through_norm`). A thread adds at most rows / 512 of them, a workgroup its 16 rows, 32 threads each 32 partial rows
of every fold of groups, and one the 32 sums: the depth of a column's sum, in roundings of the sum of magnitudes."""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from tests import delta_reference as R
from tests.helpers import say
from tests.test_gpu_norm_block import DT, FWD, make, strided, through_norm, to

pytestmark = pytest.mark.gpu
U = R.U


def expected(w, s, group, dtype):
    """name -> (terms [rows][columns], error of each besides the sum) in 64 bits, at the sum s as it was written."""
    x, N = w["x"], w["x"].shape[0]
    G = group or x.shape[1]
    xg = x.view(N, -1, G)
    xh = (xg / (xg.square().mean(-1, keepdim=True) + 1e-6).sqrt()).reshape(x.shape)
    act = w["gate"] * w["gate"].sigmoid()
    wv = w["w"].repeat(x.shape[1] // G)
    out, dp, edp = {}, w["dy"], torch.zeros_like(x)
    if s is not None:
        rr = 1 / (s.square().mean(1, keepdim=True) + 1e-6).sqrt()
        t, rh = w["dy"] * w["w_next"], s * rr
        dr = rr * (t - rh * (t * rh).mean(1, keepdim=True)) + w["ds"]
        edr = 128 * U * (through_norm(s, t, None) + w["ds"].abs())
        out["dw_next"] = (w["dy"] * rh, 0.0 * rh)
        out["dalpha"] = (dr * xh * wv * act, edr * (xh * wv * act).abs())
        dp, edp = dr * w["alpha"], edr * w["alpha"].abs()
    terms, err = dp * act * xh, edp * (act * xh).abs()
    out["dw"] = (terms.view(-1, G), err.view(-1, G))  # a row of terms for every group
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,group,pre", [(3001, 1024, None, True), (3001, 1024, 128, False), (3001, 77, None, True),
                                           (1500, 4096, None, True), (700, 8192, None, True), (700, 8192, None, False),
                                           (700, 12000, None, True), (2999, 96, 32, True), (3001, 505, 101, False),
                                           (2000, 1024, 256, True)], ids=str)
def test_sums_over_rows(N, D, group, pre, dtype):
    say(f"norm_block sums {N} {D} {group} {dtype}")
    x = make(N, D, DT[dtype], group=group, pre=pre, seed=D)
    d, w = to(x, strided), to(x, lambda t: t.double())
    f = layer.norm_block(d["x"], **{n: d[n] for n in FWD})
    b = layer.norm_block_adjoint(d["x"], d["dy"], s=f["s"], ds=d["ds"], **{n: d[n] for n in FWD if n != "residual"})
    for n, (terms, err) in expected(w, f["s"].cpu().double() if pre else None, group, DT[dtype]).items():
        fold = D // group if n == "dw" and group and pre else 1  # groups beside each other are joined last
        depth = -(-terms.shape[0] // 512) + 16 + 32 * fold + 32
        bound = (depth + 64 + 1) * U * terms.abs().sum(0) + err.sum(0)
        got = b[n].cpu().double()
        assert ((got - terms.sum(0)).abs() <= bound).all(), (n, (got - terms.sum(0)).abs().max().item(), bound.max().item())
        # one column that is off fails: without the last row of memory, or without its last group, many would be
        groups = terms.shape[0] // N
        for lost in (terms[-groups:].sum(0), terms[-1]):
            assert (lost.abs() > 2 * bound).double().mean() > 0.15, n
