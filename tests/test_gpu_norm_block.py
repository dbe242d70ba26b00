"""The norms around a block (layer.norm_block and its adjoint) against 64 bits:
whole rows and groups, odd widths and strides, 8-bit rows, every choice of
inputs, parameters' gradients over many rows, NaN and infinities, graphs.

A 32-bit value of a row collects at most 24 roundings (two norms, the gate's
sigmoid, products), sums over D or a group another log2(16384) + 8 as they are
summed in a tree of 8 per lane; gradients twice that: 64 and 128 U of the row's
largest value, before the rounding to the type. The gradient through a norm is a
difference, rstd (u - xh mean(u xh)), which may vanish (with one column it does
but for eps): its rounding goes by its two terms, of which the second is at most
rstd max|xh| sqrt(mean(u^2)), since mean(xh^2) <= 1 (`through_norm`). Sums over rows add one rounding
per row that a thread takes and log2 for the rest: at most N U of the sum of
magnitudes."""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from nonlinear_rnn_solve_newton_amd.binding import PararnnError
from tests import delta_reference as R
from tests.helpers import say

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = R.U


def make(N, D, dtype, group=None, seed=0, gate=True, w=True, pre=True, alpha=True, stride=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    rows = lambda k=1.0: (k * rnd(N, D + stride)).to(dtype)[:, :D]  # noqa: E731
    return dict(x=rows(), gate=rows() if gate else None, w=1 + 0.2 * rnd(group or D) if w else None, group=group,
                residual=rows(3.0) if pre else None, alpha=0.1 + 0.5 * rnd(D) if pre and alpha else None,
                w_next=1 + 0.2 * rnd(D) if pre else None, dy=rnd(N, D).to(dtype), ds=rnd(N, D).to(dtype) if pre else None)


def to(x, f):
    return {n: f(t) if isinstance(t, torch.Tensor) else t for n, t in x.items()}


def strided(t):
    """On the device, with the CPU tensor's row stride."""
    if t.dim() == 2 and t.stride(0) != t.shape[1]:
        b = torch.zeros(t.shape[0], t.stride(0), dtype=t.dtype, device="cuda")
        b[:, :t.shape[1]] = t.cuda()
        return b[:, :t.shape[1]]
    return t.cuda()


FWD = ("w", "gate", "group", "residual", "alpha", "w_next")


def near(name, got, want, dtype, bound):
    """Against 64 bits: `bound` (per element) before the rounding to dtype, or nothing where
    fp32 holds nothing that small (s(-200) = 1e-87, say)."""
    bound = bound + R.TINY
    err = (got.cpu().double() - want).abs()
    assert (err <= bound + R.half_step(dtype) * (want.abs() + bound)).all(), (name, err.max().item())


def rowmax(t):
    return t.abs().amax(1, keepdim=True)


def through_norm(x, u, group):
    """The largest terms of the gradient of x / sqrt(mean(x^2) + eps) for the gradient u of
    the quotient, per group, spread over its columns."""
    N, D = x.shape
    x, u = x.view(N, -1, group or D), u.reshape(N, -1, group or D)
    rstd = 1 / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    big = lambda t: t.abs().amax(-1, keepdim=True)  # noqa: E731
    return (rstd * (big(u) + big(x * rstd) * u.square().mean(-1, keepdim=True).sqrt())).expand(x.shape).reshape(N, D)


def check(x, dtype):
    d, w = to(x, strided), to(x, lambda t: t.double())
    f = layer.norm_block(d["x"], **{n: d[n] for n in FWD})
    leaves = {n: w[n].clone().requires_grad_() for n in ("x", "gate", "residual", "w", "alpha", "w_next") if w[n] is not None}
    y, s = R.norm_block(leaves["x"], **{n: leaves.get(n, x["group"] if n == "group" else None) for n in FWD})
    near("y", f["y"], y.detach(), dtype, 64 * U * rowmax(y.detach()))
    pre = s is not None
    if pre:
        near("s", f["s"], s.detach(), dtype, 64 * U * rowmax(s.detach()))
    else:
        assert f["s"] is None and f["scale"] is None
    b = layer.norm_block_adjoint(d["x"], d["dy"], s=f["s"], ds=d["ds"], **{n: d[n] for n in FWD if n != "residual"})
    if pre:
        # the adjoint takes the sum as it was written
        sr = f["s"].cpu().double().requires_grad_()
        y = sr / (sr.square().mean(1, keepdim=True) + 1e-6).sqrt() * leaves["w_next"]
        (g_s, g_wn) = torch.autograd.grad((y * w["dy"]).sum(), (sr, leaves["w_next"]))
        g_s = g_s + w["ds"]
        terms = through_norm(sr.detach(), w["dy"] * w["w_next"], None) + w["ds"].abs()
        near("dresidual", b["dresidual"], g_s, dtype, 128 * U * terms)
        rest = [leaves[n] for n in ("x", "gate", "w", "alpha") if n in leaves]
        names = [n for n in ("x", "gate", "w", "alpha") if n in leaves]
        g = dict(zip(names, torch.autograd.grad((s * g_s).sum(), rest)))
        mags = (w["dy"] * sr.detach() / (sr.detach().square().mean(1, keepdim=True) + 1e-6).sqrt()).abs().sum(0)
        near("dw_next", b["dw_next"], g_wn, torch.float64, (x["x"].shape[0] + 128) * U * mags)
    else:
        names = [n for n in ("x", "gate", "w") if n in leaves]
        g = dict(zip(names, torch.autograd.grad((y * w["dy"]).sum(), [leaves[n] for n in names])))
        assert b["dresidual"] is None and b["dw_next"] is None and b["dalpha"] is None
    # the gradient of p, its bound, and what they become
    gp, ep = (w["dy"], 0.0) if not pre else (g_s, 128 * U * terms)
    if pre and w["alpha"] is not None:
        gp, ep = w["alpha"] * gp, w["alpha"].abs() * ep
    z = w["gate"]
    act = torch.ones_like(gp) if z is None else z * z.sigmoid()
    xh = w["x"]
    if w["w"] is not None:
        gr = xh.view(xh.shape[0], -1, x["group"] or xh.shape[1])
        xh = (gr / (gr.square().mean(-1, keepdim=True) + 1e-6).sqrt()).view(xh.shape)
    wv = 1.0 if w["w"] is None else w["w"].repeat(xh.shape[1] // w["w"].numel())
    u, eu = gp * act * wv, ep * act.abs() * (wv if isinstance(wv, float) else wv.abs())
    if w["w"] is None:
        near("dx", b["dx"], g["x"], dtype, 256 * U * u.abs() + eu)
    else:
        near("dx", b["dx"], g["x"], dtype, 256 * U * through_norm(w["x"], u, x["group"]) +
             (through_norm(w["x"], eu, x["group"]) if pre else 0.0))
    if z is not None:
        dact = z.sigmoid() * (1 + z * (1 - z.sigmoid()))
        big = (xh * wv * (z.sigmoid() + (z * z.sigmoid() * (1 - z.sigmoid())).abs())).abs()
        near("dgate", b["dgate"], g["gate"], dtype, 256 * U * gp.abs() * big + ep * (xh * wv * dact).abs())
    else:
        assert b["dgate"] is None
    for n in ("w", "alpha"):
        if n in g:
            # magnitudes of the terms: at most each gradient's largest over the rows
            N = x["x"].shape[0] * (x["x"].shape[1] // g[n].numel())
            big = g_s.abs().max() * 40 if pre else w["dy"].abs().max() * 40
            near("d" + n, b["d" + n], g[n], torch.float64, (N + 256) * U * big * N ** 0.5)
        else:
            assert b["d" + n] is None


WIDTHS = [1, 7, 8, 100, 128, 129, 256, 500, 1000, 1025, 2048, 4096, 8192, 12000, 16384]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_whole_rows(D, dtype):
    say(f"norm_block {D} {dtype}")
    check(make(7, D, DT[dtype], seed=D), DT[dtype])
    check(make(3, D, DT[dtype], seed=D, pre=False), DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,group,pre", [(96, 32, True), (1024, 128, True), (2048, 512, True), (64, 8, True), (96, 32, False),
                                         (1024, 128, False), (505, 101, False), (600, 3, False), (360, 72, False),
                                         (5, 1, False), (4096, 2048, False)])
def test_groups(D, group, pre, dtype):
    say(f"norm_block groups {D} {group} {dtype}")
    check(make(9, D, DT[dtype], group=group, pre=pre, seed=group), DT[dtype])


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("w", [True, False])
@pytest.mark.parametrize("alpha", [True, False])
def test_choices(gate, w, alpha):
    say("norm_block choices")
    check(make(5, 200, torch.bfloat16, gate=gate, w=w, alpha=alpha), torch.bfloat16)


@pytest.mark.parametrize("stride", [1, 8, 24])
def test_rows_that_lie_apart(stride):
    say(f"norm_block stride {stride}")
    for group, pre in ((None, True), (32, True), (32, False), (None, False)):
        check(make(6, 256, torch.bfloat16, group=group, pre=pre, stride=stride), torch.bfloat16)


@pytest.mark.parametrize("D,group", [(1024, None), (1024, 128), (77, None)])
def test_many_rows(D, group):
    say("norm_block many rows")
    check(make(3001, D, torch.float32, group=group, pre=group is None), torch.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,group,pre", [(8, None, True), (100, None, True), (1000, None, False), (4096, None, True),
                                         (1024, 128, False), (256, 64, True), (129, None, False), (9000, None, True)])
def test_eight_bits(D, group, pre, dtype):
    """scale = max(max|y|, 2^-100) / 127 of the 32-bit y, q = round(y / scale): the
    scale to the bound of y, q to half a step of it."""
    say(f"norm_block int8 {D} {dtype}")
    x = make(11, D, DT[dtype], group=group, pre=pre, seed=D)
    if not pre:
        x["x"][3] = 0.0
    d, w = to(x, strided), to(x, lambda t: t.double())
    f = layer.norm_block(d["x"], out_dtype=torch.int8, **{n: d[n] for n in FWD})
    y, _ = R.norm_block(w["x"], **{n: w[n] for n in FWD})
    scale = y.abs().amax(1).clamp_min(2.0 ** -100) / 127
    got = f["scale"].cpu().double()
    assert f["y"].dtype == torch.int8 and ((got - scale).abs() <= 66 * U * scale).all()
    q = f["y"].cpu().double()
    assert q.abs().max() <= 127 and ((q * got[:, None] - y).abs() <= got[:, None] * (0.5 + 127 * 66 * U)).all()
    same = layer.norm_block(d["x"], **{n: d[n] for n in FWD})
    if pre:
        assert torch.equal(f["s"], same["s"])


def test_values_that_are_no_numbers_stay_in_their_row():
    say("norm_block NaN")
    x = to(make(6, 300, torch.float32), lambda t: t.cuda())
    clean = layer.norm_block(x["x"], **{n: x[n] for n in FWD})
    x["x"][1, 5], x["residual"][2, 7], x["gate"][3, 9] = float("nan"), float("inf"), float("nan")
    for dt in (None, torch.int8):
        f = layer.norm_block(x["x"], out_dtype=dt, **{n: x[n] for n in FWD})
        if dt is None:
            assert f["y"][1:4].isnan().any(1).all()
            assert torch.equal(f["y"][[0, 4, 5]], clean["y"][[0, 4, 5]])
        else:
            assert not torch.isfinite(f["scale"][1:4]).any() and torch.isfinite(f["scale"][[0, 4, 5]]).all()
    b = layer.norm_block_adjoint(x["x"], x["dy"], s=f["s"], ds=x["ds"], **{n: x[n] for n in FWD if n != "residual"})
    assert torch.isfinite(b["dx"][[0, 4, 5]]).all() and torch.isfinite(b["dgate"][[0, 4, 5]]).all()


def test_zeros_and_extremes():
    say("norm_block extremes")
    for k in (0.0, 1e-20, 1e15):
        x = make(4, 64, torch.float32)
        x["x"] = x["x"] * k
        d, w = to(x, lambda t: t.cuda()), to(x, lambda t: t.double())
        f = layer.norm_block(d["x"], **{n: d[n] for n in FWD})
        y, s = R.norm_block(w["x"], **{n: w[n] for n in FWD})
        near("y", f["y"], y, torch.float32, 64 * U * rowmax(y))
    x["gate"][:] = 200.0
    x["gate"][1] = -200.0
    check(x, torch.float32)


def test_a_replayed_graph_and_another_stream():
    say("norm_block graph")
    x = to(make(300, 256, torch.bfloat16), lambda t: t.cuda())

    def run():
        f = layer.norm_block(x["x"], **{n: x[n] for n in FWD})
        b = layer.norm_block_adjoint(x["x"], x["dy"], s=f["s"], ds=x["ds"], **{n: x[n] for n in FWD if n != "residual"})
        i = layer.norm_block(x["x"], out_dtype=torch.int8, **{n: x[n] for n in FWD})
        return {"y": f["y"], "q": i["y"], "scale": i["scale"], **{n: t for n, t in b.items() if n != "ws"}}

    want, side = run(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(got[n], want[n]) for n in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = run()
    for seed in (1, 2, 3):
        y = make(300, 256, torch.bfloat16, seed=seed)
        for n, t in x.items():
            if isinstance(t, torch.Tensor):
                t.copy_(y[n])
        g.replay()
        torch.cuda.synchronize()
        eager = run()
        assert all(torch.equal(r[n], eager[n]) for n in eager), seed


def test_refusals():
    say("norm_block refusals")
    x = to(make(4, 96, torch.bfloat16), lambda t: t.cuda())
    base = {n: x[n] for n in FWD}
    bad = [dict(gate=x["gate"].float()), dict(gate=x["gate"][:3]), dict(gate=x["gate"].cpu()), dict(w=x["w"][:95]),
           dict(w=x["w"].double()), dict(group=0), dict(group=97), dict(group=1.5), dict(w=x["w"][:24], group=24),
           dict(w_next=None), dict(alpha=x["alpha"][None]), dict(residual=None), dict(residual=x["residual"].t()),
           dict(residual=x["residual"][:1].expand(4, 96)), dict(out_dtype=torch.float16), dict(eps=-1.0),
           dict(residual=None, alpha=None, w_next=None, w=None)]
    for kw in bad:
        with pytest.raises(PararnnError):
            layer.norm_block(x["x"], **{**base, **kw})
    for t in (None, x["x"][0], x["x"].half(), x["x"][:0], x["x"].t(), torch.zeros(1, 16385, device="cuda")):
        with pytest.raises(PararnnError):
            layer.norm_block(t, w=torch.ones(16385, device="cuda"))
    f = layer.norm_block(x["x"], **base)
    base.pop("residual")
    for kw in (dict(s=f["s"][:3]), dict(s=None), dict(ds=x["ds"].float()), dict(w_next=None),
               dict(ws=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        a = {**base, "s": f["s"], "ds": x["ds"], **kw}
        with pytest.raises(PararnnError):
            layer.norm_block_adjoint(x["x"], x["dy"], **a)
    for dy in (None, x["dy"].float(), x["dy"][:3]):
        with pytest.raises(PararnnError):
            layer.norm_block_adjoint(x["x"], dy, s=f["s"], **base)
    b = layer.norm_block_adjoint(x["x"], x["dy"], s=f["s"], want_params=False, **base)
    assert b["dw"] is None and b["dalpha"] is None and b["dw_next"] is None and b["dx"] is not None
