"""RecurrentBlock.backward term by term against 64 bits: every element of each
gradient, each product at the inputs it got, with masks, carried states and
without the optional arguments; padding that holds NaN; weights that change;
other streams and graphs."""
import numpy as np
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from nonlinear_rnn_solve_newton_amd.binding import PararnnError
from nonlinear_rnn_solve_newton_amd.block import RecurrentBlock
from tests import layer_reference as R
from tests.helpers import say
from tests.test_gpu_block import inputs, make

pytestmark = pytest.mark.gpu

EPS = 1e-6


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, want, tol, what):
    """got (its own rounding included in the bound) within tol of want, element by element."""
    if got.dtype == torch.bfloat16:
        tol = tol + R.BF16_EPS * (np.abs(want) + tol)
    err = np.abs(f64(got) - want)
    assert (err <= tol + R.TINY).all(), f"{what}: {int((~(err <= tol + R.TINY)).sum())} of {err.size} outside"


def product(a, b):
    """a b of float64 arrays and its bound in fp32 sums of any order (one rounding per term at most)."""
    return a @ b, R.U * (a.shape[1] + 1) * (np.abs(a) @ np.abs(b))


def weights(blk):
    """Values of the block's 8-bit weights, exact in float64."""
    n = blk.G * blk.D
    full = layer.scale_values(blk.sw).repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :blk.E]
    return f64(blk.w8.float()) * f64(full)


def check_backward(blk, f, b, dh, ds=None, dstate=None, lengths=None, reset=None, state=None):
    """Gradients b of blk.forward's result f: the recurrence's from the gate inputs
    that the layer made, then the products and the norm's at the rounded values
    that they take (the recurrence's gradient and the norm's output, both bf16)."""
    opt = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    u, s = f["ctx"][0], f["s"]
    rec = R.gated(f64(u), f64(blk.coef), c=blk.c, h0=None if state is None else f64(state), lengths=opt(lengths),
                  reset=opt(reset), dh=f64(dh), dhT=None if dstate is None else f64(dstate))
    within(b["dcoef"], *rec["dlam"], "dcoef")
    within(b["dstate0"], *rec["dh0"], "dstate0")
    saved = f["ctx"][2]
    a = layer.gated_scan_adjoint(u, blk.coef, dh, saved, c=blk.c, dhT=dstate, lengths=lengths, reset=reset)
    within(a["du"], *rec["du"], "du")
    du = f64(a["du"]).reshape(-1, blk.G * blk.D)
    on = np.ones(s.shape[:2], bool) if lengths is None else np.arange(s.shape[1])[None] < opt(lengths)[:, None]
    on = on.reshape(-1)
    rows = f64(s).reshape(-1, blk.E)[on]
    y = f64(layer.norm_residual(s.reshape(-1, blk.E), blk.norm_w, eps=blk.eps)["y"])[on]
    within(b["dw"], *product(du[on].T, y), "dw")
    want = du[on].sum(0)
    within(b["dbias"], want, R.U * on.sum() * np.abs(du[on]).sum(0), "dbias")
    # dy: weights and the product rounded to bf16
    w = weights(blk)
    dy, e = product(du[on], w)
    e = e + R.BF16_EPS * (np.abs(du[on]) @ np.abs(w))
    e = e + R.BF16_EPS * (np.abs(dy) + e)
    nw = f64(blk.norm_w)
    dsr = None if ds is None else f64(ds).reshape(-1, blk.E)[on]
    n = R.norm_adjoint(rows, nw, dy, dsr, eps=blk.eps)
    rstd = 1.0 / np.sqrt((rows * rows).mean(1, keepdims=True) + blk.eps)
    nrm, ew = np.abs(rows * rstd), np.abs(nw) * e
    within(b["dx"].reshape(-1, blk.E)[torch.from_numpy(on).cuda()], n["dx"][0],
           n["dx"][1] + 1.01 * rstd * (ew + nrm * (ew * nrm).mean(1, keepdims=True)), "dx")
    within(b["dnorm_w"], n["dw"][0], n["dw"][1] + 1.01 * (e * nrm).sum(0), "dnorm_w")
    return on


@pytest.mark.parametrize("scale", [torch.float32, torch.float8_e8m0fnu])
@pytest.mark.parametrize("case", ["plain", "ds", "state", "masks"])
def test_every_gradient(case, scale):
    say(f"block backward: {case}, {scale}")
    B, L, E, D = 3, 150, 200, 72
    blk = make("gated", E, D, scale_dtype=scale)
    x, res = inputs(B, L, E)
    g = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    dh, ds, kw, state, dstate = n(B, L, D).bfloat16(), None, {}, None, None
    if case != "plain":
        ds = n(B, L, E).bfloat16()
    if case in ("state", "masks"):
        state, dstate = n(B, D), n(B, D)
    if case == "masks":
        kw = dict(lengths=torch.tensor([150, 97, 0], dtype=torch.int32).cuda(),
                  reset=(torch.rand(B, L, generator=g) < 0.05).cuda())
    f = blk.forward(x, res, state=state, train=True, **kw)
    b = blk.backward(f["ctx"], dh, ds, dstate)
    check_backward(blk, f, b, dh, ds, dstate, state=state, **kw)


def test_without_a_bias_or_a_residual():
    say("block backward without bias and residual")
    B, L, E, D = 2, 60, 136, 40
    full = make("gated", E, D)
    blk = RecurrentBlock("gated", full.norm_w, torch.randn(3 * D, E, generator=torch.Generator().manual_seed(3)).cuda(),
                         full.coef)
    x, _ = inputs(B, L, E)
    dh = torch.randn(B, L, D, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    f = blk.forward(x, train=True)
    check_backward(blk, f, blk.backward(f["ctx"], dh), dh)


@pytest.mark.parametrize("eps", [1e-6, 0.0])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_padding_may_hold_anything(bad, eps):
    """Steps past a row's length do not reach the weights' gradients, whatever x,
    the residual and dh hold there."""
    say(f"block backward, {bad} in the padding, eps {eps}")
    B, L, E, D = 3, 130, 128, 64
    blk = make("gated", E, D, eps=eps)
    x, res = inputs(B, L, E)
    g = torch.Generator().manual_seed(5)
    dh = torch.randn(B, L, D, generator=g).bfloat16().cuda()
    ds = torch.randn(B, L, E, generator=g).bfloat16().cuda()
    lengths = torch.tensor([130, 33, 0], dtype=torch.int32).cuda()
    on = torch.arange(L).cuda()[None] < lengths[:, None]

    def grads(fill):
        xx, rr, dd = (torch.where(on[:, :, None], t, torch.tensor(fill, dtype=t.dtype).cuda()) for t in (x, res, dh))
        f = blk.forward(xx, rr, lengths=lengths, train=True)
        return f, blk.backward(f["ctx"], dd, ds), dd

    f, got, dd = grads(bad)
    _, want, _ = grads(1.0)
    for k in ("dnorm_w", "dw", "dbias", "dcoef", "dstate0"):
        assert torch.isfinite(got[k]).all() and torch.equal(got[k], want[k]), k
    assert torch.equal(got["dx"][on], want["dx"][on])
    assert torch.equal(got["dx"][~on], ds[~on])  # s = x + residual there too, and nothing else uses it
    check_backward(blk, f, got, dd, ds, lengths=lengths)


def weights_of(seed, n, E):
    return torch.randn(n, E, generator=torch.Generator().manual_seed(seed)).cuda() / E ** 0.5


def test_gradients_follow_the_weights():
    """A training loop sets new 8-bit weights between its steps, in new tensors or
    in place: the next backward takes them."""
    say("block backward after an update of the weights")
    B, L, E, D = 2, 50, 200, 40
    x, res = inputs(B, L, E)
    dh = torch.randn(B, L, D, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    blk = make("gated", E, D)
    for k in range(3):
        if k == 1:
            blk.w8, blk.sw = layer.quantize_weight(weights_of(7, 3 * D, E), scale_dtype=blk.scale_dtype)
        if k == 2:
            w8, sw = layer.quantize_weight(weights_of(8, 3 * D, E), scale_dtype=blk.scale_dtype)
            blk.w8.copy_(w8)
            blk.sw.view(torch.uint8).copy_(sw.view(torch.uint8))
        f = blk.forward(x, res, train=True)
        check_backward(blk, f, blk.backward(f["ctx"], dh), dh)


# 32768 rows of 24 columns: the sum of dbias over many workgroups
@pytest.mark.parametrize("B,L,E,D", [(4, 1024, 256, 128), (16, 2048, 128, 8)])
def test_first_backward_in_a_graph(B, L, E, D):
    """A captured backward leaves nothing behind that an eager one before the
    first replay would read, and every replay gives the eager result."""
    say(f"block backward, captured first, {B}x{L}x{E}x{D}")
    blk, ref = make("gated", E, D), make("gated", E, D)
    x, res = inputs(B, L, E)
    dh = torch.randn(B, L, D, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()

    def step(b):
        f = b.forward(x, res, train=True)
        return b.backward(f["ctx"], dh)

    want = step(ref)  # also warms the libraries up
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(ref)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = step(blk)
    eager = step(blk)
    for k in want:
        assert torch.equal(eager[k], want[k]), f"eager before a replay: {k}"
    for i in range(4):
        for v in got.values():
            v.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(got[k], want[k]), f"replay {i}: {k}"
        step(ref)
        torch.cuda.synchronize()


def test_backward_on_two_streams():
    """The first backward on one stream, the next on another that knows nothing of it."""
    say("block backward on two streams")
    B, L, E, D = 2, 64, 256, 128
    blk, ref = make("gated", E, D), make("gated", E, D)
    x, res = inputs(B, L, E)
    dh = torch.randn(B, L, D, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    f = blk.forward(x, res, train=True)
    want = ref.backward(ref.forward(x, res, train=True)["ctx"], dh)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    out = []
    for s in streams:
        with torch.cuda.stream(s):
            out.append(blk.backward(f["ctx"], dh))
    torch.cuda.synchronize()
    for b in out:
        for k in want:
            assert torch.equal(b[k], want[k]), k
    assert not any(isinstance(v, torch.Tensor) and v.dtype == torch.bfloat16 for v in vars(blk).values())


def test_refused_shapes_and_types():
    """As many elements in another order are not the same rows, and a training
    pass is refused where its backward would be."""
    say("block: refused shapes")
    B, L, E, D = 3, 5, 128, 64
    blk = make("gated", E, D)
    x, res = inputs(B, L, E)
    f = blk.forward(x, res, train=True)
    dh = torch.zeros(B, L, D, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(4, D, device="cuda")
    bad = [
        lambda: blk.forward(x, res.transpose(0, 1).contiguous()),
        lambda: blk.forward(x, res.view(B * L, E)),
        lambda: blk.forward(x.view(B, 2 * L, E // 2), res.view(B, 2 * L, E // 2)),
        lambda: blk.forward(x.view(B * L, E)),
        lambda: blk.forward(x[0, 0]),
        lambda: blk.forward(x.cpu()),
        lambda: blk.forward(None),
        lambda: blk.forward(x, [1.0]),
        lambda: blk.forward(x.float(), res.float(), train=True),
        lambda: blk.step(x[:, 0].contiguous(), res[:, 0].t().contiguous(), pool),
        lambda: blk.step(x, res, pool),
        lambda: blk.backward(f["ctx"], dh, torch.zeros(L, B, E, dtype=torch.bfloat16, device="cuda")),
        lambda: blk.backward(f["ctx"], dh, torch.zeros(B * L, E, dtype=torch.bfloat16, device="cuda")),
        lambda: blk.backward(f["ctx"], dh, torch.zeros(B, L, E, device="cuda")),
        lambda: blk.backward(f["ctx"], dh.transpose(0, 1).contiguous()),
        lambda: blk.backward(blk.forward(x, res)["ctx"], dh),
    ]
    for i, c in enumerate(bad):
        with pytest.raises(PararnnError):
            c()
            raise AssertionError(f"refusal {i} did not come")
    # rows of any strides are taken, and fp32 rows without train
    t = torch.empty(L, B, E, dtype=torch.bfloat16, device="cuda").transpose(0, 1).copy_(res)
    assert torch.equal(blk.forward(x, t)["s"], f["s"])
    assert blk.forward(x.float(), res.float())["s"].dtype == torch.float32
