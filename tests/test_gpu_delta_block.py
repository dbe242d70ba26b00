"""The delta-rule layer end to end (block.DeltaBlock): norm, 8-bit projection,
delta rule, gated head norm and 8-bit output product against 64 bits on the
values that the layer rounds to; decoding against prefill; gradients; padding."""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from nonlinear_rnn_solve_newton_amd.binding import PararnnError
from nonlinear_rnn_solve_newton_amd.block import DeltaBlock
from tests import delta_reference as R
from tests.helpers import say

pytestmark = pytest.mark.gpu


def make(E, H, HV, dk, dv, seed=0, alpha=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    cols = 2 * H * dk + 2 * HV * dv + 2 * HV
    return DeltaBlock(1 + 0.1 * rnd(E), rnd(cols, E) / E ** 0.5, rnd(HV) - 3.0, 1 + 0.1 * rnd(dv),
                      rnd(E, HV * dv) / (HV * dv) ** 0.5, heads=H, dk=dk, alpha=1 + 0.1 * rnd(E) if alpha else None)


def inputs(B, L, E, seed=1):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, L, E, generator=g).bfloat16().cuda(), 2 * torch.randn(B, L, E, generator=g).bfloat16().cuda())


def through(x, to):
    """The value `to` with the gradient of x."""
    return x + (to.double() - x).detach()


def reference(blk, x, residual, f, lengths=None, reset=None, state=None):
    """The layer in 64 bits at the values that its parts rounded to, gradients straight
    through the roundings. Returns the result, the sum and the leaves."""
    B, L, E = x.shape
    dbl = lambda t: t.detach().double().cpu()  # noqa: E731
    leaf = lambda t: dbl(t).requires_grad_()  # noqa: E731
    w, wo = dbl(blk.w8) * dbl(blk.sw)[:, None], dbl(blk.wo8) * dbl(blk.swo)[:, None]
    ls = dict(x=leaf(x), residual=None if residual is None else leaf(residual), norm_w=leaf(blk.norm_w),
              alpha=None if blk.alpha is None else leaf(blk.alpha), w=w.requires_grad_(), lam=leaf(blk.lam),
              head_w=leaf(blk.head_w), w_out=wo.requires_grad_(),
              state0=torch.zeros(B, blk.HV, blk.dk, blk.dv, dtype=torch.float64).requires_grad_() if state is None else leaf(state))
    rows = ls["x"].view(-1, E)
    if residual is None:
        y, s = R.norm_block(rows, w=ls["norm_w"], eps=blk.eps)[0], rows
    else:
        s = ls["residual"].view(-1, E) + (rows if ls["alpha"] is None else ls["alpha"] * rows)
        s = through(s, dbl(f["s"]).view(-1, E))
        y = R.norm_block(s, w=ls["norm_w"], eps=blk.eps)[0]
    p = through(y @ ls["w"].t(), dbl(f["ctx"][3]))
    q, k, v, z, g = p.split(blk.cols, dim=-1)
    o, sT = R.delta(q.reshape(B, L, blk.H, blk.dk), k.reshape(B, L, blk.H, blk.dk), v.reshape(B, L, blk.HV, blk.dv),
                    g.reshape(B, L, 2, blk.HV), ls["lam"], c=blk.c, eps=blk.eps, s0=ls["state0"],
                    lengths=None if lengths is None else lengths.cpu(), reset=None if reset is None else reset.cpu())
    o = through(o, dbl(f["ctx"][4]))
    h = R.norm_block(o.reshape(B * L, -1), w=ls["head_w"], gate=z, group=blk.dv, eps=blk.eps)[0]
    return (h @ ls["w_out"].t()).view(B, L, E), s.view(B, L, E), sT, ls


def within(name, got, want, steps):
    """In norm: `steps` roundings to bf16, each 2^-8 of its value at most."""
    err = (got.double().cpu() - want).norm() / want.norm()
    assert err <= steps * 2.0 ** -8, (name, err.item())


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("sizes", [(256, 2, 4, 64, 64), (200, 1, 3, 40, 32), (128, 1, 1, 128, 128)], ids=str)
def test_forward_and_gradients(sizes, residual):
    say(f"delta block {sizes}")
    E, H, HV, dk, dv = sizes
    B, L = 2, 130
    blk = make(*sizes, alpha=residual)
    x, res = inputs(B, L, E)
    g = torch.Generator().manual_seed(7)
    state = (0.2 * torch.randn(B, HV, dk, dv, generator=g)).cuda()
    f = blk.forward(x, res if residual else None, state=state, train=True)
    plain = blk.forward(x, res if residual else None, state=state)
    assert torch.equal(plain["x"], f["x"]) and torch.equal(plain["s"], f["s"]) and plain["ctx"] is None
    y, s, sT, ls = reference(blk, x, res if residual else None, f, state=state)
    # the 8-bit rows in front of the output product: half of 1/127 of a row's largest value, which is at most
    # sqrt(columns) times its root mean square, in each of the sum's terms, of random sign: in norm at most
    # half of 1/127 times the largest over the root mean square (under 16 of them here)
    within("x", f["x"], y.detach(), 16)
    assert ((f["state"].double().cpu() - sT.detach()).abs() <= 8 * R.U * (dk + dv + 64 + L) * sT.abs().max()).all()
    dx, ds = inputs(B, L, E, seed=5)
    dst = (0.3 * torch.randn(B, HV, dk, dv, generator=g)).cuda()
    b = blk.backward(f["ctx"], dx, ds=ds, dstate=dst)
    loss = (y * dx.double().cpu()).sum() + (s * ds.double().cpu()).sum() + (sT * dst.double().cpu()).sum()
    names = [n for n, t in ls.items() if t is not None]
    for n, w in zip(names, torch.autograd.grad(loss, [ls[n] for n in names])):
        within("d" + n, b["d" + n], w, 8)  # no more than 8 tensors in bf16 between the loss and a gradient
    if not residual:
        assert b["dresidual"] is None and b["dalpha"] is None


def test_prefill_then_decode_is_the_whole_sequence():
    say("delta block: prefill and decode")
    B, L, T, E = 3, 70, 5, 256
    blk = make(E, 2, 4, 64, 64)
    x, res = inputs(B, L + T, E)
    whole = blk.forward(x, res)
    pre = blk.forward(x[:, :L], res[:, :L])
    pool = torch.zeros(8, 4, 64, 64, device="cuda")
    slots = torch.tensor([5, 2, 7], dtype=torch.int32, device="cuda")
    pool[slots.long()] = pre["state"]
    for t in range(L, L + T):
        y, s = blk.step(x[:, t].contiguous(), res[:, t].contiguous(), pool, slots=slots)
        assert torch.equal(s, whole["s"][:, t])
        # the same projections bit for bit (integer sums); o differs by a rounding to bf16 here and there, and
        # its 8-bit row by a step: at most one of 127 of a row's largest value
        within("x", y, whole["x"][:, t].double().cpu(), 8)
    want = whole["state"]
    assert ((pool[slots.long()] - want).abs() <= 2 * 8 * R.U * (64 + 64 + 64 + L + T) * want.abs().max()).all()
    assert not pool[[0, 1, 3, 4, 6]].any()


def test_padding_reaches_nothing():
    """Whatever lies past the lengths: the other rows' results and the weights' gradients
    are those of clean padding, bit for bit."""
    say("delta block: padding")
    B, L, E = 4, 100, 128
    blk = make(E, 1, 2, 32, 32)
    lengths = torch.tensor([100, 37, 0, 1], dtype=torch.int32, device="cuda")
    reset = torch.zeros(B, L, dtype=torch.uint8, device="cuda")
    reset[0, 64] = 1
    live = torch.arange(L, device="cuda") < lengths[:, None]
    outs = []
    for junk in (0.0, float("nan"), float("inf")):
        x, res = inputs(B, L, E)
        dx, ds = inputs(B, L, E, seed=3)
        for t in (x, res, dx, ds):
            t[~live] = junk
        f = blk.forward(x, res, lengths=lengths, reset=reset, train=True)
        b = blk.backward(f["ctx"], dx, ds=ds)
        outs.append((f["x"][live], f["state"], b))
    for x, state, b in outs[1:]:
        assert torch.equal(x, outs[0][0]) and torch.equal(state, outs[0][1])
        for n, t in b.items():
            assert torch.isfinite(t).all() and torch.equal(t, outs[0][2][n]), n


def test_one_training_step_in_a_graph():
    say("delta block: graph")
    blk = make(128, 1, 2, 32, 32)
    x, res = inputs(2, 90, 128)
    dx, ds = inputs(2, 90, 128, seed=9)

    def run():
        f = blk.forward(x, res, train=True)
        return {"y": f["x"], **blk.backward(f["ctx"], dx, ds=ds)}

    run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = run()
    for seed in (2, 4, 6):
        for t, v in zip((x, res, dx, ds), (*inputs(2, 90, 128, seed=seed), *inputs(2, 90, 128, seed=seed + 1))):
            t.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        eager = run()
        assert all(torch.equal(r[n], eager[n]) for n in eager), seed


def test_new_weights_are_seen():
    say("delta block: new weights")
    blk = make(128, 1, 1, 32, 32)
    x, res = inputs(1, 20, 128)
    a = blk.forward(x, res)["x"].clone()
    blk.w8, blk.sw = layer.quantize_weight_int8(torch.randn(sum(blk.cols), 128, device="cuda") / 11)
    assert not torch.equal(blk.forward(x, res)["x"], a)


def test_refusals():
    say("delta block: refusals")
    blk = make(128, 1, 2, 32, 32)
    x, res = inputs(2, 10, 128)
    for a in ((x[0], None), (x[..., :64], None), (None, None), (x, res[:1]), (x, res[..., :64])):
        with pytest.raises(PararnnError):
            blk.forward(*a)
    with pytest.raises(PararnnError):
        blk.forward(x.float(), res.float(), train=True)
    assert blk.forward(x.float(), res.float())["s"].dtype == torch.float32
    f = blk.forward(x, res, train=True)
    for dx, kw in ((x[:1], {}), (None, {}), (x, dict(ds=res[:, :5])), (x, dict(dstate=torch.zeros(2, 2, 32, 31, device="cuda")))):
        with pytest.raises(PararnnError):
            blk.backward(f["ctx"], dx, **kw)
    with pytest.raises(PararnnError):
        blk.backward(None, x)
    pool = torch.zeros(2, 2, 32, 32, device="cuda")
    for a in ((x, res, pool), (x[:, 0], res[:, 0], pool[:1]), (x[:, 0], res[:1, 0], pool)):
        with pytest.raises(PararnnError):
            blk.step(*a)
