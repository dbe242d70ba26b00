"""The gated delta rule on the GPU (layer.delta_scan, its adjoint, delta_step)
against the 64-bit step-by-step form: lengths from one step to several chunks,
head layouts, odd sizes, views, padding with NaN in it, document starts, keys
and gates at their limits, carried states, streams, graphs and pools."""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from nonlinear_rnn_solve_newton_amd.binding import PararnnError
from tests import delta_reference as R
from tests.helpers import say

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
GRADS = ("dq", "dk", "dv", "dgates", "dlam", "ds0")


def make(B, L, H, HV, dk, dv, dtype, seed=0, views=False, packed=False, lam=None):
    """A dict of CPU tensors in `dtype` (states and lam fp32)."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    sizes = (H * dk, H * dk, HV * dv, 2 * HV)
    p = rnd(B, L, sum(sizes)).to(dtype)
    q, k, v, gates = p.split(sizes, dim=-1)
    if not views:
        q, k, v, gates = (t.contiguous() for t in (q, k, v, gates))
    x = dict(q=q.unflatten(-1, (H, dk)), k=k.unflatten(-1, (H, dk)), v=v.unflatten(-1, (HV, dv)),
             gates=gates.unflatten(-1, (2, HV)), lam=rnd(HV) - 3.0 if lam is None else torch.full((HV,), lam),
             s0=0.3 * rnd(B, HV, dk, dv), do=rnd(B, L, HV, dv).to(dtype), dsT=0.3 * rnd(B, HV, dk, dv),
             lengths=None, reset=None, p=p)
    if packed:
        n = torch.randint(0, L + 1, (B,), generator=g, dtype=torch.int32)
        n[0] = L
        if B > 2:
            n[1], n[2] = 0, 1
        x["lengths"] = n
        x["reset"] = (torch.rand(B, L, generator=g) < 0.1).to(torch.uint8)
        x["reset"][:, min(64, L - 1)] = 1  # the first step of a chunk
    return x


def cuda(x):
    """On the device; views stay views of one buffer."""
    out = {n: None if t is None else t.cuda() for n, t in x.items()}
    if not x["q"].is_contiguous():
        p, at = x["p"].cuda(), 0
        for n in ("q", "k", "v", "gates"):
            w = x[n].shape[-1] * x[n].shape[-2]
            out[n] = p[..., at:at + w].unflatten(-1, x[n].shape[-2:])
            at += w
    return out


def run(d, s0=True, dsT=True, **kw):
    args = (d["q"], d["k"], d["v"], d["gates"], d["lam"])
    opt = dict(lengths=d["lengths"], reset=d["reset"], **kw)
    f = layer.delta_scan(*args, s0=d["s0"] if s0 else None, save=True, **opt)
    b = layer.delta_scan_adjoint(*args, d["do"], f["saved"], dsT=d["dsT"] if dsT else None, want_ds0=True, **opt)
    return {"o": f["o"], "sT": f["sT"], **{n: b[n] for n in GRADS}}


def reference(x, s0=True, dsT=True, **kw):
    w = {n: None if t is None else t.double() if t.is_floating_point() else t for n, t in x.items()}
    return R.delta_grads(w["q"], w["k"], w["v"], w["gates"], w["lam"], w["do"], dsT=w["dsT"] if dsT else None,
                         s0=w["s0"] if s0 else None, lengths=w["lengths"], reset=w["reset"], **kw)


def check(got, want, dtype, dk, dv, steps):
    for n, w in want.items():
        if n not in got:
            continue
        t = got[n].cpu()
        assert t.dtype == (torch.float32 if n in ("sT", "dlam", "ds0") else dtype), n
        atol, rtol = R.delta_tol(n, w, t.dtype if n not in ("sT", "dlam", "ds0") else torch.float64, dk, dv, steps)
        err = (t.double() - w).abs()
        assert (err <= atol + rtol * (w.abs() + atol)).all(), (n, err.max().item(), atol)


SHAPES = [(1, 1, 1, 1, 8, 8), (2, 2, 1, 1, 16, 16), (1, 63, 1, 2, 64, 64), (1, 64, 2, 2, 64, 32), (2, 65, 1, 1, 128, 128),
          (1, 200, 2, 6, 32, 40), (2, 130, 3, 3, 72, 100), (1, 129, 1, 1, 127, 33), (1, 70, 1, 2, 1, 1),
          (1, 66, 1, 1, 7, 130), (1, 80, 1, 1, 65, 513 - 1), (9, 3, 1, 1, 20, 12)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_adjoint(shape, dtype):
    say(f"delta {shape} {dtype}")
    B, L, H, HV, dk, dv = shape
    x = make(*shape, DT[dtype], seed=L + dk)
    check(run(cuda(x)), reference(x), DT[dtype], dk, dv, L)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dims", [(64, 64), (72, 100), (33, 21)], ids=str)
def test_padding_and_documents(dims, dtype):
    """Rows of length 0, 1 and L, documents that start inside, at the edge and at
    the first step of a chunk; NaN and infinities in everything past the lengths."""
    say(f"delta packed {dims} {dtype}")
    dk, dv = dims
    x = make(5, 150, 2, 4, dk, dv, DT[dtype], seed=dk, views=True, packed=True)
    x["reset"][3] = 1  # every step a document
    x["lengths"][3] = 100
    want = reference(x)
    for b, n in enumerate(x["lengths"].tolist()):
        for name in ("q", "k", "v", "gates", "do"):
            x[name][b, n:] = float("nan") if b % 2 else float("inf")
    got = run(cuda(x))
    for b, n in enumerate(x["lengths"].tolist()):
        for name in ("o", "dq", "dk", "dv", "dgates"):
            assert not got[name][b, n:].any(), name
    check(got, want, DT[dtype], dk, dv, 150)
    # a document's start hides its decay
    assert not got["dgates"][0, :, 0][x["reset"][0] != 0].any()


def test_lengths_are_clamped():
    say("delta lengths clamped")
    x = make(3, 70, 1, 1, 16, 16, torch.float32)
    x["lengths"] = torch.tensor([-5, 1000, 70], dtype=torch.int32)
    check(run(cuda(x)), reference(x), torch.float32, 16, 16, 70)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_views_of_one_product_and_gradients_into_one(dtype):
    say(f"delta views {dtype}")
    for B, L, H, HV, dk, dv in ((2, 100, 2, 4, 64, 64), (2, 100, 1, 3, 30, 18), (1, 70, 1, 1, 33, 17)):
        x = make(B, L, H, HV, dk, dv, DT[dtype], seed=dk, views=True)
        d, want = cuda(x), reference(x)
        check(run(d), want, DT[dtype], dk, dv, L)
        args = (d["q"], d["k"], d["v"], d["gates"], d["lam"])
        f = layer.delta_scan(*args, s0=d["s0"], save=True)
        buf = torch.full((B, L, x["p"].shape[-1] + 6), 7.0, dtype=DT[dtype], device="cuda")
        out, at = {}, 0
        for n, s in (("dq", (H, dk)), ("dk", (H, dk)), ("dv", (HV, dv)), ("dgates", (2, HV))):
            out[n] = buf[..., at:at + s[0] * s[1]].unflatten(-1, s)
            at += s[0] * s[1]
        b = layer.delta_scan_adjoint(*args, d["do"], f["saved"], dsT=d["dsT"], want_ds0=True, out=out)
        assert all(b[n] is out[n] for n in out)
        check({**b, "o": f["o"], "sT": f["sT"]}, want, DT[dtype], dk, dv, L)
        assert (buf[..., at:] == 7.0).all()  # what lies between the rows


def test_no_state_no_gradient_of_it():
    say("delta without states")
    x = make(2, 90, 1, 2, 24, 40, torch.bfloat16)
    check(run(cuda(x), s0=False, dsT=False), reference(x, s0=False, dsT=False), torch.bfloat16, 24, 40, 90)
    d = cuda(x)
    f = layer.delta_scan(d["q"], d["k"], d["v"], d["gates"], d["lam"], save=True)
    b = layer.delta_scan_adjoint(d["q"], d["k"], d["v"], d["gates"], d["lam"], d["do"], f["saved"], want_dlam=False)
    assert b["dlam"] is None and b["ds0"] is None


def test_options():
    say("delta options")
    x = make(1, 80, 1, 1, 24, 24, torch.float32)
    kw = dict(c=2.5, eps=0.3, scale=1.75)
    check(run(cuda(x), **kw), reference(x, **kw), torch.float32, 24, 24, 80)


@pytest.mark.parametrize("case", ["equal keys", "no decay", "all decay", "always write", "never write", "zero rows",
                                  "tiny", "huge"])
def test_limits(case):
    """Where the inverse, the decays and the lengths are at their limits."""
    say(f"delta limits: {case}")
    x = make(1, 200, 1, 1, 32, 32, torch.float32, lam={"no decay": -40.0, "all decay": 30.0}.get(case, -3.0))
    if case == "equal keys":
        x["k"][:] = x["k"][:, :1]
        x["gates"][:, :, 1] = 20.0  # written in full: the inverse's series would reach C(63, 31)
        x["lam"][:] = -40.0
    elif case == "always write":
        x["gates"][:, :, 1] = 200.0
    elif case == "never write":
        x["gates"][:, :, 1] = -200.0
    elif case == "zero rows":
        x["q"][:, ::3] = 0.0
        x["k"][:, ::2] = 0.0
        x["v"][:, 5:9] = 0.0
    elif case == "tiny":
        for n in ("q", "k", "v"):
            x[n] *= 1e-12
    elif case == "huge":
        for n in ("q", "k", "v"):
            x[n] *= 1e12
    got, want = run(cuda(x)), reference(x)
    assert all(torch.isfinite(t).all() for t in got.values())
    if case == "tiny":  # |k|^2 is far below eps: the norm's gradient is 1 / sqrt(eps) times a difference
        want = {n: want[n] for n in ("o", "sT", "dv", "ds0")}
    check(got, want, torch.float32, 32, 32, 200)


def test_two_calls_carry_the_state():
    say("delta carry")
    x = make(2, 200, 1, 2, 64, 64, torch.bfloat16)
    d = cuda(x)
    cut = lambda a, b: [d[n][:, a:b] for n in ("q", "k", "v", "gates")]  # noqa: E731
    whole = layer.delta_scan(*cut(0, 200), d["lam"], s0=d["s0"])
    first = layer.delta_scan(*cut(0, 77), d["lam"], s0=d["s0"])
    rest = layer.delta_scan(*cut(77, 200), d["lam"], s0=first["sT"])
    want = reference(x)
    for got in (whole["sT"], rest["sT"]):
        atol, _ = R.delta_tol("sT", want["sT"], torch.float32, 64, 64, 200)
        assert ((got.cpu().double() - want["sT"]).abs() <= atol).all()
    both = torch.cat([first["o"], rest["o"]], 1)
    atol, rtol = R.delta_tol("o", want["o"], torch.bfloat16, 64, 64, 200)
    assert ((both.cpu().double() - want["o"]).abs() <= atol + rtol * (want["o"].abs() + atol)).all()


def test_many_heads_and_long_rows_repeat_bit_for_bit():
    say("delta repeats")
    x = cuda(make(3, 700, 4, 8, 64, 64, torch.bfloat16))
    a, b = run(x), run(x)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_a_long_row_against_its_parts():
    """One row of many chunks, few heads: whatever the call splits the row into,
    the state is that of short calls."""
    say("delta long row")
    L = 6000
    x = cuda(make(1, L, 1, 2, 128, 128, torch.bfloat16, seed=9))
    f = layer.delta_scan(x["q"], x["k"], x["v"], x["gates"], x["lam"], s0=x["s0"])
    s, outs = x["s0"], []
    for a in range(0, L, 500):
        r = layer.delta_scan(*(x[n][:, a:a + 500] for n in ("q", "k", "v", "gates")), x["lam"], s0=s)
        s, outs = r["sT"], outs + [r["o"]]
    # each is within the bound of 64 bits: two of them within twice that
    atol = 2 * 8 * R.U * (128 + 128 + 64 + L) * s.abs().max().item()
    assert ((f["sT"] - s).abs() <= atol).all()
    o, w = f["o"].float(), torch.cat(outs, 1).float()
    atol = 2 * 8 * R.U * (128 + 128 + 64 + L) * w.abs().max().item()
    assert ((o - w).abs() <= atol + 2 * 2.0 ** -8 * w.abs()).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1100, 1, 2, 72, 100), (5, 1030, 1, 1, 128, 128), (3, 1024, 1, 2, 33, 21),
                                   (1, 2500, 2, 2, 64, 64), (1, 1090, 1, 1, 65, 512), (2, 1024, 1, 1, 128, 130)], ids=str)
def test_segments(shape, dtype):
    """Few heads over many chunks: the sequence is scanned in segments, of rows that end
    inside, at the edge and in front of them."""
    say(f"delta segments {shape} {dtype}")
    B, L, H, HV, dk, dv = shape
    x = make(*shape, DT[dtype], seed=L, packed=B > 1, lam=-6.0)  # weak decay: what a segment adds is seen in the next
    if B > 1:
        x["lengths"] = torch.tensor([0, 256, 257, 1000, L][-B:], dtype=torch.int32)
        x["reset"][-2:] = 0
        x["reset"][-1, 700] = 1
    want = reference(x)
    d = cuda(x)
    got = run(d)
    check(got, want, DT[dtype], dk, dv, L)
    for name, y in run(d).items():
        assert torch.equal(y, got[name]), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 8, 8), (3, 2, 4, 64, 64), (5, 1, 3, 72, 100), (2, 2, 2, 128, 128),
                                   (4, 1, 1, 127, 33), (2, 1, 1, 1, 1), (130, 1, 1, 16, 40)], ids=str)
def test_step(shape, dtype):
    """One token per request against one step of the sequence, in a pool of slots."""
    say(f"delta step {shape} {dtype}")
    B, H, HV, dk, dv = shape
    x = make(B, 1, H, HV, dk, dv, DT[dtype], seed=dv, views=True)
    d, S = cuda(x), 2 * B + 3
    pool = torch.randn(S, HV, dk, dv, generator=torch.Generator().manual_seed(1)).cuda()
    slots = torch.randperm(S, generator=torch.Generator().manual_seed(2))[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, S
    before = pool.clone()
    at = {n: d[n][:, 0] for n in ("q", "k", "v", "gates")}
    o = layer.delta_step(at["q"], at["k"], at["v"], at["gates"], d["lam"], pool, slots=slots.cuda())
    w = {n: x[n].double() for n in ("q", "k", "v", "gates", "lam")}
    live = (slots >= 0) & (slots < S)
    s0 = before.cpu().double()[slots.long().clamp(0, S - 1)]
    wo, ws = R.delta(w["q"], w["k"], w["v"], w["gates"], w["lam"], s0=s0)
    atol, rtol = R.delta_tol("o", wo, DT[dtype], dk, dv, 1)
    err = (o.cpu().double() - wo[:, 0]).abs()[live]
    assert (err <= atol + rtol * (wo[:, 0].abs()[live] + atol)).all()
    assert not o[~live.cuda()].any()
    untouched = torch.ones(S, dtype=torch.bool)
    untouched[slots[live].long()] = False
    assert torch.equal(pool.cpu()[untouched], before.cpu()[untouched])
    atol, _ = R.delta_tol("sT", ws, torch.float32, dk, dv, 1)
    assert ((pool.cpu().double()[slots[live].long()] - ws[live]).abs() <= atol).all()


def test_steps_without_slots_follow_the_sequence():
    say("delta steps")
    B, L, H, HV, dk, dv = 3, 20, 2, 4, 64, 64
    x = make(B, L, H, HV, dk, dv, torch.bfloat16)
    d, want = cuda(x), reference(x)
    pool = d["s0"].clone()
    for t in range(L):
        o = layer.delta_step(*(d[n][:, t] for n in ("q", "k", "v", "gates")), d["lam"], pool)
        atol, rtol = R.delta_tol("o", want["o"], torch.bfloat16, dk, dv, L)
        assert ((o.cpu().double() - want["o"][:, t]).abs() <= atol + rtol * (want["o"][:, t].abs() + atol)).all()
    atol, _ = R.delta_tol("sT", want["sT"], torch.float32, dk, dv, L)
    assert ((pool.cpu().double() - want["sT"]).abs() <= atol).all()


def test_another_stream_and_a_replayed_graph():
    """Eager on a side stream, then captured; replays on new inputs, with eager work
    and synchronizations between them, give what eager calls give."""
    say("delta graph")
    x = cuda(make(2, 150, 1, 2, 64, 64, torch.bfloat16, packed=True))
    want = run(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(x)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(got[n], want[n]) for n in want)
    pool = x["s0"].clone()
    step = lambda: layer.delta_step(*(x[n][:, 0] for n in ("q", "k", "v", "gates")), x["lam"], pool)  # noqa: E731
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r, o = run(x), step()
    for seed in (3, 4, 5):
        y = cuda(make(2, 150, 1, 2, 64, 64, torch.bfloat16, seed=seed, packed=True))
        for n in x:
            if x[n] is not None:
                x[n].copy_(y[n])
        pool.copy_(y["s0"])
        g.replay()
        torch.cuda.synchronize()
        eager = run(x)
        for n in eager:
            assert torch.equal(r[n], eager[n]), (seed, n)
        after = pool.clone()
        pool.copy_(y["s0"])
        assert torch.equal(step(), o) and torch.equal(pool, after)


def test_replayed_segments():
    """The scans of few heads over many chunks, captured: a call's launches wait for
    each other in the graph as on the stream."""
    say("delta graph of segments")
    x = cuda(make(1, 1100, 1, 2, 64, 64, torch.bfloat16, lam=-6.0))
    run(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = run(x)
    for seed in (3, 4, 5):
        y = cuda(make(1, 1100, 1, 2, 64, 64, torch.bfloat16, seed=seed, lam=-6.0))
        for n in x:
            if x[n] is not None:
                x[n].copy_(y[n])
        g.replay()
        torch.cuda.synchronize()
        eager = run(x)
        for n in eager:
            assert torch.equal(r[n], eager[n]), (seed, n)


def test_refusals():
    say("delta refusals")
    x = cuda(make(2, 20, 1, 2, 16, 16, torch.bfloat16))
    args = [x[n] for n in ("q", "k", "v", "gates", "lam")]
    ok = layer.delta_scan(*args, save=True)

    def bad(i, t, **kw):
        a = list(args)
        if i is not None:
            a[i] = t
        with pytest.raises(PararnnError):
            layer.delta_scan(*a, **kw)

    bad(0, x["q"].float())
    bad(0, x["q"].half())
    bad(0, x["q"][:, :19])
    bad(0, x["q"].cpu())
    bad(1, x["k"][..., :15])
    bad(1, x["k"].repeat(1, 1, 2, 1))
    bad(2, x["v"].transpose(2, 3))
    bad(2, x["v"][:, :, :, ::2])
    bad(2, x["v"][:1].expand(2, 20, 2, 16))  # rows that overlap
    bad(2, torch.zeros(2, 20, 2, 513, dtype=torch.bfloat16, device="cuda"))
    bad(3, x["gates"][:, :, :1])
    bad(4, x["lam"].double())
    bad(4, None)
    bad(0, torch.zeros(2, 0, 1, 16, dtype=torch.bfloat16, device="cuda"))
    for kw in (dict(c=0.0), dict(eps=0.0), dict(scale=float("inf")), dict(s0=x["s0"][:1]), dict(s0=x["s0"].half()),
               dict(lengths=torch.zeros(2, device="cuda")), dict(reset=torch.zeros(2, 19, dtype=torch.uint8, device="cuda")),
               dict(out=torch.empty(2, 20, 2, 16, device="cuda")), dict(ws=torch.empty(64, dtype=torch.uint8, device="cuda")),
               dict(ws=torch.empty(64, device="cuda"))):
        bad(None, None, **kw)
    for kw in (dict(saved=None), dict(saved=ok["saved"][:-4]), dict(do=x["do"].float()), dict(do=None),
               dict(dsT=x["dsT"].half()), dict(out={"dq": x["q"].float()}), dict(out={"dv": x["v"][:, :, :, :8]})):
        a = dict(do=x["do"], saved=ok["saved"])
        a.update(kw)
        with pytest.raises(PararnnError):
            layer.delta_scan_adjoint(*args, a.pop("do"), a.pop("saved"), **a)
    st = [t[:, 0] for t in args[:4]]
    for pool in (None, x["s0"][0], x["s0"].half(), x["s0"][:1]):
        with pytest.raises(PararnnError):
            layer.delta_step(*st, x["lam"], pool)
    with pytest.raises(PararnnError):
        layer.delta_step(*st, x["lam"], x["s0"], slots=torch.zeros(2, dtype=torch.int64, device="cuda"))
