"""GPU parity of the gated linear recurrence, its adjoint and its single-token
step (layer.gated_scan, gated_scan_adjoint, gated_step) against the 64-bit
loop, every element within the running bound of a 32-bit evaluation (plus half
an ulp of bf16 where the result is bf16)."""
import numpy as np
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from tests import layer_reference as R
from tests.helpers import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def draw(B, L, D, dtype, seed, masks="none"):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = {"u": n(B, L, 3, D).to(DT[dtype]), "h0": n(B, D), "dh": n(B, L, D).to(DT[dtype]), "dhT": n(B, D)}
    # softplus from 1e-4 to 1: memories of two to thousands of steps
    x["lam"] = torch.log(torch.expm1(torch.exp(torch.rand(D, generator=g) * 9.2 - 9.2)))
    x["lengths"] = x["reset"] = None
    if masks in ("lengths", "both"):
        ln = torch.randint(0, L + 1, (B,), generator=g)
        ln[0] = L
        if B > 1:
            ln[1] = 0
        if B > 2:
            ln[2] = 1
        x["lengths"] = ln.to(torch.int32)
    if masks in ("reset", "both"):
        x["reset"] = (torch.rand(B, L, generator=g) < 0.03).to(torch.uint8)
    return x


def to64(x):
    return {k: None if v is None else v.double().numpy() if v.is_floating_point() else v.numpy()
            for k, v in x.items()}


def run(x, train=True, **kw):
    d = {k: None if v is None else v.cuda() for k, v in x.items()}
    m = dict(lengths=d["lengths"], reset=d["reset"], **kw)
    f = layer.gated_scan(d["u"], d["lam"], h0=d["h0"], save=train, **m)
    out = {"h": f["h"], "hT": f["hT"]}
    if train:
        b = layer.gated_scan_adjoint(d["u"], d["lam"], d["dh"], f["saved"], dhT=d["dhT"], want_dh0=True, **m)
        out.update({k: b[k] for k in ("du", "dlam", "dh0")})
    torch.cuda.synchronize()
    return out


def pad_mask(x):
    """[B][L], true at the steps of a row."""
    return torch.arange(x["u"].shape[1])[None] < x["lengths"][:, None]


def close(got, want, what):
    v, e = want
    tol = e + (R.BF16_EPS * (np.abs(v) + e) if got.dtype == torch.bfloat16 else 0.0) + R.TINY
    err = np.abs(got.cpu().double().numpy() - v)
    bad = ~(err <= tol)
    if bad.any():
        k = np.unravel_index(np.argmax(np.where(bad, err / tol, 0)), err.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {err.size} outside, at {k}: got {got[k].item()!r} "
                             f"want {v[k]!r} bound {tol[k]:.3g}")


def check(x, got, c=8.0):
    w = R.gated(**to64({k: x[k] for k in ("u", "lam", "h0", "lengths", "reset", "dh", "dhT")}), c=c)
    for k in got:
        close(got[k], w[k], k)


# one step, tiny, odd widths (one channel per lane), widths of 2 mod 4, sizes
# around the chunks of 96 to 256 steps and the tiles of 32 and 64 channels
SHAPES = [(1, 1, 1), (2, 2, 3), (3, 5, 64), (1, 127, 65), (2, 128, 6), (2, 129, 4), (1, 256, 32), (1, 257, 100),
          (3, 511, 62), (2, 1000, 33), (1, 2500, 8), (5, 300, 130)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("masks", ["none", "both"])
@pytest.mark.parametrize("B,L,D", SHAPES, ids=[f"{b}x{l}x{d}" for b, l, d in SHAPES])
def test_scan_and_adjoint(dtype, masks, B, L, D):
    say(f"gated scan {dtype} masks={masks} B={B} L={L} D={D}")
    x = draw(B, L, D, dtype, 7 * B + 3 * L + D, masks)
    check(x, run(x))


@pytest.mark.parametrize("masks", ["lengths", "reset"])
def test_each_mask_alone(masks):
    say(f"gated scan masks={masks}")
    x = draw(4, 700, 72, "bf16", 5, masks)
    check(x, run(x))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("masks", ["lengths", "both"])
def test_lengths_at_chunk_borders(masks, dtype):
    """Rows that end at, before and behind the border of a chunk in either
    direction; the padding behind them holds NaN."""
    say(f"gated scan {dtype} masks={masks}, lengths at chunk borders")
    lengths = torch.tensor([800, 0, 1, 95, 96, 97, 191, 192, 193, 256, 257, 384, 385, 799], dtype=torch.int32)
    x = draw(len(lengths), 800, 68, dtype, 23, masks)
    x["lengths"] = lengths
    got = run({**x, "u": x["u"].where(pad_mask(x)[:, :, None, None], float("nan")),
               "dh": x["dh"].where(pad_mask(x)[:, :, None], float("nan"))})
    check(x, got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_chunks(dtype):
    """Several groups of chunks, so the carry goes through both of its links."""
    say(f"gated scan {dtype}, 20000 steps")
    x = draw(1, 20000, 66, dtype, 11, "reset")
    x["reset"][:, 5:] = 0
    x["reset"][0, 9000] = 1
    check(x, run(x))


def test_without_optional_arguments():
    say("gated scan: no initial state, no dhT, no dlam")
    x = draw(2, 300, 64, "f32", 3)
    x["h0"] = x["dhT"] = None
    got = run(x)
    check(x, got)
    f = layer.gated_scan(x["u"].cuda(), x["lam"].cuda())
    assert f["saved"] is None and torch.equal(f["h"], got["h"])


@pytest.mark.parametrize("c", [0.5, 64.0])
def test_decay_constant(c):
    say(f"gated scan c={c}")
    x = draw(1, 400, 32, "f32", 13)
    d = {k: None if v is None else v.cuda() for k, v in x.items()}
    f = layer.gated_scan(d["u"], d["lam"], h0=d["h0"], save=True, c=c)
    b = layer.gated_scan_adjoint(d["u"], d["lam"], d["dh"], f["saved"], dhT=d["dhT"], want_dh0=True, c=c)
    check(x, {"h": f["h"], "hT": f["hT"], "du": b["du"], "dlam": b["dlam"], "dh0": b["dh0"]}, c=c)


def test_saturated_gates():
    """Gates at 0 and 1: a decay of exactly 1 takes no input (and has a finite
    gradient), infinite arguments included."""
    say("gated scan, saturated gates")
    x = draw(1, 300, 64, "f32", 17)
    x["u"][:, 10:20, 0] = -200.0
    x["u"][:, 20:30, 0] = float("-inf")
    x["u"][:, 30:40, 0] = float("inf")
    x["u"][:, 40:50, 1] = float("-inf")
    x["u"][:, 50:60, 1] = 200.0
    got = run(x)
    for k in got:
        assert torch.isfinite(got[k]).all(), k
    u = x["u"].clone()
    u[torch.isinf(u)] = torch.sign(u[torch.isinf(u)]) * 200.0  # the same gates, to 32 bits
    x["u"] = u
    check(x, got)


@pytest.mark.parametrize("masks", ["lengths", "reset"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_masked_values_do_not_reach_the_rest(masks, bad):
    """What a mask hides may hold anything: steps past a row's length, and for
    a document the documents before (states) and after it (gradients)."""
    say(f"gated scan: {bad} hidden by {masks}")
    B, L, D = 2, 900, 64
    x = draw(B, L, D, "bf16", 19)
    if masks == "lengths":
        x["lengths"] = torch.tensor([333, 0], dtype=torch.int32)
        x["u"][0, 333:] = bad
        x["dh"][0, 333:] = bad
        x["u"][1], x["dh"][1] = bad, bad
        got = run(x)
        assert all(torch.isfinite(v).all() for v in got.values())
        x["u"] = torch.nan_to_num(x["u"], nan=0.0, posinf=0.0, neginf=0.0)
        x["dh"] = torch.nan_to_num(x["dh"], nan=0.0, posinf=0.0, neginf=0.0)
        check(x, got)
        return
    x["reset"] = torch.zeros(B, L, dtype=torch.uint8)
    x["reset"][:, 250], x["reset"][:, 600] = 1, 1
    clean = run(x)
    # the middle document gets bad values: the first and the last stay as they were
    x["u"][:, 300:310, 2] = bad
    x["u"][:, 320, 0] = float("nan")
    got = run(x)
    for k in ("h", "du"):
        assert torch.equal(got[k][:, :250], clean[k][:, :250]), k
        assert torch.equal(got[k][:, 600:], clean[k][:, 600:]), k
    assert torch.equal(got["hT"], clean["hT"]) and torch.equal(got["dh0"], clean["dh0"])
    # and bad upstream gradients in the last document leave the earlier ones alone
    x["u"] = draw(B, L, D, "bf16", 19)["u"]
    x["dh"][:, 700] = bad
    got = run(x)
    assert torch.equal(got["du"][:, :600], clean["du"][:, :600])
    assert torch.equal(got["dh0"], clean["dh0"])


def test_nan_propagates_along_its_channel():
    say("gated scan: NaN in one channel")
    x = draw(2, 700, 96, "f32", 23)
    x["u"][1, 300, 2, 7] = float("nan")
    got = run(x)
    nan = torch.isnan(got["h"].cpu())
    want = torch.zeros_like(nan)
    want[1, 300:, 7] = True
    assert torch.equal(nan, want)
    assert torch.isnan(got["hT"][1, 7]) and int(torch.isnan(got["hT"]).sum()) == 1


def test_lengths_outside_the_row_are_clamped():
    say("gated scan: lengths out of range")
    x = draw(2, 100, 16, "f32", 29)
    x["lengths"] = torch.tensor([1000, -5], dtype=torch.int32)
    check(x, run(x))


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 128), ("bf16", 66)])
def test_misaligned_tensors_use_narrower_accesses(dtype, D):
    say(f"gated scan, shifted tensors {dtype}")
    B, L = 2, 300
    x = draw(B, L, D, dtype, 31)
    want = run(x)

    def shift(t, k=1):
        s = torch.empty(t.numel() + k, dtype=t.dtype, device="cuda")
        s[k:] = t.cuda().reshape(-1)
        return s[k:].view(t.shape)

    f = layer.gated_scan(shift(x["u"]), x["lam"].cuda(), h0=shift(x["h0"]), save=True,
                         out=shift(torch.empty(B, L, D, dtype=DT[dtype])))
    b = layer.gated_scan_adjoint(shift(x["u"]), shift(x["lam"]), shift(x["dh"]), f["saved"], dhT=shift(x["dhT"]),
                                 want_dh0=True, du=shift(torch.empty(B, L, 3, D, dtype=DT[dtype])))
    got = {"h": f["h"], "hT": f["hT"], "du": b["du"], "dlam": b["dlam"], "dh0": b["dh0"]}
    check(x, got)
    check(x, want)


def test_repeats_bit_for_bit_with_a_used_workspace():
    say("gated scan: repeated calls")
    x = draw(3, 5000, 192, "bf16", 37, "both")
    first = run(x)
    d = {k: None if v is None else v.cuda() for k, v in x.items()}
    m = dict(lengths=d["lengths"], reset=d["reset"])
    ws = None
    for _ in range(3):
        f = layer.gated_scan(d["u"], d["lam"], h0=d["h0"], save=True, ws=ws, **m)
        ws = f["ws"]
        if ws is not None:
            ws.fill_(255)
        b = layer.gated_scan_adjoint(d["u"], d["lam"], d["dh"], f["saved"], dhT=d["dhT"], want_dh0=True, **m)
        for k, v in {"h": f["h"], "hT": f["hT"], "du": b["du"], "dlam": b["dlam"], "dh0": b["dh0"]}.items():
            assert torch.equal(v, first[k]), k


def test_on_another_stream_and_in_a_graph():
    say("gated scan: side stream, graph replays")
    x = draw(2, 3000, 128, "bf16", 41)
    want = run(x)
    d = {k: None if v is None else v.cuda() for k, v in x.items()}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        f = layer.gated_scan(d["u"], d["lam"], h0=d["h0"], save=True)
        layer.gated_scan_adjoint(d["u"], d["lam"], d["dh"], f["saved"], dhT=d["dhT"], want_dh0=True)
    s.synchronize()
    assert torch.equal(f["h"], want["h"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        f = layer.gated_scan(d["u"], d["lam"], h0=d["h0"], save=True)
        b = layer.gated_scan_adjoint(d["u"], d["lam"], d["dh"], f["saved"], dhT=d["dhT"], want_dh0=True)
    for k in range(4):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(f["h"], want["h"]) and torch.equal(b["du"], want["du"]), k
        assert torch.equal(b["dlam"], want["dlam"]), k
        f["h"].zero_()
        b["du"].zero_()


def test_step_continues_the_scan():
    """Single steps from the scan's final state give the scan's own next states."""
    say("gated step after a scan")
    B, L, D = 3, 70, 100
    x = draw(B, L, D, "f32", 43)
    u, lam = x["u"].cuda(), x["lam"].cuda()
    pre = layer.gated_scan(u[:, :40].contiguous(), lam)
    state = torch.full((7, D), 5.0, device="cuda")
    slots = torch.tensor([6, 0, 3], dtype=torch.int32, device="cuda")
    state[slots.long()] = pre["hT"]
    x["h0"] = None
    w, e = R.gated(**to64({k: x[k] for k in ("u", "lam", "h0")}))["h"]
    for t in range(40, L):
        h = layer.gated_step(u[:, t].contiguous(), lam, state, slots=slots)
        close(h, (w[:, t], e[:, t]), f"step {t}")
    assert torch.equal(state[slots.long()], h)
    assert (state[[1, 2, 4, 5]] == 5.0).all()


STEPS = [(1, 1, 1), (1, 64, 1), (5, 33, 9), (64, 4096, 100), (300, 130, 300), (2, 6, 4)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D,S", STEPS, ids=[f"{b}x{d}of{s}" for b, d, s in STEPS])
def test_step(dtype, B, D, S):
    say(f"gated step {dtype} B={B} D={D} S={S}")
    x = draw(B, 1, D, dtype, B + D)
    pool = torch.randn(S, D, generator=torch.Generator().manual_seed(S))
    slots = torch.randperm(S, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32)
    if B > 1:
        slots[1] = -1
    if B > 3:
        slots[3] = S  # past the pool
    live = (slots >= 0) & (slots < S)
    x["h0"] = torch.where(live[:, None], pool[slots.clamp(0, S - 1).long()], torch.zeros(1))
    w, e = R.gated(**to64({k: x[k] for k in ("u", "lam", "h0")}))["hT"]
    state = pool.clone().cuda()
    h = layer.gated_step(x["u"][:, 0].contiguous().cuda(), x["lam"].cuda(), state, slots=slots.cuda())
    lv = live.numpy()[:, None]
    close(h, (np.where(lv, w, 0.0), np.where(lv, e, 0.0)), "h")
    want, ew = pool.double().numpy().copy(), np.zeros((S, D))
    want[slots[live].long().numpy()] = w[live.numpy()]
    ew[slots[live].long().numpy()] = e[live.numpy()]
    close(state, (want, ew), "state")


def test_step_without_slots_takes_the_rows_in_order():
    say("gated step without slots")
    x = draw(4, 1, 32, "f32", 47)
    state = x["h0"].clone().cuda()
    h = layer.gated_step(x["u"][:, 0].contiguous().cuda(), x["lam"].cuda(), state)
    w = R.gated(**to64({k: x[k] for k in ("u", "lam", "h0")}))["hT"]
    close(h, w, "h")
    assert torch.equal(h, state)
