"""The gated recurrence in the kernels that long sequences and many channels
take: chunks with a carry, one and two channels per lane, groups of one and two
chunks, two ticket counters. (Sequences of up to 1024 steps with at most 256
channels in all run in one workgroup and do not come here.)"""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from tests import layer_reference as R
from tests.helpers import say
from tests.test_gpu_gated import DT, close, draw, pad_mask, run, to64

pytestmark = pytest.mark.gpu


def check(x, got, c=8.0):
    w = R.gated(**to64({k: x[k] for k in ("u", "lam", "h0", "lengths", "reset", "dh", "dhT")}), c=c)
    for k in got:
        v, e = w[k]
        # dlam of many rows: up to 225 partial rows per lane, 32 groups and a chunk's 30 steps and
        # segments are added one by one, and the reference's bound counts 64 of those roundings
        close(got[k], (v, 5 * e if k == "dlam" else e), k)


# tiles per chunk row: 800 (groups of 1, two ticket counters), 100 (groups of 2), 20 (4), 6 and fewer (8)
SHAPES = [(800, 800, 2), (800, 800, 3), (100, 1100, 4), (100, 1100, 5), (20, 900, 50), (3, 1500, 101), (1, 3000, 1),
          (2, 1025, 6)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("masks", ["none", "both"])
@pytest.mark.parametrize("B,L,D", SHAPES, ids=[f"{b}x{l}x{d}" for b, l, d in SHAPES])
def test_scan_and_adjoint(dtype, masks, B, L, D):
    say(f"gated scan {dtype} masks={masks} B={B} L={L} D={D}")
    x = draw(B, L, D, dtype, 7 * B + 3 * L + D, masks)
    if masks == "both":  # the padding holds NaN
        x["lengths"][-1] = L - 1
        pad = pad_mask(x)
        got = run({**x, "u": x["u"].where(pad[:, :, None, None], float("nan")),
                   "dh": x["dh"].where(pad[:, :, None], float("nan"))})
    else:
        got = run(x)
    check(x, got)


@pytest.mark.parametrize("D", [66, 67])
@pytest.mark.parametrize("c", [0.5, 64.0])
def test_decay_constant(c, D):
    say(f"gated scan c={c}, {D} channels")
    x = draw(1, 1300, D, "f32", 13)
    d = {k: None if v is None else v.cuda() for k, v in x.items()}
    f = layer.gated_scan(d["u"], d["lam"], h0=d["h0"], save=True, c=c)
    b = layer.gated_scan_adjoint(d["u"], d["lam"], d["dh"], f["saved"], dhT=d["dhT"], want_dh0=True, c=c)
    check(x, {"h": f["h"], "hT": f["hT"], "du": b["du"], "dlam": b["dlam"], "dh0": b["dh0"]}, c=c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [66, 67])
def test_saturated_gates(D, dtype):
    say(f"gated scan {dtype}, saturated gates, {D} channels")
    x = draw(1, 1300, D, dtype, 17)
    for at, gate, v in ((90, 0, -200.0), (600, 0, float("-inf")), (620, 0, float("inf")), (640, 1, float("-inf")),
                        (660, 1, 200.0)):
        x["u"][:, at:at + 10, gate] = v
    got = run(x)
    for k in got:
        assert torch.isfinite(got[k]).all(), k
    u = x["u"].clone()
    u[torch.isinf(u)] = torch.sign(u[torch.isinf(u)]) * 200.0  # the same gates, to 32 bits
    x["u"] = u
    check(x, got)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 131), ("f32", 64), ("f32", 67)])
def test_documents_are_apart_across_chunks(dtype, D, bad):
    """What one document holds reaches neither the next one's states nor the one
    before's gradients, over starts that lie chunks away from it."""
    say(f"gated scan {dtype}, {D} channels: {bad} in one document")
    B, L = 3, 2500
    x = draw(B, L, D, dtype, 19)
    x["reset"] = torch.zeros(B, L, dtype=torch.uint8)
    for t in (250, 600, 1500):
        x["reset"][:, t] = 1
    clean = run(x)
    u = x["u"].clone()
    x["u"][:, 700:705, 2] = bad
    x["u"][:, 900, 0] = float("nan")
    got = run(x)
    for k in ("h", "du"):
        assert torch.equal(got[k][:, :600], clean[k][:, :600]), k
        assert torch.equal(got[k][:, 1500:], clean[k][:, 1500:]), k
    assert torch.equal(got["hT"], clean["hT"]) and torch.equal(got["dh0"], clean["dh0"])
    x["u"] = u
    x["dh"][:, 2400] = bad
    x["dhT"][:] = bad
    got = run(x)
    assert torch.equal(got["du"][:, :1500], clean["du"][:, :1500])
    assert torch.equal(got["dh0"], clean["dh0"])
    assert not torch.isfinite(got["du"][:, 1500:2400].float()).any(dim=(0, 2)).all()


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 128), ("bf16", 66)])
def test_misaligned_tensors_use_narrower_accesses(dtype, D):
    say(f"gated scan, shifted tensors {dtype}, 1300 steps")
    B, L = 2, 1300
    x = draw(B, L, D, dtype, 31)

    def shift(t, k=1):
        s = torch.empty(t.numel() + k, dtype=t.dtype, device="cuda")
        s[k:] = t.cuda().reshape(-1)
        return s[k:].view(t.shape)

    f = layer.gated_scan(shift(x["u"]), x["lam"].cuda(), h0=shift(x["h0"]), save=True,
                         out=shift(torch.empty(B, L, D, dtype=DT[dtype])))
    b = layer.gated_scan_adjoint(shift(x["u"]), shift(x["lam"]), shift(x["dh"]), f["saved"], dhT=shift(x["dhT"]),
                                 want_dh0=True, du=shift(torch.empty(B, L, 3, D, dtype=DT[dtype])))
    check(x, {"h": f["h"], "hT": f["hT"], "du": b["du"], "dlam": b["dlam"], "dh0": b["dh0"]})


@pytest.mark.parametrize("B,L,D", [(800, 800, 2), (100, 1100, 5)])
def test_repeats_bit_for_bit(B, L, D):
    say(f"gated scan {B}x{L}x{D}, twice")
    x = draw(B, L, D, "bf16", 37, "both")
    a, b = run(x), run(x)
    for k in a:
        assert torch.equal(a[k], b[k]), k
