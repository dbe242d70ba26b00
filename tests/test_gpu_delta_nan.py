"""Values that are no numbers among the delta rule's steps: how far they reach, and that the zeros behind a row's
last step stay zeros."""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from tests.helpers import say
from tests.test_gpu_delta import DT, cuda, make, run

pytestmark = pytest.mark.gpu
B, L, AT, N = 2, 300, 150, 170  # row 0 has N steps, the bad one is AT, in chunk 2 of 64


def inputs(dtype, H, HV):
    x = make(B, L, H, HV, 64, 40, dtype, seed=4)
    x["lengths"] = torch.tensor([N, L], dtype=torch.int32)
    x["reset"] = torch.zeros(B, L, dtype=torch.uint8)
    x["reset"][0, 70] = 1
    return x


@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=str)
@pytest.mark.parametrize("where", ["q", "k", "v", "gates", "strength"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_reach(dtype, where, bad):
    """Results of the steps in front, of the other row and of the other heads are what they are without it, bit for
    bit; those after it are no numbers, but for q's, which only its own step reads; the row's padding holds zeros, in
    the results and in the gradients."""
    say(f"delta reach of {bad} in {where} {dtype}")
    H, HV = 2, 4
    x = inputs(DT[dtype], H, HV)
    clean = run(cuda(x))
    h = 1
    if where in ("gates", "strength"):  # the decay's, or that of what is written
        x["gates"][0, AT, int(where == "strength"), h] = bad
    else:
        x[where][0, AT, h, 3] = bad
    got = run(cuda(x))
    # value heads that take head h of q or k
    hit = [h] if where in ("v", "gates", "strength") else [hv for hv in range(HV) if hv // (HV // H) == h]
    free = [hv for hv in range(HV) if hv not in hit]
    for n in ("o", "dv"):
        assert torch.equal(got[n][1], clean[n][1]) and torch.equal(got[n][0][:, free], clean[n][0][:, free]), n
    assert torch.equal(got["o"][0, :AT], clean["o"][0, :AT])
    if where == "q":
        assert torch.equal(got["o"][0, AT + 1:N], clean["o"][0, AT + 1:N]) and torch.equal(got["sT"], clean["sT"])
    elif where == "k" or bad != bad:  # (an infinite gate is the limit of large ones)
        c = [3] if where == "v" else list(range(40))
        assert torch.isnan(got["o"][0, AT:N][:, hit][..., c]).all() and torch.isnan(got["sT"][0, hit][..., c]).all()
    for n in ("sT", "ds0"):
        assert torch.equal(got[n][1], clean[n][1]) and torch.equal(got[n][0][free], clean[n][0][free]), n
    assert torch.equal(got["dlam"][free], clean["dlam"][free])
    for n in ("dq", "dk", "dgates"):
        assert torch.equal(got[n][1], clean[n][1]), n
    qh = hit[0] // (HV // H)
    for n in ("dq", "dk"):
        assert torch.equal(got[n][0][:, 1 - qh], clean[n][0][:, 1 - qh]), n
    if where == "v":
        assert torch.equal(got["o"][0, :, h, :3], clean["o"][0, :, h, :3])  # the other columns
    for n in ("o", "dq", "dk", "dv", "dgates"):
        assert not got[n][0, N:].any(), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_state_that_is_no_number(dtype):
    say(f"delta NaN state {dtype}")
    x = inputs(DT[dtype], 1, 1)
    x["s0"][0, 0, 5, 7] = float("nan")
    d = cuda(x)
    r = layer.delta_scan(d["q"], d["k"], d["v"], d["gates"], d["lam"], s0=d["s0"], lengths=d["lengths"])
    assert not r["o"][0, N:].any() and torch.isfinite(r["o"][1]).all()
    assert torch.isnan(r["o"][0, :N, 0, 7]).all() and torch.isfinite(r["o"][0, :, 0, :7]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["k", "v", "gates"])
def test_reach_over_segments(dtype, where):
    """A sequence that is scanned in segments: as in one piece."""
    say(f"delta reach over segments {where} {dtype}")
    n, at = 2200, 1333
    x = make(1, n, 1, 2, 128, 72, DT[dtype], seed=6, lam=-6.0)
    args = lambda: [t.cuda() for t in (x["q"], x["k"], x["v"], x["gates"], x["lam"])]  # noqa: E731
    clean = layer.delta_scan(*args(), s0=x["s0"].cuda())["o"]
    t = x[where]
    t.view(1, n, -1)[0, at, 0] = float("nan")
    got = layer.delta_scan(*args(), s0=x["s0"].cuda())["o"]
    assert torch.equal(got[:, :at], clean[:, :at])
    heads = slice(None) if where == "k" else slice(0, 1)
    cols = slice(0, 1) if where == "v" else slice(None)
    assert torch.isnan(got[:, at:, heads, cols]).all()
    if where != "k":
        assert torch.equal(got[:, :, 1], clean[:, :, 1])
