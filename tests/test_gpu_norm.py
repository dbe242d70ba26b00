"""GPU parity of the root-mean-square norm with the residual's addition and
8-bit output, and of its adjoint (layer.norm_residual, norm_residual_adjoint),
against 64 bits, every element within the bound of a 32-bit evaluation plus
half an ulp of the output's type."""
import numpy as np
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from tests import layer_reference as R
from tests.helpers import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SC = {"f32": torch.float32, "e8m0": torch.float8_e8m0fnu}
# one element, rows shorter than a block, odd widths (single-element accesses),
# every launch shape up to the widest, and sizes next to its limits
SHAPES = [(1, 1), (3, 7), (5, 128), (2, 129), (7, 512), (9, 520), (6, 1000), (1, 1024), (5, 1025), (4, 2048),
          (3, 4096), (2, 4099), (2, 8192), (2, 8200), (1, 16384), (700, 264)]
IDS = [f"{n}x{d}" for n, d in SHAPES]


def draw(N, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = {"x": n(N, D), "residual": 3 * n(N, D), "dy": n(N, D), "ds": n(N, D)}
    x = {k: v.to(DT[dtype]) for k, v in x.items()}
    x["w"] = 1.0 + 0.3 * n(D)
    return x


def f64(t):
    return t.detach().cpu().double().numpy()


def scale_values(s):
    s = s.cpu()
    if s.dtype == torch.float32:
        return s.double().numpy()
    b = s.view(torch.uint8).numpy().astype(np.float64)
    return np.where(b == 255, np.nan, 2.0 ** (b - 127))


def close(got, want, what):
    v, e = want
    tol = e + (R.BF16_EPS * (np.abs(v) + e) if got.dtype == torch.bfloat16 else 0.0)
    err = np.abs(f64(got) - v)
    assert (err <= tol).all(), f"{what}: {int((~(err <= tol)).sum())} outside, worst {np.nanmax(err / tol):.3g} bounds"


def check_fp8(r, want, scale):
    """The scales, and each value within half an ulp of e4m3 of y / scale."""
    y, e = want
    s = scale_values(r["scale"]).T  # [N][blocks]
    m = R.blocks_max(y) / 448.0
    rel = 52 * R.U
    if scale == "f32":
        assert (np.abs(s - m) <= rel * m).all()
    else:
        lo, hi = 2.0 ** np.ceil(np.log2(m * (1 - rel))), 2.0 ** np.ceil(np.log2(m * (1 + rel)))
        assert ((s == lo) | (s == hi)).all()
    full = np.repeat(s, 128, axis=1)[:, :y.shape[1]]
    q = f64(r["y"].float())
    v = y / full
    half = np.maximum(2.0 ** -4 * 2.0 ** np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -30))), 2.0 ** -10)
    assert (np.abs(q - v) <= half + rel * np.abs(v)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D", SHAPES, ids=IDS)
def test_norm(dtype, N, D):
    say(f"norm {dtype} {N}x{D}")
    x = draw(N, D, dtype, N + D)
    d = {k: v.cuda() for k, v in x.items()}
    want = R.norm(f64(x["x"]), f64(x["w"]), f64(x["residual"]))
    r = layer.norm_residual(d["x"], d["w"], residual=d["residual"])
    assert r["scale"] is None
    close(r["s"], want["s"], "s")
    close(r["y"], want["y"], "y")
    for scale in SC:
        q = layer.norm_residual(d["x"], d["w"], residual=d["residual"], scale_dtype=SC[scale])
        assert torch.equal(q["s"], r["s"]) and q["scale"].shape == (-(-D // 128), N)
        check_fp8(q, want["y"], scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D", SHAPES, ids=IDS)
def test_norm_adjoint(dtype, N, D):
    say(f"norm adjoint {dtype} {N}x{D}")
    x = draw(N, D, dtype, 3 * N + D)
    d = {k: v.cuda() for k, v in x.items()}
    a = layer.norm_residual_adjoint(d["x"], d["w"], d["dy"], ds=d["ds"])
    want = R.norm_adjoint(f64(x["x"]), f64(x["w"]), f64(x["dy"]), f64(x["ds"]))
    close(a["dx"], want["dx"], "dx")
    close(a["dw"], want["dw"], "dw")
    b = layer.norm_residual_adjoint(d["x"], d["w"], d["dy"], want_dw=False)
    assert b["dw"] is None
    close(b["dx"], R.norm_adjoint(f64(x["x"]), f64(x["w"]), f64(x["dy"]))["dx"], "dx without ds")


def test_without_residual_and_eps():
    say("norm without a residual, eps 0 and 1")
    x = draw(4, 300, "bf16", 1)
    for eps in (0.0, 1.0):
        r = layer.norm_residual(x["x"].cuda(), x["w"].cuda(), eps=eps)
        close(r["y"], R.norm(f64(x["x"]), f64(x["w"]), eps=eps)["y"], "y")
        assert torch.equal(r["s"].cpu(), x["x"])


@pytest.mark.parametrize("scale", list(SC))
def test_zero_rows_and_zero_blocks(scale):
    """A row of zeros gives zeros (also with 8 bits), and a block of zeros has
    the smallest scale."""
    say(f"norm of zeros, {scale} scales")
    x = torch.zeros(3, 384)
    x[1, :128] = torch.randn(128, generator=torch.Generator().manual_seed(2))
    w = torch.ones(384)
    r = layer.norm_residual(x.cuda(), w.cuda(), scale_dtype=SC[scale])
    want = R.norm(x.double().numpy(), w.double().numpy())
    check_fp8(r, want["y"], scale)
    assert (r["y"].float()[[0, 2]] == 0).all() and (r["y"].float()[1, 128:] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("scale", list(SC))
def test_a_bad_value_stays_in_its_row(scale, bad):
    say(f"norm with {bad}, {scale} scales")
    x = draw(6, 512, "f32", 5)
    xx = x["x"].clone()
    xx[3, 200] = bad
    good = layer.norm_residual(x["x"].cuda(), x["w"].cuda(), scale_dtype=SC[scale])
    r = layer.norm_residual(xx.cuda(), x["w"].cuda(), scale_dtype=SC[scale])
    keep = [0, 1, 2, 4, 5]
    assert torch.equal(r["y"].view(torch.uint8)[keep], good["y"].view(torch.uint8)[keep])
    v = r["y"].float().cpu().double().numpy() * np.repeat(scale_values(r["scale"]).T, 128, axis=1)
    assert np.isnan(v[3, 128:256]).all()


def test_misaligned_rows_use_single_accesses():
    say("norm, shifted tensors")
    N, D = 5, 256
    x = draw(N, D, "bf16", 7)

    def shift(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        s[1:] = t.cuda().reshape(-1)
        return s[1:].view(t.shape)

    a = layer.norm_residual(x["x"].cuda(), x["w"].cuda(), residual=x["residual"].cuda(), scale_dtype=torch.float32)
    b = layer.norm_residual(shift(x["x"]), x["w"].cuda(), residual=shift(x["residual"]), scale_dtype=torch.float32)
    for k in ("y", "s", "scale"):
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k
    a = layer.norm_residual_adjoint(x["x"].cuda(), x["w"].cuda(), x["dy"].cuda(), ds=x["ds"].cuda())
    b = layer.norm_residual_adjoint(shift(x["x"]), x["w"].cuda(), shift(x["dy"]), ds=shift(x["ds"]))
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dw"], b["dw"])


def test_many_rows_repeat_bit_for_bit():
    say("norm adjoint of 20001 rows, twice")
    x = draw(20001, 72, "bf16", 9)
    d = {k: v.cuda() for k, v in x.items()}
    a = layer.norm_residual_adjoint(d["x"], d["w"], d["dy"])
    b = layer.norm_residual_adjoint(d["x"], d["w"], d["dy"], ws=a["ws"].fill_(255))
    assert torch.equal(a["dw"], b["dw"]) and torch.equal(a["dx"], b["dx"])
    want = R.norm_adjoint(f64(x["x"]), f64(x["w"]), f64(x["dy"]))
    close(a["dw"], want["dw"], "dw")
    close(a["dx"], want["dx"], "dx")
