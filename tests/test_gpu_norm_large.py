"""The norm and its adjoint past the last-level cache (accesses that go past the
caches) and with more rows than one round of workgroups: the same bits as the
same rows in smaller calls, which run the cached kernels, and the sums over
all rows against 64 bits."""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from tests import layer_reference as R
from tests import test_gpu_norm as N
from tests.helpers import say

pytestmark = pytest.mark.gpu

PARTS = 6
# every launch shape by columns; rows so that the call's bytes pass 256 MiB (7 and 8 per element in bf16)
WIDTHS = [512, 1000, 2048, 4096, 8192, 16384]


def draw(N, D, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return [n(N, D).to(dtype) for _ in range(4)] + [1.0 + 0.3 * n(D)]


def parts(N):
    """Slices of rows, the last one shorter."""
    k = -(-N // PARTS)
    return [slice(i, min(i + k, N)) for i in range(0, N, k)]


def bits(t):
    return t.view(torch.uint8)


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm(dtype, D):
    N = (1 << 28) // (D * (7 if dtype is torch.bfloat16 else 13)) + 37
    say(f"norm {dtype} {N}x{D}")
    x, r, _, _, w = draw(N, D, dtype, D)
    for sc in (None, torch.float32, torch.float8_e8m0fnu):
        whole = layer.norm_residual(x, w, residual=r, scale_dtype=sc)
        for sl in parts(N):
            p = layer.norm_residual(x[sl], w, residual=r[sl], scale_dtype=sc)
            assert torch.equal(bits(whole["y"][sl]), bits(p["y"])), (sc, sl)
            assert torch.equal(whole["s"][sl], p["s"]), (sc, sl)
            if sc is not None:
                assert torch.equal(whole["scale"].view(torch.uint8 if sc.itemsize == 1 else torch.int32)[:, sl],
                                   p["scale"].view(torch.uint8 if sc.itemsize == 1 else torch.int32)), (sc, sl)


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_adjoint(dtype, D):
    N = (1 << 28) // (D * 4 * dtype.itemsize) + 37
    say(f"norm adjoint {dtype} {N}x{D}")
    s, dy, ds, _, w = draw(N, D, dtype, D + 1)
    whole = layer.norm_residual_adjoint(s, w, dy, ds=ds)
    mag = torch.zeros(D, dtype=torch.float64, device="cuda")
    dw = torch.zeros_like(mag)
    for sl in parts(N):
        p = layer.norm_residual_adjoint(s[sl], w, dy[sl], ds=ds[sl])
        assert torch.equal(whole["dx"][sl], p["dx"]), sl
        t = s[sl].double()
        t = dy[sl].double() * t / (t.square().mean(1, keepdim=True) + 1e-6).sqrt()
        dw += t.sum(0)
        mag += t.abs().sum(0)
    # the norm's statistics (96 roundings), then a lane's rows and the partial rows, added one by one
    assert ((whole["dw"].double() - dw).abs() <= R.U * (96 + N / 256) * mag + R.TINY).all()
    assert torch.equal(whole["dw"], layer.norm_residual_adjoint(s, w, dy, ds=ds, ws=whole["ws"].fill_(255))["dw"])


@pytest.mark.parametrize("D", [1032, 2056])
def test_second_round_of_workgroups(D):
    """More rows than the 8192 workgroups of a forward pass, below the caches' size."""
    N = 8192 + 301
    say(f"norm {N}x{D}")
    x, r, _, _, w = draw(N, D, torch.bfloat16, 3)
    whole = layer.norm_residual(x, w, residual=r)
    for sl in parts(N):
        p = layer.norm_residual(x[sl], w, residual=r[sl])
        assert torch.equal(whole["y"][sl], p["y"]) and torch.equal(whole["s"][sl], p["s"])


# widths that are not whole vectors of 8, one for each launch shape that the narrower tests leave out
@pytest.mark.parametrize("D", [777, 3001, 16383])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_odd_widths(dtype, D):
    say(f"norm and adjoint {dtype} 5x{D}")
    x = N.draw(5, D, dtype, D)
    d = {k: v.cuda() for k, v in x.items()}
    want = R.norm(*(N.f64(x[k]) for k in ("x", "w", "residual")))
    r = layer.norm_residual(d["x"], d["w"], residual=d["residual"])
    N.close(r["s"], want["s"], "s")
    N.close(r["y"], want["y"], "y")
    for scale in N.SC:
        q = layer.norm_residual(d["x"], d["w"], residual=d["residual"], scale_dtype=N.SC[scale])
        N.check_fp8(q, want["y"], scale)
    a = layer.norm_residual_adjoint(d["x"], d["w"], d["dy"], ds=d["ds"])
    want = R.norm_adjoint(*(N.f64(x[k]) for k in ("x", "w", "dy", "ds")))
    N.close(a["dx"], want["dx"], "dx")
    N.close(a["dw"], want["dw"], "dw")
