"""The 8-bit integer product against 64-bit integers: every launch shape, odd
sizes, the largest sums, scales at their limits. The integer sum is exact; its
rounding to fp32, two products and the bias are four roundings of at most U of
the value in front of them, then half a step of the result's type."""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from nonlinear_rnn_solve_newton_amd.binding import PararnnError
from tests import delta_reference as R
from tests.helpers import say

pytestmark = pytest.mark.gpu
U = R.U


def make(M, N, K, seed=0, bias=True):
    g = torch.Generator().manual_seed(seed)
    i8 = lambda *s: torch.randint(-128, 128, s, generator=g, dtype=torch.int8)  # noqa: E731
    return dict(a=i8(M, K), w=i8(N, K), sa=torch.rand(M, generator=g) + 0.01, sw=torch.rand(N, generator=g) * 0.1 + 1e-3,
                bias=torch.randn(N, generator=g) if bias else None)


def check(x, dtype, out=None):
    d = {n: None if t is None else t.cuda() for n, t in x.items()}
    y = layer.matmul_int8(d["a"], d["sa"], d["w"], d["sw"], bias=d["bias"], out_dtype=dtype, out=out)
    exact = (d["a"].double() @ d["w"].double().t()) * d["sa"].double()[:, None] * d["sw"].double()
    want = exact if d["bias"] is None else exact + d["bias"].double()
    bound = 3 * U * exact.abs() + U * want.abs()
    err = (y.double() - want).abs()
    assert y.dtype == dtype and (err <= bound + R.half_step(dtype) * (want.abs() + bound)).all(), err.max().item()
    return y


SIZES = [(1, 1, 1), (1, 1, 16), (1, 16, 128), (3, 5, 7), (16, 64, 128), (17, 100, 144), (16, 8192, 256), (32, 12288, 272),
         (33, 1000, 512), (64, 2048, 384), (65, 65, 65), (100, 300, 1333), (128, 128, 4096), (256, 256, 2048), (777, 1000, 1333),
         (300, 4096, 1024), (1024, 4096, 512), (3000, 2500, 640), (4096, 6144, 256), (2048, 8192, 1040), (5000, 37, 96),
         (40, 40, 131071), (1, 20000, 128), (20000, 1, 128)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_product(size, dtype):
    say(f"int8 {size}")
    check(make(*size, seed=sum(size), bias=size[0] % 2 == 0), dtype)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_largest_sums_are_exact(M):
    """131071 products of -128 by -128: 2^14 short of 2^31, and a number of fp32."""
    say("int8 largest sums")
    K, N = 131071, 33
    d = dict(a=torch.full((M, K), -128, dtype=torch.int8), w=torch.full((N, K), -128, dtype=torch.int8), sa=torch.ones(M),
             sw=torch.ones(N), bias=None)
    y = check(d, torch.float32)
    assert (y == 2.0 ** 31 - 2.0 ** 14).all()
    d["w"].fill_(127)
    check(d, torch.float32)


def test_scales_at_their_limits():
    say("int8 scales")
    x = make(20, 30, 256, bias=False)
    x["sa"][0], x["sa"][1], x["sa"][2] = 0.0, 2.0 ** -100 / 127, float("nan")
    x["sw"][0], x["sw"][1] = 2.0 ** -20, float("inf")
    d = {n: t.cuda() for n, t in x.items() if t is not None}
    y = layer.matmul_int8(d["a"], d["sa"], d["w"], d["sw"], out_dtype=torch.float32).cpu()
    assert y[2].isnan().all() and (y[0, 2:] == 0).all() and not torch.isfinite(y[3:, 1]).any()
    assert torch.isfinite(y[3:, 2:]).all()


def test_unaligned_operands_and_outputs():
    say("int8 unaligned")
    x = make(70, 200, 256)
    for k in (1, 4, 8):
        d = {n: None if t is None else t.cuda() for n, t in x.items()}
        buf = torch.zeros(70 * 256 + 16, dtype=torch.int8, device="cuda")
        a = buf[k:k + 70 * 256].view(70, 256)
        a.copy_(d["a"])
        want = layer.matmul_int8(d["a"], d["sa"], d["w"], d["sw"], bias=d["bias"])
        assert torch.equal(layer.matmul_int8(a, d["sa"], d["w"], d["sw"], bias=d["bias"]), want)
        obuf = torch.full((70 * 200 + 32,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = obuf[k:k + 70 * 200].view(70, 200)
        assert torch.equal(layer.matmul_int8(d["a"], d["sa"], d["w"], d["sw"], bias=d["bias"], out=out), want)
        assert (obuf[:k] == 7).all() and (obuf[k + 70 * 200:] == 7).all()


def test_quantized_weights():
    """Against the unquantized product: half a step of each row's scale per weight."""
    say("int8 weights")
    g = torch.Generator().manual_seed(2)
    w = torch.randn(300, 512, generator=g).cuda()
    w8, sw = layer.quantize_weight_int8(w)
    x = make(9, 300, 512, bias=False)
    a, sa = x["a"].cuda(), x["sa"].cuda()
    y = layer.matmul_int8(a, sa, w8, sw, out_dtype=torch.float32).double()
    av = a.double() * sa.double()[:, None]
    bound = av.abs().sum(1)[:, None] * sw.double() * 0.501
    assert ((y - av @ w.double().t()).abs() <= bound).all()


def test_a_replayed_graph():
    say("int8 graph")
    d = {n: t.cuda() for n, t in make(300, 500, 640).items()}
    run = lambda: layer.matmul_int8(d["a"], d["sa"], d["w"], d["sw"], bias=d["bias"])  # noqa: E731
    run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = run()
    for seed in (1, 2, 3):
        for n, t in make(300, 500, 640, seed=seed).items():
            d[n].copy_(t)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(r, run()), seed


def test_refusals():
    say("int8 refusals")
    d = {n: t.cuda() for n, t in make(4, 6, 32).items()}
    ok = (d["a"], d["sa"], d["w"], d["sw"])
    for i, t in ((0, d["a"].float()), (0, d["a"].view(torch.uint8)), (0, d["a"][:, :31]), (0, None), (1, d["sa"][:3]), (1, None),
                 (1, d["sa"].double()), (2, d["w"][:, :16]), (2, d["w"].t()), (2, None), (3, d["sw"][None]), (3, None),
                 (0, d["a"].cpu()), (2, d["w"].cpu())):
        a = list(ok)
        a[i] = t
        with pytest.raises(PararnnError):
            layer.matmul_int8(*a)
    for kw in (dict(bias=d["bias"][:5]), dict(out_dtype=torch.float16), dict(out=torch.empty(4, 6, device="cuda"))):
        with pytest.raises(PararnnError):
            layer.matmul_int8(*ok, **kw)
    big = torch.zeros(1, 131072, dtype=torch.int8, device="cuda")
    one = torch.ones(1, device="cuda")
    with pytest.raises(PararnnError):
        layer.matmul_int8(big, one, big, one)
