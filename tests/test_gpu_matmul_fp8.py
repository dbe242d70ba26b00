"""GPU parity of the 8-bit product with block scales (layer.matmul_fp8) against
64 bits, every element within the bound of its arithmetic."""
import numpy as np
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from tests import layer_reference as R
from tests.helpers import say

pytestmark = pytest.mark.gpu

SC = {"f32": torch.float32, "e8m0": torch.float8_e8m0fnu}
OUT = {"f32": torch.float32, "bf16": torch.bfloat16}


def values(s):
    s = s.cpu()
    return s.double().numpy() if s.dtype == torch.float32 else 2.0 ** (s.view(torch.uint8).numpy().astype(float) - 127)


def draw(M, N, K, scale, rows, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))
    x[:, ::37] *= 12.0
    a, sa = layer.quantize_weight(x, rows=1, scale_dtype=SC[scale])  # per row and 128 columns
    sa = sa.view(torch.uint8).t().contiguous().view(SC[scale]) if scale == "e8m0" else sa.t().contiguous()
    w, sw = layer.quantize_weight(torch.randn(N, K, generator=g) / K ** 0.5, rows=rows, scale_dtype=SC[scale])
    return a, sa, w, sw, torch.randn(N, generator=g)


def check(a, sa, w, sw, bias, rows, out, got):
    v, e = R.matmul(a.double().numpy(), values(sa), w.double().numpy(), values(sw), rows,
                    None if bias is None else bias.double().numpy(), fp32=out == "f32")
    tol = e + (R.BF16_EPS * (np.abs(v) + e) if out == "bf16" else 0.0)
    err = np.abs(got.cpu().double().numpy() - v)
    assert (err <= tol).all(), f"{int((~(err <= tol)).sum())} of {err.size} outside, worst {np.nanmax(err / tol):.3g} bounds"


# one element, single rows and columns, few rows, sizes next to the tiles,
# K below, at and next to the blocks of 128 and the 16-byte pieces
SHAPES = [(1, 1, 1), (1, 200, 256), (3, 17, 40), (16, 256, 512), (5, 130, 127), (16, 100, 128), (17, 64, 129),
          (33, 128, 144), (64, 512, 1024), (65, 300, 384), (130, 129, 400), (127, 1000, 250), (256, 256, 256),
          (257, 384, 1040), (300, 520, 333)]
IDS = ["x".join(map(str, s)) for s in SHAPES]


@pytest.mark.parametrize("scale", list(SC))
@pytest.mark.parametrize("out", list(OUT))
@pytest.mark.parametrize("rows", [128, 1])
@pytest.mark.parametrize("M,N,K", SHAPES, ids=IDS)
def test_matmul(scale, out, rows, M, N, K):
    say(f"matmul {M}x{N}x{K} {scale} rows={rows} -> {out}")
    a, sa, w, sw, bias = draw(M, N, K, scale, rows, M + N + K)
    d = [t.cuda() for t in (a, sa, w, sw)]
    check(a, sa, w, sw, bias, rows, out, layer.matmul_fp8(*d, bias=bias.cuda(), out_dtype=OUT[out]))
    check(a, sa, w, sw, None, rows, out, layer.matmul_fp8(*d, out_dtype=OUT[out]))


@pytest.mark.parametrize("M,N,K", [(1100, 1300, 384), (2000, 4096, 128), (300, 700, 1333), (70, 96, 4112)])
@pytest.mark.parametrize("scale", list(SC))
def test_many_tiles(scale, M, N, K):
    say(f"matmul {M}x{N}x{K} {scale}")
    a, sa, w, sw, bias = draw(M, N, K, scale, 128, 3)
    got = layer.matmul_fp8(*(t.cuda() for t in (a, sa, w, sw)), bias=bias.cuda())
    check(a, sa, w, sw, bias, 128, "bf16", got)
    again = layer.matmul_fp8(*(t.cuda() for t in (a, sa, w, sw)), bias=bias.cuda())
    assert torch.equal(got, again)


@pytest.mark.parametrize("out", list(OUT))
@pytest.mark.parametrize("scale,rows", [("f32", 128), ("f32", 1), ("e8m0", 128), ("e8m0", 1)])
@pytest.mark.parametrize("M,N", [(1, 8210), (16, 8192), (17, 8210), (1, 12301), (16, 12300), (32, 12300), (64, 2050),
                                 (50, 4100)])
def test_few_rows_of_wide_products(M, N, scale, rows, out):
    """One to four times 16 rows, 16 to 64 columns per workgroup, the last one partly past the end."""
    K = 1296
    say(f"matmul {M}x{N}x{K} {scale} rows={rows} -> {out}")
    a, sa, w, sw, bias = draw(M, N, K, scale, rows, M + N)
    got = layer.matmul_fp8(*(t.cuda() for t in (a, sa, w, sw)), bias=bias.cuda(), out_dtype=OUT[out])
    check(a, sa, w, sw, bias, rows, out, got)


@pytest.mark.parametrize("N", [4140, 4152, 4097])
@pytest.mark.parametrize("scale,rows", [("f32", 128), ("f32", 1), ("e8m0", 128), ("e8m0", 1)])
def test_enough_tiles_for_every_cu(scale, rows, N):
    """The shape that large products take, with partial tiles on every side."""
    say(f"matmul 4100x{N}x400 {scale} rows={rows}")
    M, K = 4100, 400
    a, sa, w, sw, bias = draw(M, N, K, scale, rows, 11)
    got = layer.matmul_fp8(*(t.cuda() for t in (a, sa, w, sw)), bias=bias.cuda())
    check(a, sa, w, sw, bias, rows, "bf16", got)


@pytest.mark.parametrize("M", [8, 200])
@pytest.mark.parametrize("K", [256, 250])
def test_shifted_tensors(M, K):
    say(f"matmul, shifted tensors, {M} rows, K={K}")
    a, sa, w, sw, bias = draw(M, 150, K, "f32", 128, 5)

    def shift(t):
        b = t.view(torch.uint8).reshape(-1) if t.dtype == torch.float8_e4m3fn else t.reshape(-1)
        s = torch.empty(b.numel() + 1, dtype=b.dtype, device="cuda")
        s[1:] = b.cuda()
        return s[1:].view(t.dtype).view(t.shape) if b.dtype == torch.uint8 else s[1:].view(t.shape)

    out = shift(torch.empty(M, 150))
    layer.matmul_fp8(shift(a), shift(sa), shift(w), shift(sw), bias=shift(bias), out_dtype=torch.float32, out=out)
    check(a, sa, w, sw, bias, 128, "f32", out)


@pytest.mark.parametrize("M", [4, 300])
@pytest.mark.parametrize("scale", list(SC))
@pytest.mark.parametrize("K", [256, 272, 137])
def test_a_nan_stays_in_its_row_and_column(M, scale, K):
    """A NaN in row m of a gives row m of y, one in row n of w column n; what
    lies behind a row's end (the next row) does not enter it."""
    say(f"matmul with NaN, {M} rows, K={K}, {scale}")
    N = 150
    a, sa, w, sw, bias = draw(M, N, K, scale, 128, 7)
    ab, wb = a.view(torch.uint8).clone(), w.view(torch.uint8).clone()
    ab[2, 0] = 0x7f
    wb[20, 0] = 0xff
    got = layer.matmul_fp8(ab.view(a.dtype).cuda(), sa.cuda(), wb.view(a.dtype).cuda(), sw.cuda(), bias=bias.cuda())
    nan = torch.isnan(got.float()).cpu()
    want = torch.zeros(M, N, dtype=torch.bool)
    want[2], want[:, 20] = True, True
    assert torch.equal(nan, want)
    ref = layer.matmul_fp8(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), bias=bias.cuda())
    assert torch.equal(got[~want.cuda()], ref[~want.cuda()])


def test_offsets_past_32_bits():
    """a of 2^31 + 2^20 bytes: the first and the last rows against 64 bits."""
    say("matmul, large offsets")
    K, N = 65536, 64
    M = 2 ** 15 + 16
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randint(0, 120, (M, K), generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    w = torch.randint(0, 120, (N, K), generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    sa = torch.rand(K // 128, M, generator=g, device="cuda") * 1e-4
    sw = torch.rand(1, K // 128, generator=g, device="cuda") * 1e-4
    y = layer.matmul_fp8(a, sa, w, sw, out_dtype=torch.float32)
    for m in (0, 2 ** 15 - 8, M - 8):
        check(a[m:m + 8].cpu(), sa[:, m:m + 8], w.cpu(), sw, None, 128, "f32", y[m:m + 8])


def test_quantize_weight_round_trip():
    say("quantize_weight")
    w = torch.randn(300, 333, generator=torch.Generator().manual_seed(3))
    for rows in (1, 128):
        for sc in SC:
            q, s = layer.quantize_weight(w, rows=rows, scale_dtype=SC[sc])
            full = np.repeat(np.repeat(values(s), rows, axis=0)[:300], 128, axis=1)[:, :333]
            v = w.double().numpy() / full
            half = np.maximum(2.0 ** -4 * 2.0 ** np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -30))), 2.0 ** -10)
            assert (np.abs(v) <= 448.001).all() and (np.abs(q.double().numpy() - v) <= half * (1 + 1e-5)).all()
