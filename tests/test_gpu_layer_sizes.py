"""Sizes past 32 bits, which the library takes as 32-bit numbers: refused, not cut to their low bits."""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from nonlinear_rnn_solve_newton_amd.binding import PararnnError
from tests.helpers import say

pytestmark = pytest.mark.gpu
N = 2 ** 32 + 3


def empty(dtype, *shape):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def refused(what, f, *args, **kw):
    say(f"layer sizes: {what}")
    with pytest.raises(PararnnError, match="2147483647"):
        f(*args, **kw)
    torch.cuda.synchronize()


def test_rows_of_the_products():
    one = torch.ones(1, 1, dtype=torch.int8, device="cuda")
    s1 = torch.ones(1, device="cuda")
    refused("int8 rows", layer.matmul_int8, empty(torch.int8, N, 1), empty(torch.float32, N), one, s1)
    refused("int8 columns", layer.matmul_int8, one, s1, empty(torch.int8, N, 1), empty(torch.float32, N))
    w8, sw = layer.quantize_weight(torch.ones(1, 1, device="cuda"))
    refused("fp8 rows", layer.matmul_fp8, empty(torch.float8_e4m3fn, N, 1), empty(torch.float32, 1, N), w8, sw)


def test_steps_and_requests():
    bf, f = torch.bfloat16, torch.float32
    lam = torch.zeros(1, device="cuda")
    q = empty(bf, 1, N, 1, 1)
    refused("delta steps", layer.delta_scan, q, q, q, empty(bf, 1, N, 2, 1), lam)
    q = q.view(N, 1, 1, 1)
    refused("delta rows", layer.delta_scan, q, q, q, empty(bf, N, 1, 2, 1), lam)
    one = empty(bf, 1, 1, 1)
    refused("delta pool", layer.delta_step, one, one, one, empty(bf, 1, 2, 1), lam, empty(f, N, 1, 1, 1))
    refused("gated steps", layer.gated_scan, empty(bf, 1, N, 3, 1), lam)
    refused("gated pool", layer.gated_step, empty(bf, 1, 3, 1), lam, empty(f, N, 1))


def test_columns_of_the_norms():
    x, w = empty(torch.bfloat16, 1, N), empty(torch.float32, N)
    refused("norm columns", layer.norm_residual, x, w)
    refused("norm adjoint columns", layer.norm_residual_adjoint, x, w, x)
    refused("norm_block columns", layer.norm_block, x, w=w)
    refused("norm_block adjoint columns", layer.norm_block_adjoint, x, x, w=w)


def test_the_largest_size_is_taken():
    """2^31 - 257 rows of one column: within the product's limits."""
    say("layer sizes: largest")
    M = 2 ** 31 - 257
    a, sa = torch.ones(M, 1, dtype=torch.int8, device="cuda"), torch.full((M,), 0.5, device="cuda")
    y = layer.matmul_int8(a, sa, torch.full((1, 1), 3, dtype=torch.int8, device="cuda"), torch.full((1,), 2.0, device="cuda"))
    assert y.shape == (M, 1) and bool((y == 3.0).all())
