"""Repeated calls of the delta rule give the same bits, over kernels of many workgroups that
run beside each other in ever new orders, and the gates' gradients hold both halves of the pairs' matrix."""
import pytest
import torch

from tests.helpers import say
from tests.test_gpu_delta import DT, check, cuda, make, reference, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(8, 320, 4, 8, 64, 64), (8, 320, 8, 8, 128, 128), (4, 320, 2, 6, 72, 100)], ids=str)
def test_every_gradient_repeats(shape, dtype):
    say(f"delta gradients repeat {shape} {dtype}")
    x = cuda(make(*shape, DT[dtype], seed=11))
    want = run(x)
    for _ in range(12):
        got = run(x)
        for n in want:
            assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dims", [(64, 64), (128, 128)], ids=str)
def test_the_decays_gradient_through_the_keys(dims, dtype):
    """q = 0 and no weight on the last state's own part: all that a decay's gradient holds goes through what keys
    read of each other's values (the second half of the pairs' matrix) and through the states."""
    say(f"delta decays through keys {dims} {dtype}")
    dk, dv = dims
    x = make(2, 192, 1, 2, dk, dv, DT[dtype], seed=5, lam=-4.0)
    x["q"][:] = 0.0
    x["k"][:] = x["k"][:, :1] + 0.25 * x["k"]  # keys of one direction: their products are large
    want = reference(x)
    assert want["dgates"][:, :, 0].abs().max() > 1e-3 and want["dlam"].abs().max() > 1e-3
    check(run(cuda(x)), want, DT[dtype], dk, dv, 192)
