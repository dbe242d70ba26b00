"""8-bit values of the norm's output: the quotient y / scale, rounded to nearest
even, bit for bit."""
import numpy as np
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from tests.helpers import say

pytestmark = pytest.mark.gpu


def quotients_at_ties(seed, blocks):
    """Rows of 128 weights: a largest magnitude m, and values whose fp32 quotient
    by m / 448 lies at a tie of e4m3 or next to it."""
    rng = np.random.default_rng(seed)
    q = torch.arange(0, 0x7f, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()  # 0 to 448
    ties = (q[:-1] + q[1:]) / 2
    m = np.exp(rng.uniform(-3, 3, blocks)).astype(np.float32)
    scale = m / np.float32(448)
    v = (ties[rng.integers(0, len(ties), (blocks, 128))] * scale.astype(np.float64)[:, None]).astype(np.float32)
    for _ in range(2):  # up to two ulp to either side
        v = np.nextafter(v, np.where(rng.random(v.shape) < 0.4, np.float32(np.inf), np.where(
            rng.random(v.shape) < 0.5, np.float32(-np.inf), v)).astype(np.float32))
    v *= np.where(rng.random(v.shape) < 0.5, -1, 1).astype(np.float32)
    v = np.clip(v, -m[:, None], m[:, None])
    v[:, 17] = m
    return v.reshape(-1), scale


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [128, 1024, 4096])
def test_quotient_is_rounded_once(dtype, D):
    """Rows of +-1 have a root mean square of 1, so that y is the weights, exactly."""
    say(f"norm to 8 bits at ties, {D} columns")
    for seed in range(4):
        w, scale = quotients_at_ties(seed, D // 128)
        sign = torch.from_numpy(np.random.default_rng(seed).integers(0, 2, (3, D)) * 2.0 - 1.0)
        y = sign.numpy().astype(np.float32) * w
        quotient = (y.reshape(3, -1, 128) / scale[:, None]).reshape(3, D)  # fp32, correctly rounded
        want = torch.from_numpy(quotient).to(torch.float8_e4m3fn).view(torch.uint8)
        r = layer.norm_residual(sign.to(dtype).cuda(), torch.from_numpy(w).cuda(), eps=0.0, scale_dtype=torch.float32)
        assert np.array_equal(r["scale"].cpu().numpy(), np.repeat(scale[:, None], 3, axis=1))
        got = r["y"].view(torch.uint8).cpu()
        assert torch.equal(got, want), f"{int((got != want).sum())} of {want.numel()} differ"
