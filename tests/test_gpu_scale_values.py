"""Scales as values: powers of two are exact, and weights are laid out the same
on the card and on the host."""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from tests.helpers import say

pytestmark = pytest.mark.gpu


def test_values_of_every_e8m0_scale():
    say("scale values, e8m0")
    bits = torch.arange(256, dtype=torch.uint8)
    want = (2.0 ** (bits.double() - 127)).float()  # each of them, 2^-127 too, is an fp32 value
    want[255] = float("nan")
    for dev in ("cpu", "cuda"):
        got = layer.scale_values(bits.to(dev).view(torch.float8_e8m0fnu)).cpu()
        assert got.dtype == torch.float32
        assert torch.equal(got.view(torch.int32)[:255], want.view(torch.int32)[:255]), dev
        assert torch.isnan(got[255]), dev


def test_weights_at_ties_of_their_8_bits():
    """Blocks whose scale is each power of two in turn, holding values half way
    between two e4m3 values: the quotient is exact, and goes to the even one."""
    say("quantize_weight at ties, e8m0")
    q = torch.arange(0, 0x7f, dtype=torch.uint8).view(torch.float8_e4m3fn).float()  # 0 to 448
    ties = torch.cat([(q[:-1] + q[1:]) / 2, q[-1:], q[-1:]])
    scale = 2.0 ** torch.arange(-100, 100).double()
    w = (ties.double() * scale[:, None]).float()  # one row of 128 per scale
    want = ties.to(torch.float8_e4m3fn).view(torch.uint8).expand(len(scale), 128)
    for dev in ("cpu", "cuda"):
        w8, sw = layer.quantize_weight(w.to(dev), rows=1, scale_dtype=torch.float8_e8m0fnu)
        assert torch.equal(sw.cpu().view(torch.uint8)[:, 0].int(), torch.arange(27, 227).int()), dev
        got = w8.cpu().view(torch.uint8)
        assert torch.equal(got, want), f"{dev}: {int((got != want).sum())} of {want.numel()} differ"
