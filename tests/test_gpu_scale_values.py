"""Scales as values: powers of two are exact, and weights are laid out the same
on the card and on the host."""
import numpy as np
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


@pytest.mark.parametrize("scale_dtype", [torch.float32, torch.float8_e8m0fnu])
@pytest.mark.parametrize("rows", [1, 128])
def test_the_same_layout_on_host_and_card(rows, scale_dtype):
    """max / 448 is a correctly rounded quotient on both."""
    say(f"quantize_weight on host and card, rows={rows}")
    g = torch.Generator().manual_seed(1)
    w = torch.randn(700, 900, generator=g) * torch.exp(3 * torch.randn(700, 1, generator=g))
    a, sa = layer.quantize_weight(w, rows=rows, scale_dtype=scale_dtype)
    b, sb = layer.quantize_weight(w.cuda(), rows=rows, scale_dtype=scale_dtype)
    assert torch.equal(sa.view(torch.uint8), sb.cpu().view(torch.uint8))
    assert torch.equal(a.view(torch.uint8), b.cpu().view(torch.uint8))
    if scale_dtype == torch.float32:
        p = torch.nn.functional.pad(w.abs(), (0, 124, 0, -700 % rows)).view(-1, rows, 8, 128)
        want = p.amax(dim=(1, 3)).numpy() / np.float32(448)
        assert np.array_equal(sa.numpy(), want)
