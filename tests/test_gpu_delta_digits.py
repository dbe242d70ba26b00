"""bf16 outputs of the delta rule are 32-bit results rounded once: inputs for which the exact result is known and
an operand cut to fewer bits than fp32's falls to the other side of a rounding."""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from tests.delta_reference import U
from tests.helpers import say

pytestmark = pytest.mark.gpu
OFF, ON = -200.0, 200.0  # gates whose sigmoid is 0 and 1
DIMS = [(64, 64), (128, 128), (33, 40)]


def one_hot(B, L, H, d, at):
    x = torch.zeros(B, L, H, d)
    x[..., at] = 1.0
    return x


def scan(q, k, v, gates, **kw):
    HV = v.shape[2]
    b = lambda t: t.bfloat16().cuda()  # noqa: E731
    # unit q and k stay what they are: 1 + 1e-30 is 1
    return layer.delta_scan(b(q), b(k), b(v), b(gates), torch.zeros(HV).cuda(), eps=1e-30, scale=1.0, **kw)


@pytest.mark.parametrize("dims", DIMS, ids=str)
def test_the_state_is_read_in_32_bits(dims):
    """Nothing decays, nothing is written and q picks a row: o is that row of the state, rounded. Its values lie
    2^-20 of themselves beside the middle between two bf16 numbers."""
    say(f"delta digits: state {dims}")
    dk, dv = dims
    B, L, HV = 3, 130, 2
    g = torch.Generator().manual_seed(1)
    base = torch.randn(B, HV, dk, dv, generator=g).bfloat16().float().clamp_min(2.0 ** -6)
    ulp = 2.0 ** (torch.floor(torch.log2(base)) - 7)
    side = torch.where(torch.rand(B, HV, dk, dv, generator=g) < 0.5, 1.0, -1.0)
    s0 = base + ulp * (0.5 + side * 2.0 ** -13)  # 21 bits: exact in fp32
    gates = torch.full((B, L, 2, HV), OFF)
    r = scan(one_hot(B, L, HV, dk, 5), one_hot(B, L, HV, dk, 2), torch.randn(B, L, HV, dv, generator=g), gates, s0=s0.cuda())
    assert torch.equal(r["sT"].cpu(), s0)
    assert torch.equal(r["o"].cpu(), s0[:, None, :, 5].bfloat16().expand(B, L, HV, dv))


@pytest.mark.parametrize("dims", DIMS, ids=str)
def test_the_write_strength_counts_in_32_bits(dims):
    """Every step a document whose q is its k: o = b v. b is off by a few roundings, and so are its
    factors and the product: 16 of them, 2^-20; then half a step of bf16."""
    say(f"delta digits: write strength {dims}")
    dk, dv = dims
    B, L, HV = 8, 128, 2
    g = torch.Generator().manual_seed(2)
    gates = torch.randn(B, L, 2, HV, generator=g).bfloat16()
    v = torch.randn(B, L, HV, dv, generator=g).bfloat16()
    key = one_hot(B, L, HV, dk, 3)
    o = scan(key, key, v, gates, reset=torch.ones(B, L, dtype=torch.uint8, device="cuda"))["o"].cpu().double()
    want = gates[:, :, 1].double().sigmoid()[..., None] * v.double()
    half = 2.0 ** (torch.floor(torch.log2(want.abs())) - 8)
    assert ((o - want).abs() <= half + 16 * U * want.abs()).all()


@pytest.mark.parametrize("dims", DIMS, ids=str)
def test_the_values_count_in_32_bits(dims):
    """Documents of two steps with one key, the second written in full: what it writes replaces what the first
    wrote, and o is its v. v_2 is 2^-9 to 2^-8 of v_1, so half a step of bf16 of it is 2^-18 of v_1; the difference
    b_2 (v_2 - b_1 v_1) + b_1 v_1 is off by 8 roundings of v_1, 2^-21."""
    say(f"delta digits: values {dims}")
    dk, dv = dims
    B, L, HV = 8, 128, 2
    g = torch.Generator().manual_seed(3)
    gates = torch.randn(B, L, 2, HV, generator=g)
    gates[:, :, 0] = OFF
    gates[:, 1::2, 1] = ON
    v = 1.0 + torch.rand(B, L, HV, dv, generator=g)
    v = torch.where(torch.rand(B, L, HV, dv, generator=g) < 0.5, v, -v).bfloat16().float()
    v[:, 1::2] *= 2.0 ** -8
    reset = torch.zeros(B, L, dtype=torch.uint8)
    reset[:, ::2] = 1
    key = one_hot(B, L, HV, dk, 7)
    o = scan(key, key, v, gates, reset=reset.cuda())["o"].cpu()
    assert torch.equal(o[:, 1::2], v[:, 1::2].bfloat16())
