"""The recurrent layer end to end (block.RecurrentBlock): norm, 8-bit gate
projection and recurrence against 64 bits on the values the layer rounds to,
decoding against prefill, gradients against differences, and the refusals of
the operators' Python entry points."""
import numpy as np
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from nonlinear_rnn_solve_newton_amd.binding import PararnnError
from nonlinear_rnn_solve_newton_amd.block import GATES, RecurrentBlock
from tests import layer_reference as R
from tests.helpers import say

pytestmark = pytest.mark.gpu


def make(cell, E, D, seed=0, **kw):
    g = torch.Generator().manual_seed(seed)
    G = GATES[cell]
    norm_w = 1.0 + 0.1 * torch.randn(E, generator=g)
    w = torch.randn(G * D, E, generator=g) / E ** 0.5
    bias = 0.1 * torch.randn(G * D, generator=g)
    coef = torch.randn(D, generator=g) - 4.0 if cell == "gated" else 2 * torch.rand(G, D, generator=g) - 1
    return RecurrentBlock(cell, norm_w.cuda(), w.cuda(), coef.cuda(), bias=bias.cuda(), **kw)


def inputs(B, L, E, seed=1):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, L, E, generator=g).bfloat16().cuda(), 2 * torch.randn(B, L, E, generator=g).bfloat16().cuda())


@pytest.mark.parametrize("cell", list(GATES))
@pytest.mark.parametrize("scale", [torch.float32, torch.float8_e8m0fnu])
def test_forward(cell, scale):
    """Each operator of the layer against 64 bits, at the inputs it got."""
    say(f"block {cell}")
    B, L, E, D = 2, 130, 200, 72
    blk = make(cell, E, D, scale_dtype=scale)
    x, res = inputs(B, L, E)
    out = blk.forward(x, res)
    n = layer.norm_residual(x.view(-1, E), blk.norm_w, residual=res.view(-1, E), scale_dtype=scale)
    assert torch.equal(n["s"].view(B, L, E), out["s"])
    u, _ = blk.gates(x, res)
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    want, e = R.matmul(f64(n["y"].float()), f64(layer.scale_values(n["scale"])), f64(blk.w8.float()),
                       f64(layer.scale_values(blk.sw)), 128, f64(blk.bias), fp32=False)
    got = f64(u).reshape(want.shape)
    assert (np.abs(got - want) <= e + R.BF16_EPS * (np.abs(want) + e)).all()
    # the 8-bit weights and activations stay near the unrounded layer: 2^-4 of a
    # value at most, over sums of 200 terms of random sign
    if cell == "gated":
        v, eh = R.gated(f64(u), f64(blk.coef))["h"]
        assert (np.abs(f64(out["h"]) - v) <= eh + R.BF16_EPS * (np.abs(v) + eh)).all()
    else:
        from oracle import oracle as O
        st = O.newton(cell, u.cpu(), blk.coef.cpu(), K=3)[0]
        assert np.abs(f64(out["h"]) - st[-1]).max() <= 1e-4


def test_prefill_then_decode_is_the_whole_sequence():
    """A prefill of ragged rows, then single steps on a pool of states, against
    one pass over everything."""
    say("block: prefill and decode")
    B, L, T, E, D = 3, 40, 6, 256, 128
    blk = make("gated", E, D)
    x, res = inputs(B, L + T, E)
    whole = blk.forward(x, res)
    pre = blk.forward(x[:, :L].contiguous(), res[:, :L].contiguous())
    pool = torch.zeros(8, D, device="cuda")
    slots = torch.tensor([5, 2, 7], dtype=torch.int32, device="cuda")
    pool[slots.long()] = pre["state"]
    for t in range(L, L + T):
        h, s = blk.step(x[:, t].contiguous(), res[:, t].contiguous(), pool, slots=slots)
        # the same gate inputs (to the order of sums of 128-blocks in bf16), states to 32 bits
        assert torch.allclose(h.float(), whole["h"][:, t].float(), atol=2e-2, rtol=2e-2)
        assert torch.equal(s, whole["s"][:, t])
    assert torch.allclose(pool[slots.long()], whole["state"], atol=2e-2, rtol=2e-2)


def test_backward_against_differences():
    """Directional derivatives of the layer's loss, in 64 bits on the layer's own
    weights without its roundings to 8 bits and bf16, against the gradients:
    both see the same function up to those roundings (2^-4 of a value, averaged
    over thousands of terms), hence 5 %."""
    say("block: gradients against differences")
    B, L, E, D = 2, 96, 128, 64
    blk = make("gated", E, D)
    x, res = inputs(B, L, E)
    g = torch.Generator().manual_seed(5)
    dh = torch.randn(B, L, D, generator=g).bfloat16().cuda()
    ds = torch.randn(B, L, E, generator=g).bfloat16().cuda()
    f = blk.forward(x, res, train=True)
    b = blk.backward(f["ctx"], dh, ds)
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    full = layer.scale_values(blk.sw).repeat_interleave(128, 0)[:3 * D].repeat_interleave(128, 1)[:, :E]
    p = {"x": f64(x) + f64(res), "norm_w": f64(blk.norm_w), "w": f64(blk.w8.float() * full), "bias": f64(blk.bias),
         "coef": f64(blk.coef)}

    def loss(q):
        s = q["x"]
        y = s / np.sqrt((s * s).mean(-1, keepdims=True) + 1e-6) * q["norm_w"]
        u = (y @ q["w"].T + q["bias"]).reshape(B, L, 3, D)
        return (R.gated(u, q["coef"])["h"][0] * f64(dh)).sum() + (s * f64(ds)).sum()

    grads = {"x": "dx", "norm_w": "dnorm_w", "w": "dw", "bias": "dbias", "coef": "dcoef"}
    rng = np.random.default_rng(3)
    for k, gname in grads.items():
        want = f64(b[gname])
        # along the gradient itself, so that the derivative is not a sum that cancels
        d = want / np.linalg.norm(want) + 0.1 * rng.standard_normal(want.shape) / np.sqrt(want.size)
        eps = 1e-5
        up, dn = dict(p), dict(p)
        up[k], dn[k] = p[k] + eps * d, p[k] - eps * d
        num = (loss(up) - loss(dn)) / (2 * eps)
        assert abs(num - (want * d).sum()) <= 0.05 * abs(num), (k, num, (want * d).sum())


def test_refusals():
    say("layer: refused arguments")
    d = torch.device("cuda")
    u, lam = torch.zeros(2, 5, 3, 8, device=d), torch.zeros(8, device=d)
    bad = [
        lambda: layer.gated_scan(u[:, :, :2].contiguous(), lam),
        lambda: layer.gated_scan(u.cpu(), lam),
        lambda: layer.gated_scan(u.half(), lam),
        lambda: layer.gated_scan(u.transpose(0, 1), lam),
        lambda: layer.gated_scan(u, lam.double()),
        lambda: layer.gated_scan(u, lam[:7].contiguous()),
        lambda: layer.gated_scan(u, lam, c=0.0),
        lambda: layer.gated_scan(u, lam, c=float("nan")),
        lambda: layer.gated_scan(u, lam, lengths=torch.zeros(2, device=d, dtype=torch.int64)),
        lambda: layer.gated_scan(u, lam, reset=torch.zeros(2, 4, device=d, dtype=torch.uint8)),
        lambda: layer.gated_scan(u, lam, h0=torch.zeros(2, 8)),
        lambda: layer.gated_scan(torch.zeros(2, 0, 3, 8, device=d), lam),
        lambda: layer.gated_scan(torch.zeros(2, 2000, 3, 8, device=d), lam, ws=torch.zeros(8, dtype=torch.uint8, device=d)),
        lambda: layer.gated_scan_adjoint(u, lam, torch.zeros(2, 5, 8, device=d), None),
        lambda: layer.gated_scan_adjoint(u, lam, torch.zeros(2, 5, 8, device=d), torch.zeros(2, 2, 8, device=d)),
        lambda: layer.gated_scan_adjoint(u, lam, torch.zeros(2, 5, 8, device=d).bfloat16(), torch.zeros(1, 2, 8, device=d)),
        lambda: layer.gated_step(u[:, 0].contiguous(), lam, torch.zeros(1, 8, device=d)),
        lambda: layer.gated_step(u[:, 0].contiguous(), lam, torch.zeros(4, 8, device=d), slots=torch.zeros(3, dtype=torch.int32, device=d)),
        lambda: layer.norm_residual(torch.zeros(2, 8, device=d), torch.ones(7, device=d)),
        lambda: layer.norm_residual(torch.zeros(2, 8, device=d).half(), lam),
        lambda: layer.norm_residual(torch.zeros(2, 8, device=d), lam, scale_dtype=torch.bfloat16),
        lambda: layer.norm_residual(torch.zeros(2, 8, device=d), lam, residual=torch.zeros(2, 8, device=d).bfloat16()),
        lambda: layer.norm_residual(torch.zeros(1, 16385, device=d), torch.ones(16385, device=d)),
        lambda: layer.norm_residual(torch.zeros(2, 8, device=d), lam, eps=-1.0),
        lambda: layer.norm_residual_adjoint(torch.zeros(2, 8, device=d), lam, torch.zeros(2, 9, device=d)),
        lambda: layer.norm_residual_adjoint(torch.zeros(1, 16385, device=d), torch.ones(16385, device=d), torch.zeros(1, 16385, device=d)),
    ]
    a8, w8 = torch.zeros(4, 256, device=d).to(torch.float8_e4m3fn), torch.zeros(130, 256, device=d).to(torch.float8_e4m3fn)
    sa, sw = torch.ones(2, 4, device=d), torch.ones(2, 2, device=d)
    bad += [
        lambda: layer.matmul_fp8(a8.float(), sa, w8, sw),
        lambda: layer.matmul_fp8(a8, sa.t().contiguous(), w8, sw),
        lambda: layer.matmul_fp8(a8, sa, w8, sw.to(torch.float8_e8m0fnu)),
        lambda: layer.matmul_fp8(a8, sa, w8, torch.ones(3, 2, device=d)),
        lambda: layer.matmul_fp8(a8, sa, w8[:, :128].contiguous(), sw),
        lambda: layer.matmul_fp8(a8, sa, w8, sw, bias=torch.ones(129, device=d)),
        lambda: layer.matmul_fp8(a8, sa, w8, sw, out_dtype=torch.float16),
        lambda: layer.matmul_fp8(a8, sa, w8, sw, out=torch.zeros(4, 130, device=d)),
        lambda: layer.quantize_weight(torch.zeros(4, 4), rows=64),
        lambda: layer.quantize_weight(torch.zeros(4, 4), scale_dtype=torch.bfloat16),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(PararnnError):
            f()
            raise AssertionError(f"refusal {i} did not come")
    assert layer.matmul_fp8(a8, sa, w8, sw).shape == (4, 130)
