"""Results do not depend on what the workspace held: it is filled with NaN, and one of the adjoint's size
serves both directions."""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from tests.helpers import say
from tests.test_gpu_delta import DT, GRADS, cuda, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 8, 8), (5, 150, 2, 4, 33, 21), (3, 1100, 1, 2, 72, 100), (1, 2500, 2, 2, 64, 64),
                                   (5, 1030, 1, 1, 128, 128)], ids=str)
def test_whatever_the_workspace_holds(shape, dtype):
    say(f"delta workspace {shape} {dtype}")
    B, L, H, HV, dk, dv = shape
    x = make(*shape, DT[dtype], seed=L, packed=B > 1, lam=-6.0)
    if B > 3 and L > 1000:
        x["lengths"] = torch.tensor([0, 256, 257, 1000, L], dtype=torch.int32)
    d = cuda(x)
    args = (d["q"], d["k"], d["v"], d["gates"], d["lam"])
    opt = dict(lengths=d["lengths"], reset=d["reset"])
    need = layer._delta_bytes(1, *shape, layer._DTYPE[DT[dtype]])
    assert need >= layer._delta_bytes(0, *shape, layer._DTYPE[DT[dtype]])

    def call(fill):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        f = layer.delta_scan(*args, s0=d["s0"], save=True, ws=ws, **opt)
        ws.fill_(fill)
        b = layer.delta_scan_adjoint(*args, d["do"], f["saved"], dsT=d["dsT"], want_ds0=True, ws=ws, **opt)
        return {"o": f["o"], "sT": f["sT"], **{n: b[n] for n in GRADS}}

    a, b = call(0), call(255)
    for n in a:
        assert torch.isfinite(b[n]).all() and torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,group,pre", [(3, 100, None, True), (5000, 1000, None, True), (777, 1024, 128, False),
                                           (9, 360, 72, False), (40, 9000, None, True), (6, 96, 32, True)])
def test_the_norms_adjoint(N, D, group, pre, dtype):
    say(f"norm_block workspace {N} {D} {group} {dtype}")
    g = torch.Generator().manual_seed(N)
    t = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    dt = DT[dtype]
    x, gate, s, dy = (t(N, D).to(dt) for _ in range(4))
    kw = dict(w=t(group or D), gate=gate, group=group, **(dict(s=s, alpha=t(D), w_next=t(D)) if pre else {}))
    need = layer._norm_block_bytes(N, D, group or D, layer._DTYPE[dt], pre)
    a, b = (layer.norm_block_adjoint(x, dy, ws=torch.full((need,), fill, dtype=torch.uint8, device="cuda"), **kw) for fill in (0, 255))
    for n in a:
        if n != "ws" and a[n] is not None:
            assert torch.isfinite(b[n]).all() and torch.equal(a[n], b[n]), n
