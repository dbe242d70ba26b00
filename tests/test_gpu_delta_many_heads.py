"""Many value heads to one head of q and k, with rows that have no steps in some of their chunks."""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from tests.helpers import say
from tests.test_gpu_delta import DT, check, cuda, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("HV", [512, 513, 1100])
def test_gradients_of_chunks_without_steps(HV, dtype):
    """Whatever the workspace holds before the call."""
    say(f"delta {HV} value heads {dtype}")
    B, L, dk, dv = 3, 70, 8, 4
    x = make(B, L, 1, HV, dk, dv, DT[dtype], seed=HV)
    x["lengths"] = torch.tensor([0, L, 60], dtype=torch.int32)
    d = cuda(x)
    args = (d["q"], d["k"], d["v"], d["gates"], d["lam"])
    f = layer.delta_scan(*args, s0=d["s0"], lengths=d["lengths"], save=True)
    need = layer._delta_bytes(1, B, L, 1, HV, dk, dv, layer._DTYPE[DT[dtype]])
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN in every float
    b = layer.delta_scan_adjoint(*args, d["do"], f["saved"], dsT=d["dsT"], lengths=d["lengths"], want_ds0=True, ws=ws)
    check({**b, "o": f["o"], "sT": f["sT"]}, reference(x), DT[dtype], dk, dv, L)
