"""Arguments of the layer's Python entry points that are no tensors at all get
the same error as every other refused one."""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd import layer
from nonlinear_rnn_solve_newton_amd.binding import PararnnError
from tests.helpers import say

pytestmark = pytest.mark.gpu


def test_arguments_that_are_no_tensors():
    say("layer: arguments that are no tensors")
    d = torch.device("cuda")
    u, lam = torch.zeros(2, 2000, 3, 8, device=d), torch.zeros(8, device=d)
    f = layer.gated_scan(u, lam, save=True)
    dh = torch.zeros(2, 2000, 8, device=d)
    x, w = torch.zeros(2, 8, device=d), torch.ones(8, device=d)
    bad = [
        lambda: layer.gated_scan(u, lam, reset=[[0] * 2000] * 2),
        lambda: layer.gated_scan(u, lam, reset=1),
        lambda: layer.gated_scan(u, lam, ws=4096),
        lambda: layer.gated_scan_adjoint(u, lam, dh, f["saved"], reset=True),
        lambda: layer.gated_scan_adjoint(u, lam, dh, f["saved"], ws=bytearray(1 << 20)),
        lambda: layer.gated_scan_adjoint(u, lam, None, f["saved"]),
        lambda: layer.gated_scan(u, None),
        lambda: layer.gated_step(u[:, 0].contiguous(), None, torch.zeros(2, 8, device=d)),
        lambda: layer.norm_residual(x, None),
        lambda: layer.norm_residual_adjoint(x, None, x),
        lambda: layer.norm_residual_adjoint(x, w, None),
        lambda: layer.norm_residual_adjoint(x, w, x, ws=1),
        lambda: layer.quantize_weight([[1.0]]),
    ]
    for i, c in enumerate(bad):
        with pytest.raises(PararnnError):
            c()
            raise AssertionError(f"refusal {i} did not come")
