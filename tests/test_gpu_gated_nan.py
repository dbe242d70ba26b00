"""The gated recurrence where a gate input is not a number: every value and
gradient that the formula makes NaN is NaN, and the others keep their bits."""
import numpy as np
import pytest
import torch

from tests import layer_reference as R
from tests.helpers import say
from tests.test_gpu_gated import draw, run, to64

pytestmark = pytest.mark.gpu


# one workgroup per sequence; chunks, with two channels per lane and with one
@pytest.mark.parametrize("L,D", [(120, 8), (1200, 66), (1200, 67)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [0, 1, 2])
def test_nan_gate(gate, dtype, L, D):
    say(f"gated scan {dtype} {L}x{D}: NaN in gate {gate}")
    x = draw(1, L, D, dtype, 3)
    x["reset"] = torch.zeros(1, L, dtype=torch.uint8)
    x["reset"][0, 40] = x["reset"][0, 100] = 1
    x["u"][0, 70, gate, 5] = 0.0
    clean = run(x)
    x["u"][0, 70, gate, 5] = float("nan")
    got = run(x)
    want = R.gated(**to64({k: x[k] for k in ("u", "lam", "h0", "reset", "dh", "dhT")}))
    for k in got:
        nan = torch.isnan(got[k])
        assert np.array_equal(nan.cpu().numpy(), np.isnan(want[k][0])), k
        assert torch.equal(got[k][~nan], clean[k][~nan]), k
