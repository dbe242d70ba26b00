"""What DeltaBlock.backward refuses, and what it leaves at padded steps."""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd.binding import PararnnError
from tests.helpers import say
from tests.test_gpu_delta_block import inputs, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("residual", [True, False])
def test_gradients_of_another_type_or_place(residual):
    say(f"delta block: refused gradients, residual {residual}")
    blk = make(128, 1, 2, 32, 32, alpha=residual)
    x, res = inputs(2, 10, 128)
    f = blk.forward(x, res if residual else None, train=True)
    for kw in (dict(dx=x.float()), dict(dx=x.half()), dict(dx=x.cpu()), dict(dx=x, ds=x.float()), dict(dx=x, ds=x.cpu()),
               dict(dx=x, dstate=torch.zeros(2, 2, 32, 32)), dict(dx=x, dstate=f["state"].half())):
        with pytest.raises(PararnnError):
            blk.backward(f["ctx"], **kw)


def test_padded_steps_have_no_gradient():
    """Whatever reaches them by the residual stream."""
    say("delta block: padded gradients")
    blk = make(128, 1, 2, 32, 32)
    x, res = inputs(3, 20, 128)
    dx, ds = inputs(3, 20, 128, seed=3)
    lengths = torch.tensor([20, 7, 0], dtype=torch.int32, device="cuda")
    off = torch.arange(20, device="cuda") >= lengths[:, None]
    for r in (res, None):
        f = blk.forward(x, r, lengths=lengths, train=True)
        b = blk.backward(f["ctx"], dx, ds=ds)
        for n in ("dx", "dresidual"):
            if b[n] is not None:
                assert not b[n][off].any() and b[n][~off].any(), n
