"""DeltaBlock takes the sizes that its parts take, and says so where it is made: on the CPU, where its weights are
laid out as on any device."""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd.binding import PararnnError
from nonlinear_rnn_solve_newton_amd.block import DeltaBlock


def make(E=32, H=1, HV=2, dk=16, dv=8, **kw):
    cols = 2 * H * dk + 2 * HV * dv + 2 * HV
    return DeltaBlock(torch.ones(E), torch.ones(1, 1).expand(cols, E), torch.zeros(HV), torch.ones(dv),
                      torch.ones(1, 1).expand(E, HV * dv), heads=H, dk=dk, **kw)


@pytest.mark.parametrize("dv", [8, 16, 32, 64, 128, 256, 512])
def test_taken(dv):
    assert make(dv=dv).dv == dv and make(HV=1, dv=dv - 1).dv == dv - 1 and make(dk=128, dv=dv).dk == 128
    assert make(alpha=torch.ones(32)).alpha.shape == (32,)


@pytest.mark.parametrize("kw", [dict(dv=72), dict(dv=96), dict(dv=100), dict(dv=192), dict(dv=4), dict(dv=1024), dict(HV=1, dv=513),
                                dict(dk=129), dict(dk=256), dict(HV=64, dv=512), dict(E=16385, dv=8), dict(HV=0), dict(dv=0),
                                dict(HV=1, dv=0), dict(E=0), dict(alpha=torch.ones(31)), dict(alpha=1.0)], ids=str)
def test_refused(kw):
    with pytest.raises(PararnnError):
        make(**kw)
