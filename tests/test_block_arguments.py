"""RecurrentBlock's own checks, on the CPU: its weights are laid out on any device."""
import pytest
import torch

from nonlinear_rnn_solve_newton_amd.binding import PararnnError
from nonlinear_rnn_solve_newton_amd.block import RecurrentBlock


def test_refused_weights():
    nw, w, lam = torch.ones(32), torch.zeros(24, 32), torch.zeros(8)
    blk = RecurrentBlock("gated", nw, w, lam)
    assert blk.w8.shape == (24, 32) and blk.D == 8 and blk.E == 32
    bad = [("rnn", nw, w, lam), ("gated", [1.0] * 32, w, lam), ("gated", nw, None, lam), ("gated", nw, w, 1.0),
           ("gated", torch.ones(()), w, lam), ("gated", torch.ones(32, 1), w, lam), ("gated", nw, w[:23], lam),
           ("gated", nw, w[:, :31], lam), ("lstm", nw, w[:22], lam), ("gated", nw, w.int(), lam)]
    for args in bad:
        with pytest.raises(PararnnError):
            RecurrentBlock(*args)


def test_refused_calls_come_before_any_launch():
    blk = RecurrentBlock("gated", torch.ones(32), torch.zeros(24, 32), torch.zeros(8))
    x = torch.zeros(2, 3, 32, dtype=torch.bfloat16)
    for f in (lambda: blk.forward(x[0]), lambda: blk.forward(x[:, :, :16]), lambda: blk.forward(x, x.transpose(0, 1)),
              lambda: blk.forward(x.float(), train=True), lambda: blk.step(x, None, torch.zeros(2, 8)),
              lambda: blk.backward(None, x), lambda: blk.forward(x)):  # the last: host tensors
        with pytest.raises(PararnnError):
            f()
