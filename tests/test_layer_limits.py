"""Sizes whose launch would have 2^32 threads or more are refused before
anything is launched: a launch's size in threads is a 32-bit number, and a
larger one would run as its low 32 bits, without an error. CPU only; the
pointers are never dereferenced."""
import ctypes

import pytest

from nonlinear_rnn_solve_newton_amd import layer
from nonlinear_rnn_solve_newton_amd.binding import BF16, F32
from tests.test_layer_abi import P, lib  # noqa: F401

EINVAL, OK = -1, 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("adj", [0, 1])
def test_gated_scan(lib, adj, dtype):  # noqa: F811
    """512 threads per 32 or 64 channels of a row and per 96 steps or more."""
    n = ctypes.c_size_t()

    def size(B, L, D):
        return lib.pararnn_gated_workspace_bytes(adj, ctypes.byref(layer.GatedOpts(B, L, D, dtype, 8.0, None, None)),
                                                 ctypes.byref(n))

    most = (2 ** 32 - 1) // 512
    assert size(most - 8, 1, 1) == OK and size(most - 8, 1, 32) == OK
    assert size(most + 2, 1, 1) == EINVAL and size(2 ** 30, 1, 1) == EINVAL
    assert size(2 ** 20, 1, 1024) == EINVAL  # 2^24 workgroups or more
    assert size(1, 2 ** 31 - 4096, 1) == (EINVAL if adj or dtype == BF16 else OK)  # 96, 128 and 256 steps a workgroup
    o = layer.GatedOpts(most + 2, 1, 1, dtype, 8.0, None, None)
    if adj:
        rc = lib.pararnn_gated_scan_adjoint(P(1), P(1), P(1), P(1), None, P(1), None, None, P(2), 1 << 50,
                                            ctypes.byref(o), None)
    else:
        rc = lib.pararnn_gated_scan(P(1), P(1), None, P(1), None, None, P(2), 1 << 50, ctypes.byref(o), None)
    assert rc == EINVAL


def test_gated_step(lib):  # noqa: F811
    def step(B, D, dtype, off=0):
        u = ctypes.c_void_p(4096 + off)
        return lib.pararnn_gated_step(u, P(1), None, P(1), P(1), B, D, B, dtype, 8.0, None)

    for dtype in (F32, BF16):
        assert step(2 ** 20, 4099, dtype) == EINVAL  # a thread per channel
        assert step(2 ** 24, 1024, dtype) == EINVAL  # a thread per 4 channels: 2^32
        assert step(2 ** 22, 1024, dtype, off=4 if dtype == F32 else 2) == EINVAL  # per channel, by the alignment


def test_matmul(lib):  # noqa: F811
    def mm(M, N, K, dt):
        o = layer.MatmulOpts(M, N, K, 128, 0, dt)
        return lib.pararnn_matmul_fp8(P(1), P(1), P(1), P(1), None, P(1), ctypes.byref(o), None)

    for dt in (F32, BF16):
        assert mm(1, 2 ** 30, 16, dt) == EINVAL  # few rows: 512 threads per 64 columns
        assert mm(2 ** 20, 2 ** 20, 17, dt) == EINVAL  # 256 threads per 128 x 128
    assert mm(2 ** 20, 2 ** 20, 16, BF16) == EINVAL
