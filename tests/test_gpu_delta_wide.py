"""Values wider than the keys: dv of several slices of columns, rows that take the widest loads and such that do not."""
import pytest

from tests.helpers import say
from tests.test_gpu_delta import DT, check, cuda, make, reference, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("views", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 200, 1, 2, 128, 512), (1, 130, 2, 2, 64, 256), (1, 100, 1, 3, 128, 192), (1, 90, 1, 1, 40, 488),
                                   (1, 1100, 1, 1, 128, 256)], ids=str)
def test_forward_and_adjoint(shape, dtype, views):
    say(f"delta wide {shape} {dtype} views {views}")
    B, L, H, HV, dk, dv = shape
    x = make(*shape, DT[dtype], seed=dv, views=views, packed=B > 1)
    check(run(cuda(x)), reference(x), DT[dtype], dk, dv, L)
