"""The forms of the gated tail's gradient at the widths where the rule that chooses them changes: a
form that the rule asks for and that was not built is an error of the call."""
import pytest
import torch

from dual_epsilon_sandwich_gb300 import mrn
from test_gpu_gate import check_backward, factors, operands, run_backward
from test_gpu_train import DTYPES, make

pytestmark = pytest.mark.gpu

# slots of eight elements on the lower side of each border
BORDERS = (96, 128, 144, 160, 192, 384, 400, 448, 560, 640, 700, 896, 1024, 4096)


@pytest.fixture(scope="module", autouse=True)
def library(gpu_lib):
    return gpu_lib


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("border", BORDERS)
def test_both_sides_of_each_border(border, dtype):
    """More rows than SMs, so that the rule is asked; rows with ends and without, the residual not
    read, read for a scalar's gradient and for one value per channel."""
    rows = torch.cuda.get_device_properties(0).multi_processor_count + 3
    for slots in (border, border + 1):
        n = 8 * slots
        b, res, g1, g2 = operands(400 + slots, rows, n, dtype)
        s, dn, ds = (make(401 + slots + k, rows, n, dtype) for k in range(3))
        for scale in ("none", "scalar", "channel"):
            gate, alpha = factors(402 + slots, rows, n, dtype, "row", scale)
            for shift in (0, 1):
                launches = mrn.mrn_launch_count()
                got = run_backward(dn, b, s, g1, g2, gate, alpha, res, ds, dtype, shift)
                assert mrn.mrn_launch_count() - launches == 2
                check_backward(got, dn, b, s, g1, g2, gate, alpha, res, ds, dtype,
                               f"{slots} slots, scale {scale}, shift {shift}")
