"""The range of the gated tail's gradient: a row's sums are of products of its operands as they are, and
the gradients hold the usual bounds as long as those are numbers of f32's normal range."""
import pytest

from test_gpu_gate import check_backward, factors, operands, run_backward
from test_gpu_train import DTYPES, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library(gpu_lib):
    return gpu_lib


def scaled(t, by):
    return (t.double() * by).to(t.dtype)


# dnormed, dstream, block_out, out_stream: products of two between 1e-34 and 1e34, which a few
# thousand elements leave inside of f32's 1e-38 to 3e38
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", (33, 1024, 4097, 6656))
@pytest.mark.parametrize("by", [(1e18, 1.0, 1e16, 1.0), (1.0, 1e17, 1e17, 1.0), (1e17, 1e17, 1.0, 1e17),
                                (1.0, 1.0, 1e17, 1e17), (1e-17, 1e-17, 1e-17, 1.0),
                                (1e-17, 1e-20, 1.0, 1e-17)])
def test_large_and_small_operands(by, n, dtype):
    rows = 9
    b, res, g1, g2 = operands(500 + n, rows, n, dtype)
    s, dn, ds = (make(501 + n + k, rows, n, dtype) for k in range(3))
    dn, ds, b, s = (scaled(t, k) for t, k in zip((dn, ds, b, s), by))
    for pair in (("scalar", "scalar"), ("channel", "channel"), ("row", "none")):
        gate, scale = factors(502, rows, n, dtype, *pair)
        got = run_backward(dn, b, s, g1, g2, gate, scale, res, ds, dtype)
        check_backward(got, dn, b, s, g1, g2, gate, scale, res, ds, dtype, f"{by} {pair}")
