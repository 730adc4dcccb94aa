"""LayerNorm's row statistics on the GPU, held to tight bounds: rows whose mean is far from
zero beside their spread, and constant rows."""
import numpy as np
import pytest
import torch

import train_bounds as tight
import train_reference as ref
from dual_epsilon_sandwich_gb300 import mrn
from test_gpu_train import DTYPES, TYPES, Buf, f64, make, run_layernorm, weights

pytestmark = pytest.mark.gpu

# lanes, warps, one CTA of 1 to 4 slots a thread, few rows and more rows than SMs, clusters,
# and rows that no tile holds
SHAPES = [(4, 33), (200, 129), (5, 768), (300, 1000), (200, 1543), (5, 4095), (200, 4095),
          (200, 4096), (200, 6655), (4, 6656), (200, 6656), (170, 12295), (160, 16384),
          (155, 16391), (3, 33000), (153, 65544), (2, 140001)]


@pytest.fixture(scope="module", autouse=True)
def library(gpu_lib):
    return gpu_lib


def run(x, gamma, beta, eps, dtype, path):
    """(y, mean, rstd) by the row tiles, aligned or not, by the kernel for operands at
    different offsets, or after an add of zeros."""
    if path == "aligned":
        return run_layernorm(x, gamma, beta, eps, dtype)
    if path == "shifted":
        return run_layernorm(x, gamma, beta, eps, dtype, 1)
    rows, n = x.shape
    t = TYPES[dtype]
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    if path == "apart":
        y = mrn.layernorm(Buf((rows, n), t, x, 1).t, gamma.cuda(), beta.cuda(), eps,
                          out=Buf((rows, n), t, None, 2).t, mean=mean, rstd=rstd)
    else:
        s, y = mrn.dropout_add_layernorm(x.cuda(), torch.zeros(rows, n, dtype=t, device="cuda"),
                                         gamma.cuda(), beta.cuda(), eps, 0.0, None, mean=mean,
                                         rstd=rstd)
        assert torch.equal(s.cpu(), x)
    return f64(y), f64(mean), f64(rstd)


PATHS = ("aligned", "shifted", "apart", "added")


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", SHAPES)
def test_constant_rows(rows, n, dtype, path):
    """A row that holds one value of few bits, whose sums are exact in f32 in any order, has that
    value for its mean, and gives beta."""
    values = torch.tensor([3.0, 100.0, 1.0 / 1024, -48.0, -65536.0, 2.0 ** -20, 1000.0])
    if n * 125 >= 2 ** 24:                   # (1000 is 125 times 8, 100 is 25 times 4)
        values = values[:-1]
    x = values[torch.arange(rows) % len(values)][:, None].expand(rows, n).to(TYPES[dtype]).contiguous()
    gamma, beta = weights(1, n, dtype)
    eps = 1e-8
    y, mean, rstd = run(x, gamma, beta, eps, dtype, path)
    assert np.array_equal(mean, f64(x)[:, 0])
    assert np.array_equal(y, np.repeat(f64(beta)[None], rows, 0))
    want = 1 / np.sqrt(float(np.float32(eps)))
    assert (np.abs(rstd / want - 1) <= 8 * ref.U).all()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", (2, 3, 7, 33, 49, 129, 515, 1000, 1543, 2049, 4095, 4099, 6655, 8191,
                               12295, 16391, 33000, 65539, 131071, 140001))
def test_the_mean_is_the_quotient_rounded_once(n, dtype, path):
    """Rows of small whole numbers, whose sums are exact: the mean has the bits of the sum's
    division by n in f32."""
    rows = 200 if n <= 16391 else 40
    g = torch.Generator().manual_seed(n)
    x = (torch.randint(0, 4, (rows, n), generator=g) + torch.arange(rows)[:, None] % 100).to(TYPES[dtype])
    x[1::2] *= -1
    sums = x.double().sum(1).numpy()
    assert (np.abs(sums) < 2 ** 24).all()
    gamma, beta = weights(3, n, dtype)
    _, mean, _ = run(x, gamma, beta, 1e-5, dtype, path)
    assert np.array_equal(mean, (sums.astype(np.float32) / np.float32(n)).astype(np.float64))


def test_the_mean_of_a_row_with_an_infinity():
    """... is that infinity, and the other rows are as they are without it."""
    for n in (33, 1000, 4096, 16391):
        x = make(n, 6, n, "f32")
        x[2, n // 2], x[4, 0], x[5, n - 1] = float("inf"), float("-inf"), float("nan")
        y, mean, _ = run_layernorm(x, *weights(4, n, "f32"), 1e-5, "f32")
        assert mean[2] == np.inf and mean[4] == -np.inf and np.isnan(mean[5])
        assert np.isfinite(mean[[0, 1, 3]]).all() and np.isfinite(y[[0, 1, 3]]).all()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", SHAPES)
@pytest.mark.parametrize("mean,scale", [(1000.0, 0.25), (-30.0, 0.01), (0.0, 1.0), (0.5, 2.0)])
def test_rows_far_from_zero_and_near(rows, n, dtype, path, mean, scale):
    if dtype == "bf16":
        scale = max(scale, abs(mean) / 64)      # (a few of the type's steps)
    x = make(rows + n, rows, n, dtype, scale, mean)
    gamma, beta = weights(2, n, dtype)
    eps = 1e-8
    got = run(x, gamma, beta, eps, dtype, path)
    want, tol = tight.layernorm(f64(x), f64(gamma), f64(beta), float(np.float32(eps)))
    for name, g, w, t, kind in zip(("y", "mean", "rstd"), got, want, tol, (dtype, "f32", "f32")):
        ref.check(g, w, t, kind, name)
