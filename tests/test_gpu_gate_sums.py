"""What the gated tail's gradient does better than sums in f32: the gradients of scalar factors
lose nothing of a sum over all elements, and the roots are within one unit in the last place.

The inputs make every product exact, so that only the additions count, and the results are
compared bit for bit or within what the root's definition leaves."""
import numpy as np
import pytest
import torch

from dual_epsilon_sandwich_gb300 import mrn
from test_gpu_train import DTYPES, TYPES, Buf, f64

pytestmark = pytest.mark.gpu

BIG = 2.0 ** 28


@pytest.fixture(scope="module", autouse=True)
def library(gpu_lib):
    return gpu_lib


# rows in warps, in a CTA and over clusters, with ends and without, and the kernel for any width;
# at least three turns of a thread (of 8 CTAs an SM, each with 4 to 16 rows where they share warps)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,shift,apart", [
    (90000, 64, 0, 0), (60000, 64, 1, 0), (15000, 512, 0, 0), (15000, 512, 1, 0), (15000, 1024, 0, 0),
    (15000, 1024, 1, 0), (3000, 4096, 0, 0), (3000, 4096, 1, 0), (500, 32768, 0, 0),
    (500, 32768, 1, 0), (15000, 1024, 0, 1)])
def test_scalar_gradients_lose_nothing(rows, n, shift, apart, dtype):
    """A third of the rows adds 2^28 for every element, a third 1 and the last third -2^28: both
    gradients are the number of elements of the middle third.  A sum in f32 has lost the ones by
    the time that it meets them (its steps are 64 at 2^29 and wider beyond), and every partial
    sum of the right one is a whole number below 2^53."""
    assert np.float32(8 * BIG) + np.float32(8) == np.float32(8 * BIG)
    third = rows // 3
    g = torch.Generator(device="cuda").manual_seed(n + shift)
    b = torch.randint(0, 2, (rows, n), generator=g, device="cuda").float() * 2 - 1
    v = torch.full((rows, 1), -BIG, device="cuda")
    v[:third], v[third:2 * third], v[3 * third:] = BIG, 1.0, 0.0
    t = TYPES[dtype]
    ds = Buf((rows, n), t, b * v, shift).t
    b, res = Buf((rows, n), t, b, shift).t, Buf((rows, n), t, b, shift + apart).t
    zero, s = Buf((rows, n), t, torch.zeros(rows, n), shift).t, Buf((rows, n), t, b, shift).t
    db, dr = Buf((rows, n), t, None, shift), Buf((rows, n), t, None, shift)
    one = torch.ones(n, dtype=t, device="cuda")
    gate, scale = one[:1] * 0.5, one[:1] * 2.0
    # the mean of squares is 1 and eps_post far below its last place: xh = b
    got = mrn.norm_gate_residual_norm_backward(zero, b, s, one, one, gate, scale, residual=res,
                                               eps_post=1e-30, dstream=ds, dblock=db.t,
                                               dresidual=dr.t)
    assert db.guards_hold() and dr.guards_hold()
    assert float(got[4]) == third * n and float(got[5]) == third * n
    # each row's share of the residual's gradient is exact as well
    assert torch.equal(got[1], ds * scale)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n,shift", [(200, 256, 0), (200, 256, 1), (250, 1024, 0), (300, 2048, 1),
                                          (300, 4096, 0), (8, 4096, 0), (200, 32768, 0),
                                          (40, 262144, 0)])
def test_roots_within_a_unit(rows, n, shift, dtype):
    """dgate of a gate per row is inv(block_out), and dgamma_pre of column r inv(out_stream) of
    row r, where the incoming gradients have a single one in that row.  Whole numbers make the
    sums of squares exact, and n a power of two their mean; what is left is the sum with eps,
    rounded once (half a unit, half of which reaches the root), and the root within a unit, 2^-23
    of its value at most."""
    g = torch.Generator().manual_seed(rows + n)
    # values of up to 2^k and rows of all scales between 1 and that, n * 2^2k below 2^24
    k = min(4, (24 - n.bit_length()) // 2)
    top = torch.randint(1, 2 ** k + 1, (rows, 1), generator=g).double()
    v = [(torch.rand(rows, n, generator=g).double() * 2 * top - top).round() for _ in range(2)]
    at = torch.arange(rows) % n
    for x in v:
        x[torch.arange(rows), at] = 1.0
    single = torch.zeros(rows, n)
    single[torch.arange(rows), at] = 1.0
    t = TYPES[dtype]
    b, s, one_each = (Buf((rows, n), t, x, shift).t for x in (*v, single))
    ones = torch.ones(n, dtype=t, device="cuda")
    gate = torch.ones(rows, 1, dtype=t, device="cuda")
    zero = Buf((rows, n), t, torch.zeros(rows, n), shift).t

    def call(dn, ds):
        db, dr = Buf((rows, n), t, None, shift), Buf((rows, n), t, None, shift)
        return mrn.norm_gate_residual_norm_backward(dn, b, s, ones, ones, gate, dstream=ds,
                                                    dblock=db.t, dresidual=dr.t)

    tol = 1.01 * (2.0 ** -23 + 2.0 ** -25)
    want = [1.0 / np.sqrt((x.numpy() ** 2).mean(1) + float(np.float32(e)))
            for x, e in zip(v, (1e-8, 1e-5))]
    dgate = f64(call(zero, one_each)[4])[:, 0]
    assert (np.abs(dgate - want[0]) <= tol * want[0]).all(), np.abs(dgate / want[0] - 1).max() * 2 ** 23
    if rows <= n:
        pre = f64(call(one_each, zero)[3])[:rows]
        assert (np.abs(pre - want[1]) <= tol * want[1]).all(), np.abs(pre / want[1] - 1).max() * 2 ** 23
