"""The norm of lists that are mostly zeros: blocks of zeros of either sign are left out, a value among
them is not, however small its square is."""
import math

import pytest
import torch

from dual_epsilon_sandwich_gb300 import mrn
from test_gpu_grad_norm import check_norm
from test_gpu_train import TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library(gpu_lib):
    return gpu_lib


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("value", (1.0, 2.0 ** -60, 2.0 ** -100))
def test_one_value_among_zeros(value, dtype):
    """At the ends and inside of whole steps of a CTA, and in the slots behind the last whole one;
    a power of two, whose norm is exact."""
    count = 5 * 16384 + 13
    t = torch.zeros(count, dtype=TYPES[dtype], device="cuda")
    t[1::2] = -0.0
    assert float(mrn.grad_norm([t])) == 0.0
    for at in (0, 7, 8, 2047, 2048, 8 * 256 * 3 + 5, 16383, 16384, 3 * 16384 + 1234, count - 14,
               count - 13, count - 1):
        t[at] = -value
        assert float(mrn.grad_norm([t])) == value, at
        t[at] = 0.0


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_rows_of_zeros_beside_others(dtype):
    """An embedding's gradient of which a few rows are not zero, some of them tiny, in a list and
    clipped."""
    g = torch.Generator().manual_seed(5)
    t = torch.zeros(3001, 320)
    t[::97] = torch.randn(31, 320, generator=g)
    t[5::389] = 1e-25 * torch.randn(8, 320, generator=g)
    t = t.to(TYPES[dtype])
    other = torch.randn(1000, generator=g).to(TYPES[dtype])
    grads = [t.cuda(), other.cuda(), torch.zeros(70001, dtype=TYPES[dtype], device="cuda")]
    want = check_norm(mrn.grad_norm(grads), grads)
    norm, out = mrn.clip_grad_norm(grads, 0.5 * want, out=[torch.empty_like(v) for v in grads])
    check_norm(norm, grads)
    assert math.isclose(check_norm(mrn.grad_norm(out), out), 0.5 * want, rel_tol=2.0 ** -8)
    assert torch.equal(out[0] != 0, grads[0] != 0) and not out[2].any()
