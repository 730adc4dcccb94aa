"""Sizes that the training entry points refuse because a byte count leaves 64 bits (no GPU: the
buffers are addresses only, and every call is refused before a launch)."""
import pytest

from dual_epsilon_sandwich_gb300 import _build, mrn
from test_train_host import dln, dlnb, ln, lnb, rmb


@pytest.fixture(scope="module", autouse=True)
def library():
    _build.build()
    return mrn.lib()


@pytest.mark.parametrize("call", (ln, dln, lnb, dlnb, rmb))
@pytest.mark.parametrize("rows", (2 ** 62 - 1, 2 ** 61))
def test_statistics_past_64_bits(call, rows):
    """bf16 rows of one element take two bytes each, their statistics four."""
    assert call(rows=rows, n=1, dt=mrn.MRN_BF16) == mrn.MRN_ERR_INVALID_SIZE
    assert mrn.mrn_launch_count() == 0
