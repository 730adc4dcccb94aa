"""The longest chain of additions in the gated tail's sums over rows, counted from what its workspace
holds, against what the bounds of its tests allow.

A column's sum: the rows of one thread, one after the other (at least eight rows are in work at
once where there are as many); the rows that share a CTA, 128 at most and those only of up to
1031 elements; then a warp of the join adds its share of the partial rows, 32 warps up to 1024
columns and 16 above, and one thread the warps'.  Up to 2048 columns there are eight partial rows
for each SM and four above, where the norms' gradients, for which tests/train_bounds.py spells out
its count, have four."""
import pytest

from dual_epsilon_sandwich_gb300 import _build, mrn
from train_bounds import row_chain


@pytest.fixture(scope="module", autouse=True)
def library():
    _build.build()
    return mrn.lib()


def partial_rows(rows, n):
    """From the workspace: three sets of partial rows, whole slots of eight floats and up to seven
    elements before them, and two scalars of 16 CTAs in 64 bits for each."""
    return mrn.mrn_norm_gate_backward_workspace(rows, n) // (3 * 4 * ((n + 15) // 8 * 8) + 2 * 16 * 8)


@pytest.mark.parametrize("n", (1, 7, 64, 255, 1024, 1025, 1031, 1032, 2048, 2049, 4096, 6656, 65536, 270001))
@pytest.mark.parametrize("rows", (1, 8, 100, 1216, 1500, 16384, 1000000))
def test_row_chain_covers_the_partial_rows(rows, n):
    parts = partial_rows(rows, n)
    assert 1 <= parts <= min(rows, 2048)
    warps = 32 if n <= 1024 else 16
    share_a_cta = 1 if n > 1031 else 128
    chain = 1 + rows / 8 + share_a_cta + -(-parts // warps) + warps
    assert chain <= row_chain(rows), (parts, chain)
