"""The bounds that the GPU tests of the 8-bit attention hold each row to are tight enough to see a row's faults; no GPU."""
import numpy as np
import pytest

from tests.attn_util import bounds, extreme_case
from tests.test_gpu_attn import BF, F32, Case


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[1, 1], [70, 9]])
def test_no_row_could_be_zeros_or_another_heads(dtype, lens):
    """With exponents far apart too.  (The row of queries of 1e4, whose scores of 1e5 fp32 knows to a whole unit, is the
    one that the bound says little about.)"""
    c = extreme_case(Case, lens, dtype)
    out, _, tol, ltol = bounds(c)
    keep = np.ones(out.shape[:2], dtype=bool)
    keep[0, 0] = False
    assert ltol[keep].max() < 1e-2
    assert (np.abs(out) / tol).max(-1)[keep].min() > 100
    assert (np.abs(out - np.roll(out, 1, 1)) / tol).max(-1)[1:].min() > 1


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_lost_exponent_shows(dtype):
    c = extreme_case(Case, [70, 9], dtype)
    out, _, tol, _ = bounds(c)
    c.np["v_exp"][c.table[1, :10]] += 1
    assert (np.abs(bounds(c)[0] - out) / tol).max(-1)[70:].min() > 50
