"""The 8-bit paged attention on the GPU within bounds taken row by row (tests/attn_util.py), at options, exponents
and magnitudes far from the usual ones."""
import pytest
import torch

from tests.attn_util import check_rows, extreme_case
from tests.test_gpu_attn import BF, F32, Case, call, random_tree

pytestmark = pytest.mark.gpu

MODES = [("decode", 1), ("verify", 4), ("tree", 4), ("extend", 0)]


def lens_of(mode, D, n):
    return [90, 1, 30, 7][:n] if mode == "extend" else [D] * n


def attend(c, mode, D, ref=None, **kw):
    """One call and its check; kw: options of `call`, ref: those options under the definition's names."""
    parents = random_tree(c.rng, len(c.kv), D) if mode == "tree" else None
    got = call(c, "verify" if mode == "tree" else mode, D=D, parents=parents, **kw)
    check_rows(c, got, parents=parents, **(ref or {}))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mode,D", MODES)
@pytest.mark.parametrize("hq,hkv", [(4, 2), (60, 1)])  # the kernel of split tokens (extend aside) and that of tiles
@pytest.mark.parametrize("cap", [1e-39, 0.5, 256.0, 257.0, 1e4, 1e6, 1e30, 3e38])
def test_caps_of_any_size(dtype, mode, D, hq, hkv, cap):
    """A cap far above the scores changes nothing, and one far below them makes them equal in size: the error does not
    grow with the cap."""
    c = Case(lens_of(mode, D, 4), [700, 20, 130, 257], hq, hkv, 128 if hq == 4 else 64, 32, dtype, seed=51)
    c.q[0, 1] = 0.0
    attend(c, mode, D, dict(cap=cap), logit_cap=cap)
    attend(c, mode, D, dict(cap=cap, window=100, slopes=[0.1] * hq), logit_cap=cap, window=100, slopes=[0.1] * hq)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mode,D", MODES)
@pytest.mark.parametrize("hq,hkv", [(4, 2), (60, 1)])
@pytest.mark.parametrize("power", [123, 80, -80, -118])
def test_queries_of_any_magnitude(dtype, mode, D, hq, hkv, power):
    """Queries at both ends of their type's range, under a scale that brings the scores back to ordinary ones."""
    c = Case(lens_of(mode, D, 3), [300, 20, 130], hq, hkv, 64 if hq == 4 else 128, 16, dtype, seed=52,
             qscale=1.5 * 2.0 ** power)
    scale = 0.1 * 2.0 ** -power
    attend(c, mode, D, dict(scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mode,D", MODES)
@pytest.mark.parametrize("hq", [4, 100])
def test_exponents_far_apart(dtype, mode, D, hq):
    attend(extreme_case(Case, lens_of(mode, D, 2), dtype, hq), mode, D)
