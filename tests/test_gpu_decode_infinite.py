"""The layer for a few tokens: what an infinite weight of a chosen expert reaches."""
import numpy as np
import pytest

from test_gpu_decode import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [4, 11])
def test_an_infinite_weight_stays_in_its_row(T):
    """w_down's infinities make their own output columns, of the tokens that chose their expert, infinite or NaN."""
    c = Case(T, 256, 8, 2, 256)
    c.idx[:] = [[i % 7, 7] if i % 3 == 0 else [i % 7, (i + 1) % 7] for i in range(T)]
    clean = c.routed()
    c.down[7, 2, 9], c.down[7, 130, 0] = np.inf, -np.inf
    got = c.routed()
    hit = np.zeros(got.shape, dtype=bool)
    hit[np.ix_((c.idx == 7).any(1), (2, 130))] = True
    assert hit.any() and not np.isfinite(got[hit]).any()
    assert np.array_equal(got[~hit], clean[~hit])
