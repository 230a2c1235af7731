"""The layer for a few tokens: experts masked by their bias beside logits that are not numbers."""
import numpy as np
import pytest

from test_gpu_decode import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(1, 256, 12, 4, 128, 0), (5, 256, 12, 4, 128, 1), (11, 384, 200, 8, 128, 0)])
def test_a_masked_expert_is_not_chosen_for_its_logit(shape):
    """A bias of -inf masks its expert whatever its logit: a NaN, an infinity of either sign (router weights that hold
    one): the bits of the pass with an ordinary row in its place."""
    c = Case(*shape, bias=True)
    c.bias[[0, 3, 5, 9]] = -np.inf
    clean = c.forward()
    c.check_choice(clean[1], clean[2])
    c.x[:, 7] = np.abs(c.x[:, 7]) + 0.5
    want = c.forward()
    c.router[0, 4] = np.nan
    c.router[3, 7], c.router[5, 7] = np.inf, -np.inf
    got = c.forward()
    assert not np.isin(got[1], (0, 3, 5, 9)).any()
    assert all(np.array_equal(a, b) for a, b in zip(got, want))


def test_a_nan_that_is_not_masked_ranks_first():
    c = Case(3, 256, 12, 4, 128, bias=True)
    c.bias[[2, 6]] = -np.inf
    c.router[[2, 4, 6], 1] = np.nan
    out, idx, w = c.forward()
    assert np.all(idx[:, 0] == 4) and not np.isin(idx, (2, 6)).any()
    assert np.all(np.isnan(w)) and np.all(np.isnan(out))
