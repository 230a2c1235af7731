"""Masked experts beside logits that are not numbers, against the definition in
64 bits."""
import numpy as np
import pytest

import _ops_ref as ref
from test_gpu_router import forward, settings, weight_tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,groups", [(16, 1), (64, 1), (64, 4), (60, 4)])
def test_an_expert_masked_by_its_bias_is_not_chosen_for_a_nan(E, groups, score, renorm):
    """A NaN logit ranks above every number, but a bias of -inf masks its expert
    whatever the logit is (and, in a softmax's row, whatever any logit is).
    Groups of 16 are whole lanes of 8 experts, groups of 15 are not."""
    rng = np.random.default_rng(E + groups)
    r = settings(E, 4, score, groups, max(1, groups - 1), renorm=renorm)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32).astype(np.float64)
    bias[[0, 3, 5, 20 % E]] = -np.inf
    l = ref.clear_logits(rng, 6, r, bias)
    l[0, 3] = np.nan                       # at a masked expert
    l[1, 7] = np.nan                       # at one that is not
    l[2, [3, 7]] = np.nan
    l[3] = np.nan                          # everywhere
    l[4, [0, 3]] = [np.nan, -np.inf]
    masked = np.flatnonzero(np.isneginf(bias))
    idx, w, counts = forward(r, l, bias)
    assert not np.isin(idx, masked).any()
    assert np.all(counts[masked] == 0)
    with np.errstate(all="ignore"):
        want_idx, want_w = ref.route(l, r, bias)
    assert np.array_equal(idx, want_idx)
    assert np.array_equal(np.isnan(w), np.isnan(want_w))
    fin = ~np.isnan(want_w)
    tol = np.broadcast_to(weight_tolerance(l), w.shape)
    assert np.all(np.abs(w - want_w)[fin] <= (tol * np.abs(want_w) + 2.0 ** -126)[fin])
