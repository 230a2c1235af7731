"""The limits of the 4-bit experts' error tell a kernel that rounds its weights
to bf16 from those that do not (on the CPU, the roundings put into the formula)."""
import numpy as np
import pytest

import _ops_ref as ref
import _w4_bounds as bounds
from test_gpu_w4 import Case
from test_gpu_w4_bounds import PATHS


def to_11_bits(v):
    m, e = np.frexp(v)
    return np.ldexp(np.round(m * 2.0 ** 11), e - 11)


def rounded(c, weights):
    """out with the weights rounded as `weights` does, h and out to bf16."""
    T, d, E, k, f, S, group, zeros = c.shape
    G, U, D = (weights(ref.values(*m)) for m in (c.gate, c.up, c.down))
    out = np.zeros((T, d))
    for t in range(T):
        for e, v in [*zip(c.idx[t], c.w[t].astype(np.float64))] + ([(E, 1.0)] if S else []):
            z = G[e] @ c.x[t]
            out[t] += v * (D[e] @ ref.bf16(z / (1 + np.exp(-z)) * (U[e] @ c.x[t])))
    return ref.bf16(out)


@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
@pytest.mark.parametrize("name", list(PATHS))
def test_the_norm_tells_weights_of_8_bits(name, group, zeros):
    T, d, E, k, f, S, tiles = PATHS[name]
    c = Case(min(T, 40), d, E, k, f, S, group, zeros, seed=T + group)
    want, off = bounds.experts(c.x, c.idx, c.w.astype(np.float64), c.gate, c.up, c.down, E, S, tiles)
    size = np.linalg.norm(want)
    right = rounded(c, to_11_bits if tiles else lambda v: v)
    assert np.linalg.norm(right - want) <= bounds.NORM * size
    assert np.all(np.abs(right - want) <= off)
    assert np.linalg.norm(rounded(c, ref.bf16) - want) > bounds.NORM * size
