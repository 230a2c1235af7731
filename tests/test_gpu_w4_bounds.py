"""The 4-bit experts within the roundings that each kind of kernels makes, and
at the ends of the ranges that they take."""
import numpy as np
import pytest

import _ops_ref as ref
import _w4_bounds as bounds
from test_gpu_w4 import Case

pytestmark = pytest.mark.gpu

#: T, d, E, k, f, S and whether the tile kernels run: from 9 rows an expert on,
#: and 33 slots
PATHS = {
    "one_token": (1, 512, 8, 2, 640, 0, False),
    "listed_by_a_warp": (16, 512, 8, 2, 640, 1, False),
    "listed_by_a_kernel": (40, 512, 32, 2, 640, 1, False),
    "eight_rows": (33, 512, 8, 2, 640, 0, False),
    "tiles_of_32": (30, 512, 4, 2, 640, 0, True),
    "tiles_of_64": (40, 512, 4, 2, 640, 0, True),
    "tiles_of_96": (130, 512, 4, 2, 640, 1, True),
    "tiles_of_128": (300, 512, 2, 1, 640, 0, True),
}


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, False), (128, True)])
@pytest.mark.parametrize("name", list(PATHS))
def test_no_rounding_but_those_stated(name, group, zeros):
    T, d, E, k, f, S, tiles = PATHS[name]
    c = Case(T, d, E, k, f, S, group, zeros, seed=T + group)
    got = c.run()
    want, off = bounds.experts(c.x, c.idx, c.w.astype(np.float64), c.gate, c.up, c.down, E, S, tiles)
    assert np.all(np.abs(got - want) <= off)
    assert np.linalg.norm(got - want) <= bounds.NORM * np.linalg.norm(want)


def powers(c, gate_up, down):
    """The case with its scales times powers of two."""
    for name, e in (("gate", gate_up), ("up", gate_up), ("down", down)):
        codes, scales, z = getattr(c, name)
        setattr(c, name, (codes, scales * 2.0 ** e, z))
    return c


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("end", ["small", "large", "mixed"])
def test_magnitudes_up_to_the_ends_of_the_ranges(end, T, zeros):
    """Every token row by itself, so that a large one hides no other: x about 2^-48
    and 2^-30 and scales about 2^20 (h about 2^-47, above the 2^-57 that counts
    as zero); x about 2^40 and 2^10 with scales down to 2^-86 (h about 2^56, below
    2^64); and rows 2^52 apart in one batch.  40 rows of two experts run on the
    tile kernels, 3 on the others."""
    c = Case(T, 256, 2, 1, 384, 0, 32, zeros, seed=T)
    c.idx[:, 0] = np.arange(T) % 7 == 3
    odd = np.arange(T)[:, None] % 2
    if end == "small":
        c.x = c.x * 2.0 ** np.where(odd, -48, -30)
        powers(c, 25, 28)
    elif end == "large":
        c.x = c.x * 2.0 ** np.where(odd, 40, 10)
        powers(c, -12, -78)
    else:
        c.x = c.x * 2.0 ** np.where(odd, 22, -30)
        powers(c, 6, -10)
    got = c.run()
    with np.errstate(over="ignore"):
        want, off = ref.experts(c.x, c.idx, c.w.astype(np.float64), c.gate, c.up, c.down, 2, 0)
    assert np.all(np.isfinite(got))
    # a row's h are a few hundred numbers, its error's norm that of four bf16
    # roundings at most, as for whole batches
    assert np.all(np.linalg.norm(got - want, axis=1) <= ref.EXPERTS_NORM * np.linalg.norm(want, axis=1))
    assert np.all(np.linalg.norm(want, axis=1) > 2.0 ** -100)
