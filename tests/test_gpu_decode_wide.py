"""The layer for a few tokens where 9 to 16 of them meet wide layers: tiles of more than 16 rows, several tiles of down's
rows and chunks of f a block, gate and up's tiles cut short for their tokens' columns."""
import pytest

from test_gpu_decode import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(16, 7168, 2, 2, 2176, 1), (13, 5120, 2, 2, 2176, 0), (16, 4096, 2, 2, 2048, 0),
                                   (9, 7168, 4, 3, 1152, 1)])
def test_wide_layers_and_many_tokens(shape):
    c = Case(*shape, bias=True)
    n, weights = c.make(), c.weights()
    out, idx, w = c.forward(n, weights)
    c.check_choice(idx, w)
    c.check_out(out, idx, w)
    c.idx[2, 0], c.idx[-1] = -1, -1
    c.check_out(c.routed(n, weights), c.idx, c.w)
