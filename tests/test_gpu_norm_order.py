"""The order of the norms' sums: what it depends on, and what it does not."""
import numpy as np
import pytest

from test_gpu_norm import Case, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d", [(700, 1024), (320, 7168), (2000, 64)])
@pytest.mark.parametrize("pre,post,gate,res", [("rms", "rms", "channel", "bfloat16"), ("layer", "layer", "element", "float32")])
def test_rows_of_any_buffer_with_the_same_alignment(T, d, pre, post, gate, res):
    """Rows next to each other, and as columns of a wider buffer whose rows are aligned too: the same bits."""
    got = []
    for pad in (0, 16):
        c = Case(T, d, pre, post, gate, res=res, pad=pad)
        forward = c.forward()
        gradients, _ = c.backward()
        got.append({**{k: forward[k] for k in ("out", "norm", "stats")}, **gradients})
    assert got[0].keys() == got[1].keys()
    for k in got[0]:
        assert np.array_equal(got[0][k], got[1][k]), k


@pytest.mark.parametrize("d", [64, 1024])
def test_rows_that_are_not_aligned_are_summed_in_an_order_of_their_own(d):
    """The same values without alignment: within the bound of any order."""
    for pad in (0, 6):
        c = Case(3000, d, "layer", "rms", "channel", pad=pad)
        c.check_forward()
        c.check_backward()


def test_the_gradients_of_calls_in_between_change_nothing():
    """A handle's workspace holds one pass's sums: what a pass of more rows left there is not read."""
    import torch
    c = Case(50, 512, "rms", "rms", "channel")
    n, p = c.make(), c.params()
    n.reserve()

    def gradient(T, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        go, gn, out, y = (torch.randn(T, 512, generator=g, device="cuda").to(torch.bfloat16) for _ in range(4))
        st = torch.rand(T, 4, generator=g, device="cuda")
        grads = {k: torch.empty(512, device="cuda") for k in ("grad_pre_gain", "grad_post_gain", "grad_gate")}
        n.backward(go, gn, None, None, stats=st, out=out, y=y, **p, **grads)
        return [host(t) for t in grads.values()]

    first = gradient(50, 1)
    gradient(20000, 2)
    assert all(np.array_equal(a, b) for a, b in zip(first, gradient(50, 1)))
