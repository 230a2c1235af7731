"""The norms about a block with gains and shifts that are not given: 1 and 0."""
import pytest

from test_gpu_norm import Case

pytestmark = pytest.mark.gpu

LEFT_OUT = [("pre_gain", "pre_shift", "post_gain", "post_shift"), ("pre_gain",), ("post_gain",), ("pre_shift",), ("post_shift",),
            ("pre_gain", "post_shift"), ("post_gain", "pre_shift")]


@pytest.mark.parametrize("left_out", LEFT_OUT)
@pytest.mark.parametrize("pre,post,gate", [("layer", "layer", "channel"), ("rms", "rms", "none"), ("layer", "rms", "element"),
                                           ("rms", "layer", "token")])
def test_what_is_left_out(left_out, pre, post, gate):
    for i, (T, d, pad) in enumerate(((5, 200, 0), (3, 77, 3), (310, 4104, 0))):
        c = Case(T, d, pre, post, gate, res=("float32", "bfloat16")[i % 2], par=("bfloat16", "float32")[i % 2],
                 offset=bool(i % 2), scale=0.5, pad=pad)
        for name in left_out:
            c.p[name] = None
        c.check_forward(save=i == 0)
        c.check_backward(save=i == 0)
