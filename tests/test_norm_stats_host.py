"""The norms' gradient asks for stats where a norm is passed through, on CPU."""
import persistent_megakernel_sm_gb300 as pkg
from test_block_host import _bwd, _params, lib  # noqa: F401


def test_stats_are_asked_for_where_a_norm_is_passed_through(lib):  # noqa: F811
    h = lib.moe_norm_create(64, 1, 1, 2, 1e-6, 1.0, 0, 128)
    p = _params(pre_gain=16, post_gain=16, gate=16)
    kept = dict(out=64, out_stride=64, y=64, y_stride=64)
    no = pkg.MOE_E_INVAL
    try:
        assert _bwd(lib, h, p=p, kept=kept) == no                                           # both
        assert _bwd(lib, h, p=p, kept=kept, gy=None) == no                                  # the pre norm
        assert _bwd(lib, h, p=p, kept=kept, gn=None) == no                                  # the post norm, for grad_y
        assert _bwd(lib, h, p=p, kept=kept, gn=None, gy=None, grads=dict(gate=16)) == no    # and for the gate's gradient
    finally:
        lib.moe_norm_destroy(h)
