"""The norms about a block without rows, on CPU: what has a row a token may be null, what has not is asked for."""
import ctypes

import pytest

import persistent_megakernel_sm_gb300 as pkg
from persistent_megakernel_sm_gb300 import binding
from test_block_host import _bwd, _fwd, _params, lib  # noqa: F401

NONE, CHANNEL, TOKEN, ELEMENT = range(4)


@pytest.mark.parametrize("gate", [NONE, CHANNEL, TOKEN, ELEMENT])
def test_no_rows(lib, gate):  # noqa: F811
    h = lib.moe_norm_create(64, 1, 1, gate, 1e-6, 1.0, 0, 128)
    empty = binding._Rows8(None, None)
    held, p = ctypes.byref(empty), _params(pre_gain=16, post_gain=16, gate=16 if gate == CHANNEL else None)
    kept = dict(out8=ctypes.addressof(empty), y8=ctypes.addressof(empty))
    try:
        assert _fwd(lib, h, T=0, r=None, y=None, out=None, n=None, p=p, out8=held, y8=held) == pkg.MOE_OK
        assert _bwd(lib, h, T=0, go=None, gn=None, gr=None, gy=None, p=p, kept=kept) == pkg.MOE_OK
        if gate == CHANNEL:  # a vector has no rows
            assert _fwd(lib, h, T=0, p=_params(pre_gain=16, post_gain=16)) == pkg.MOE_E_INVAL
        for T in (1, 4):
            assert _fwd(lib, h, T=T, p=p, out8=held) == pkg.MOE_E_INVAL
            if gate in (TOKEN, ELEMENT):
                assert _fwd(lib, h, T=T, p=p) == pkg.MOE_E_INVAL
    finally:
        lib.moe_norm_destroy(h)
