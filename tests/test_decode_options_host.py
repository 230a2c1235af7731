"""The options of the layer for a few tokens, on CPU."""
import persistent_megakernel_sm_gb300 as pkg
from persistent_megakernel_sm_gb300 import binding
from test_block_host import lib  # noqa: F401
from test_ops_host import rec  # noqa: F401


def test_options_validate(lib):  # noqa: F811
    h = lib.moe_decode_create(256, 512, 8, 2, 1)
    limit, drop = pkg.OPTIONS["timeout_ns"], pkg.OPTIONS["fault_drop_task"]
    try:
        for key, good, bad in ((limit, (1000, 2_000_000_000, 1 << 62), (999, 0, -1)), (drop, (-1, 0, 1), (-2, 2))):
            assert all(lib.moe_decode_set_option(h, key, v) == pkg.MOE_OK for v in good)
            assert all(lib.moe_decode_set_option(h, key, v) == pkg.MOE_E_INVAL for v in bad)
            assert lib.moe_decode_set_option(None, key, good[0]) == pkg.MOE_E_INVAL
        for key in (pkg.OPTIONS["mode"], 0, 99):
            assert lib.moe_decode_set_option(h, key, 1) == pkg.MOE_E_INVAL
    finally:
        lib.moe_decode_destroy(h)


def test_the_binding_passes_them_on(rec):  # noqa: F811
    n = binding.MoEDecode(256, 384, 8, 2)
    n.set_option("timeout_ns", 5_000_000)
    assert "moe_decode_set_option" in rec.calls
    n.close()
