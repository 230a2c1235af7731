"""The largest numbers of rows that the 8-bit conversions refuse, on CPU."""
import pytest

import persistent_megakernel_sm_gb300 as pkg
from test_block_host import lib  # noqa: F401


@pytest.mark.parametrize("rows,cols", [((1 << 34) - 7, 1), ((1 << 33) - 3, 257), ((1 << 28) + 1, 1 << 10)])
def test_more_pieces_or_values_than_there_may_be(lib, rows, cols):  # noqa: F811
    for call in (lib.moe_rows8_quantize, lib.moe_rows8_dequantize):
        for group in (32, 64, 128):
            assert call(rows, cols, 1, group, 16 if cols % group else 18, 16, 16, None) == pkg.MOE_E_INVAL
            assert lib.moe_last_error() in (b"too many rows", b"more than 2^38 values")
