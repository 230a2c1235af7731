"""The norms about a block over 8-bit rows with more than 2^31 codes: the first and the last rows are right."""
import numpy as np
import pytest

import _block_ref as br
from test_gpu_norm import B32, C32, U16, dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [32768, 32765])
def test_offsets_beyond_32_bits_in_rows_kept_in_8_bits(d):
    import torch
    from persistent_megakernel_sm_gb300 import MoEBlockNorm
    T, group, at = (1 << 31) // d + 5, 32, [0, 1, -2, -1]
    rng = np.random.default_rng(d)
    r, gn = (br.bf16(rng.standard_normal((4, d))) for _ in range(2))
    bf = dict(dtype=torch.bfloat16, device="cuda")

    def rows(v):
        t = torch.zeros(T, d, **bf)
        t[at] = dev(v, "bfloat16")
        return t

    n = MoEBlockNorm(d, pre="rms", group=group)
    residual, norm, stats = rows(r), torch.empty(T, d, **bf), torch.empty(T, 4, device="cuda")
    held = torch.empty(T, d, dtype=torch.int8, device="cuda"), torch.empty(T, -(-d // group), **bf)
    n.forward(residual, None, None, norm, stats=stats, out8=held)
    c = dict(pre="rms", post="none", gate="none", eps=1e-6, scale=1.0, one=0.0)
    p = dict.fromkeys(("pre_gain", "pre_shift", "post_gain", "post_shift"))
    want, m, rstd, size = br.normed(c, r, p)
    assert np.all(np.abs(host(norm[at]) - want) <= U16 * np.abs(want) + (1 + U16) * C32 * size)
    codes, scales = br.rows8(r, group, "bfloat16")
    assert np.array_equal(held[0][at].cpu().numpy(), codes) and np.array_equal(host(held[1][at]), scales)
    del residual
    gr = norm  # its memory
    n.backward(None, rows(gn), gr, None, stats=stats, out=held)
    kept, st = br.rows8_values(codes, scales, group), host(stats[at])
    want, size = br.backward(c, p, None, st, None, gn, kept, None)["residual"]
    assert np.all(np.abs(host(gr[at]) - want) <= U16 * np.abs(want) + (1 + U16) * B32 * size)
