"""A zero point is its byte's low four bits, in every operator that takes one."""
import numpy as np
import pytest

import _ops_ref as ref
from test_gpu_w4 import Case, dev, dev_bf16, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [32, 64, 128])
def test_the_way_back_takes_four_bits(group):
    import torch
    from persistent_megakernel_sm_gb300 import w4_dequantize
    rng = np.random.default_rng(group)
    codes, scales, _ = ref.make_w4(rng, 24, 384, group, False)
    zeros = rng.integers(0, 256, scales.shape, dtype=np.uint8)
    zeros[0, :2] = 255, 16
    back = torch.full((24, 384), 7.0, dtype=torch.bfloat16, device="cuda")
    w4_dequantize(dev(codes), dev_bf16(scales), dev(zeros), back)
    assert np.array_equal(host(back), ref.bf16(ref.values(codes, scales, zeros & 15)))


@pytest.mark.parametrize("T", [2, 40])
def test_the_experts_take_four_bits(T):
    c = Case(T, 256, 2, 1, 128, 0, 32, True, seed=T)
    want = c.run()
    rng = np.random.default_rng(1)
    for name in ("gate", "up", "down"):
        codes, scales, z = getattr(c, name)
        setattr(c, name, (codes, scales, z | rng.integers(0, 16, z.shape, dtype=np.uint8) << 4))
    assert np.array_equal(c.run(), want)
