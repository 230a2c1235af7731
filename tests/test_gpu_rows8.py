"""8-bit rows against their definition: codes and scales to the bit."""
import numpy as np
import pytest

import _block_ref as br

pytestmark = pytest.mark.gpu


def convert(v, group, kind, shift=0):
    """codes, scales and the values read back; tensors begin `shift` elements into their memory."""
    import torch
    from persistent_megakernel_sm_gb300 import rows8_dequantize, rows8_quantize
    dtype = getattr(torch, kind)
    T, d = v.shape

    def at(shape, dtype):
        n = int(np.prod(shape))
        return torch.full((n + shift + 8,), 7, dtype=dtype, device="cuda")[shift:shift + n].view(shape)

    src, codes = at(v.shape, dtype), at(v.shape, torch.int8)
    src.copy_(torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)))
    scales, back = at((T, -(-d // group)), torch.bfloat16), at(v.shape, dtype)
    rows8_quantize(src, codes, scales, group=group)
    rows8_dequantize(codes, scales, back, group=group)
    torch.cuda.synchronize()
    behind = [t.untyped_storage() for t in (codes, scales, back)]
    for t, s in zip((codes, scales, back), behind):  # nothing around the tensors is touched
        flat = torch.empty(0, dtype=t.dtype, device="cuda").set_(s, 0, (t.numel() + shift + 8,))
        assert torch.all(flat[:shift] == 7) and torch.all(flat[shift + t.numel():] == 7)
    return codes.cpu().numpy(), scales.float().cpu().numpy().astype(np.float64), back.float().cpu().numpy().astype(np.float64)


def check(v, group, kind, shift=0):
    v = br.as_type(v, kind)
    codes, scales, back = convert(v, group, kind, shift)
    want_codes, want_scales = br.rows8(v, group, kind)
    assert np.array_equal(scales, want_scales, equal_nan=True)
    assert np.array_equal(codes, want_codes)
    # 7 bits times 8: exact in fp32, then rounded once
    assert np.array_equal(back, br.as_type(br.rows8_values(codes, scales, group), kind), equal_nan=True)


@pytest.mark.parametrize("kind", ["bfloat16", "float32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,d", [(1, 1), (3, 128), (5, 31), (2, 33), (37, 1408), (19, 257), (700, 200), (1, 32768)])
def test_rows(T, d, group, kind):
    rng = np.random.default_rng(T + d + group)
    check(rng.standard_normal((T, d)) * np.exp(2 * rng.standard_normal((T, 1))), group, kind)


@pytest.mark.parametrize("kind", ["bfloat16", "float32"])
def test_tensors_that_begin_anywhere(kind):
    rng = np.random.default_rng(3)
    for shift in (1, 4, 8):
        check(rng.standard_normal((7, 256)), 64, kind, shift)


@pytest.mark.parametrize("kind", ["bfloat16", "float32"])
def test_rows_at_the_edges(kind):
    """Exact halves between two codes, zeros, the largest and the smallest numbers."""
    big, small = 3.3895313892515355e38, 2.0 ** -133
    half = np.array([127, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5] * 16)
    rows = [np.zeros(128), half, half * 2.0 ** -120, half * 2.0 ** 100, np.tile([big, -big], 64), np.tile([small, -2 * small], 64),
            np.tile([1e-38, 0.0], 64), -np.arange(128.0), np.full(128, -0.0)]
    for group in (32, 128):
        check(np.array(rows), group, kind)
        check(np.array(rows)[:, :100], group, kind)


@pytest.mark.parametrize("kind", ["bfloat16", "float32"])
@pytest.mark.parametrize("d", [128, 100])
def test_groups_that_are_not_finite_become_nan(kind, d):
    v = np.ones((4, d))
    v[1, 5], v[2, 70], v[3, 99] = np.nan, np.inf, -np.inf
    check(v, 32, kind)


def test_empty():
    import torch
    from persistent_megakernel_sm_gb300 import rows8_dequantize, rows8_quantize
    for shape, scales in (((0, 64), (0, 1)), ((4, 0), (4, 0))):
        t = [torch.empty(shape, dtype=k, device="cuda") for k in (torch.bfloat16, torch.int8)]
        s = torch.empty(scales, dtype=torch.bfloat16, device="cuda")
        rows8_quantize(t[0], t[1], s, group=64)
        rows8_dequantize(t[1], s, t[0], group=64)
    torch.cuda.synchronize()


def test_offsets_beyond_32_bits():
    """More than 2^31 codes: the last rows are right, and the first."""
    import torch
    from persistent_megakernel_sm_gb300 import rows8_dequantize, rows8_quantize
    for d in (4096, 4095):
        T = (1 << 31) // d + 3
        v = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
        rng = np.random.default_rng(1)
        part = torch.from_numpy(rng.standard_normal((4, d)).astype(np.float32)).to(torch.bfloat16).cuda()
        v[:2], v[-2:] = part[:2], part[2:]
        codes = torch.empty(T, d, dtype=torch.int8, device="cuda")
        scales = torch.empty(T, -(-d // 128), dtype=torch.bfloat16, device="cuda")
        rows8_quantize(v, codes, scales)
        v.zero_()
        rows8_dequantize(codes, scales, v)
        want_codes, want_scales = br.rows8(part.float().cpu().numpy(), 128, "bfloat16")
        got = torch.cat((codes[:2], codes[-2:])).cpu().numpy()
        assert np.array_equal(got, want_codes)
        back = torch.cat((v[:2], v[-2:])).float().cpu().numpy()
        assert np.array_equal(back, br.bf16(br.rows8_values(want_codes, want_scales, 128)))
        del v, codes, scales


@pytest.mark.parametrize("kind", ["bfloat16", "float32"])
@pytest.mark.parametrize("d", [128, 127])
def test_quotients_next_to_halves(kind, d):
    """Values a rounding from halfway between two codes, over scales of every mantissa and of many sizes."""
    rng = np.random.default_rng(8)
    rows = []
    for i in range(400):
        s = np.float32((128 + i % 128) / 128 * 2.0 ** rng.integers(-110, 100))
        half = (rng.integers(-127, 127, d) + 0.5).astype(np.float32) * s
        v = half.copy()
        for _ in range(2):
            v = np.where(rng.random(d) < 0.4, np.nextafter(v, rng.choice([-np.inf, np.inf], d).astype(np.float32)), v)
        v[0] = 127 * s
        rows.append(v)
    check(np.array(rows), 128, kind)
