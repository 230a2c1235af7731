"""4-bit weights: their conversion and the experts on them, against their
definitions in 64 bits; and a decode step as it would be used."""
import numpy as np
import pytest

import _harness as hz
import _ops_ref as ref

pytestmark = pytest.mark.gpu


def dev_bf16(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


def dev(a):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------ conversion

def convert(w, group, zeros):
    import torch
    from persistent_megakernel_sm_gb300 import w4_dequantize, w4_quantize
    src = dev_bf16(w)
    n, k = w.shape
    codes = torch.full((n, k // 2), 7, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, k // group), 7.0, dtype=torch.bfloat16, device="cuda")
    z = torch.full((n, k // group), 7, dtype=torch.uint8, device="cuda") if zeros else None
    back = torch.full((n, k), 7.0, dtype=torch.bfloat16, device="cuda")
    w4_quantize(src, codes, scales, z)
    w4_dequantize(codes, scales, z, back)
    torch.cuda.synchronize()
    return codes.cpu().numpy(), host(scales), None if z is None else z.cpu().numpy(), host(back)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,k", [(1, 128), (3, 256), (37, 1408), (1000, 640)])
def test_conversion(n, k, group, zeros):
    rng = np.random.default_rng(n + k + group)
    w = ref.bf16(rng.standard_normal((n, k)) * np.exp(2 * rng.standard_normal((n, 1))))
    codes, scales, z, back = convert(w, group, zeros)
    want_codes, want_scales, want_z = ref.quantize(w, group, zeros)
    assert np.array_equal(scales, want_scales)
    assert np.array_equal(codes, want_codes)
    assert z is None or np.array_equal(z, want_z)
    # a 4-bit number times a bf16 scale, rounded once: exactly the bf16 value
    assert np.array_equal(back, ref.bf16(ref.values(codes, scales, z)))


@pytest.mark.parametrize("zeros", [False, True])
def test_conversion_at_the_edges(zeros):
    """Exact halves between two codes, all zeros, one sign only, the largest and
    the smallest numbers."""
    big = 3.3895313892515355e38
    rows = [np.zeros(64), np.full(64, 0.5), -np.arange(64.0), np.tile([7.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, -7.0], 8),
            np.tile([15.0, 0.5, 1.5, 2.5, 3.5, 12.5, 13.5, 0.0], 8), np.tile([big, -big], 32),
            np.tile([2.0 ** -133, -(2.0 ** -132)], 32), np.tile([1e-38, 0.0], 32), np.tile([-3.5, 0.25, 0.75, 1.25], 16)]
    w = ref.bf16(np.array(rows))
    codes, scales, z, back = convert(w, 64, zeros)
    want_codes, want_scales, want_z = ref.quantize(w, 64, zeros)
    assert np.array_equal(scales, want_scales)
    assert np.array_equal(codes, want_codes)
    assert z is None or np.array_equal(z, want_z)


@pytest.mark.parametrize("zeros", [False, True])
def test_groups_that_are_not_finite_become_nan(zeros):
    w = np.ones((4, 128))
    w[1, 5], w[2, 70], w[3, 127] = np.nan, np.inf, -np.inf
    codes, scales, z, back = convert(w, 64, zeros)
    bad = np.zeros((4, 2), dtype=bool)
    bad[1, 0] = bad[2, 1] = bad[3, 1] = True
    assert np.array_equal(np.isnan(scales), bad)
    assert np.array_equal(np.isnan(back), np.repeat(bad, 64, 1))
    assert np.all(codes[1, :32] == 0x88) and (z is None or z[1, 0] == 8)
    assert np.array_equal(back[~np.repeat(bad, 64, 1)], np.round(back[~np.repeat(bad, 64, 1)] * 64) / 64)


# --------------------------------------------------------------------- experts

class Case:
    def __init__(self, T, d, E, k, f, S=0, group=128, zeros=False, seed=0):
        rng = np.random.default_rng(seed)
        self.shape = (T, d, E, k, f, S, group, zeros)
        self.gate, self.up = (ref.make_w4(rng, f, d, group, zeros, (E + S,)) for _ in range(2))
        self.down = ref.make_w4(rng, d, f, group, zeros, (E + S,))
        self.x = ref.bf16(rng.standard_normal((T, d)))
        self.idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
        w = np.exp(rng.standard_normal((T, k)))
        self.w = (w / w.sum(1, keepdims=True)).astype(np.float32)

    def layer(self, T_max=None):
        from persistent_megakernel_sm_gb300 import W4Experts
        T, d, E, k, f, S, group, zeros = self.shape
        e = W4Experts(d, f, E, k, shared_experts=S, group=group)
        e.reserve(T_max or max(T, 1))
        self.dev = [(dev(c), dev_bf16(s), dev(z)) for c, s, z in (self.gate, self.up, self.down)]
        e.set_weights(*self.dev)
        return e

    def run(self, layer=None):
        import torch
        T, d = self.shape[:2]
        layer = layer or self.layer()
        out = torch.full((T, d), 77.0, dtype=torch.bfloat16, device="cuda")
        layer.forward(dev_bf16(self.x), dev(self.idx), dev(self.w), out)
        torch.cuda.synchronize()
        return host(out)

    def check(self, got):
        T, d, E, k, f, S, group, zeros = self.shape
        want, off = ref.experts(self.x, self.idx, self.w.astype(np.float64), self.gate, self.up, self.down, E, S)
        assert np.all(np.abs(got - want) <= off)
        if want.any():
            assert np.linalg.norm(got - want) <= ref.EXPERTS_NORM * np.linalg.norm(want)


    def checked(self):
        layer = self.layer()
        self.check(self.run(layer))
        layer.check()


CASES = {
    # T, d, E, k, f, S, group, zeros
    "one_token": (1, 256, 8, 2, 384, 0, 128, False),
    "one_expert": (1, 128, 1, 1, 128, 0, 32, True),
    "groups_of_32": (5, 256, 8, 3, 512, 0, 32, False),
    "zero_points_shared": (13, 384, 6, 2, 256, 1, 64, True),
    "nine_rows": (9, 256, 1, 1, 256, 0, 128, True),
    "seventeen_rows": (17, 128, 1, 1, 640, 0, 64, False),
    "thirtythree_rows": (33, 256, 2, 2, 256, 1, 32, True),
    "many_rows": (150, 256, 3, 2, 256, 0, 128, False),
    "top16": (40, 128, 32, 16, 128, 1, 32, False),
    "many_experts": (3, 128, 256, 8, 128, 0, 128, True),
    "long_rows": (2, 2048, 2, 2, 128, 0, 128, False),
    "long_rows_down": (3, 128, 4, 2, 2176, 0, 128, False),
    "over_1024_slots": (130, 128, 16, 16, 128, 0, 128, False),
}


@pytest.mark.parametrize("name", list(CASES))
def test_experts(name):
    c = Case(*CASES[name], seed=len(name))
    c.check(c.run())


def test_padded_rows_dropped_slots_and_outside_indices():
    c = Case(20, 256, 8, 3, 256, 0, 64, True, seed=5)
    c.idx[15:] = -1
    c.idx[3, 1] = -1
    c.idx[4] = [8, -7, np.iinfo(np.int32).max]
    c.w[15:] = np.nan            # weights of slots without an expert are not read into anything
    c.w[3, 1] = np.inf
    c.x[17] = np.nan             # nor are the rows
    got = c.run()
    assert np.all(got[15:] == 0) and np.all(got[4] == 0)
    c.w[15:], c.w[3, 1], c.x[17] = 0, 0, 0
    c.check(got)


def test_shared_expert_reads_padded_rows():
    c = Case(6, 128, 4, 2, 128, 1, 32, False, seed=6)
    c.idx[4:] = -1
    c.check(c.run())


def test_an_expert_named_twice_counts_twice():
    c = Case(12, 128, 4, 4, 256, 0, 128, False, seed=7)
    c.idx[:] = 2                 # 48 rows for one expert
    c.idx[5] = [1, 1, 3, 1]
    c.check(c.run())


def test_all_to_one_expert():
    c = Case(100, 128, 16, 1, 128, 0, 64, False, seed=8)
    c.idx[:] = 11
    c.check(c.run())


def test_smaller_batches_on_a_larger_workspace_and_repeats_give_the_same_bits():
    import torch
    big = Case(64, 256, 8, 2, 256, 0, 32, True, seed=9)
    layer = big.layer(T_max=200)
    first = big.run(layer)
    big.check(first)
    x, idx, w = dev_bf16(big.x), dev(big.idx), dev(big.w)
    for T in (0, 1, 2, 7, 64):
        out = torch.full((T, 256), 3.0, dtype=torch.bfloat16, device="cuda")
        layer.forward(x[:T], idx[:T], w[:T], out)
        want, off = ref.experts(big.x[:T], big.idx[:T], big.w[:T].astype(np.float64), big.gate, big.up, big.down, 8, 0)
        assert np.all(np.abs(host(out) - want) <= off)
    assert np.array_equal(big.run(layer), first)


def test_graph_replay_on_a_side_stream():
    import torch
    a, b = (Case(24, 256, 8, 2, 256, 1, 128, False, seed=10) for _ in range(2))
    layer = a.layer()
    rng = np.random.default_rng(3)
    b.x = ref.bf16(rng.standard_normal(b.x.shape))
    b.idx = np.roll(b.idx, 5, axis=0)
    want = [a.run(layer), b.run(layer)]
    x, idx, w = dev_bf16(a.x), dev(a.idx), dev(a.w)
    out = torch.empty(24, 256, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            layer.forward(x, idx, w, out)
    for c, o in ((a, want[0]), (b, want[1]), (a, want[0])):
        x.copy_(dev_bf16(c.x))
        idx.copy_(dev(c.idx))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(out), o)


def test_calls_one_after_another_without_waiting():
    """Passes of several layers and sizes queued on one stream."""
    cases = [Case(T, 256, 8, 2, 384, 0, 64, False, seed=20 + T) for T in (1, 40, 2, 17)]
    import torch
    layers = [c.layer() for c in cases]
    ins = [(dev_bf16(c.x), dev(c.idx), dev(c.w), torch.empty(c.shape[0], 256, dtype=torch.bfloat16, device="cuda"))
           for c in cases]
    for _ in range(20):
        for layer, (x, idx, w, out) in zip(layers, ins):
            layer.forward(x, idx, w, out)
    torch.cuda.synchronize()
    for c, i in zip(cases, ins):
        c.check(host(i[3]))


# ------------------------------------------------------- as it would be used

def test_route_then_experts_and_the_bf16_layer_on_the_same_weights():
    """A decode step: convert the layer's bf16 weights, route on the logits,
    run the 4-bit experts; and the bf16 layer on the converted values (the
    prompt's path), whose routing is the softmax router's."""
    import torch
    from persistent_megakernel_sm_gb300 import MoERouter, W4Experts, w4_dequantize, w4_quantize
    T, d, E, k, f, S, group = 48, 256, 8, 2, 512, 1, 64
    w, inp = hz.custom_case(T, d, E, k, f, S)
    up = hz.upload(inp)
    w4, back = [], []
    for name in ("w_gate", "w_up", "w_down"):
        m = up[name]
        codes = torch.empty(*m.shape[:-1], m.shape[-1] // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(*m.shape[:-1], m.shape[-1] // group, dtype=torch.bfloat16, device="cuda")
        zeros = torch.empty(*m.shape[:-1], m.shape[-1] // group, dtype=torch.uint8, device="cuda")
        w4_quantize(m, codes, scales, zeros)
        w4.append((codes, scales, zeros))
        back.append(w4_dequantize(codes, scales, zeros, torch.empty_like(m)))
    logits = up["x"].float() @ up["router_w"].float().t()
    idx, wt = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    MoERouter(E, k).forward(logits, idx, wt)
    experts = W4Experts(d, f, E, k, shared_experts=S, group=group)
    experts.reserve(T)
    experts.set_weights(*w4)
    out = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    experts.forward(up["x"], idx, wt, out)
    torch.cuda.synchronize()
    mats = [(c.cpu().numpy(), host(s), z.cpu().numpy()) for c, s, z in w4]
    want, off = ref.experts(host(up["x"]), idx.cpu().numpy(), wt.cpu().numpy().astype(np.float64), *mats, E, S)
    assert np.all(np.abs(host(out) - want) <= off)
    # the bf16 layer on the values the 4-bit weights stand for
    layer = hz.make_layer(w)
    full, routing = hz.run_layer(layer, w, dict(up, w_gate=back[0], w_up=back[1], w_down=back[2]))
    layer.close()
    assert np.array_equal(np.sort(routing["idx"], 1), np.sort(idx.cpu().numpy(), 1))
    assert np.all(np.abs(hz.bf16_to_f64(full) - host(out)) <= 1e-2 + 1e-2 * np.abs(host(out)) + off)


def test_conversion_of_more_than_2_to_the_31_weights():
    import torch
    from persistent_megakernel_sm_gb300 import w4_dequantize, w4_quantize
    n, k = (1 << 17) + 8, 1 << 14
    w = torch.zeros(n, k, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(3)
    rows = ref.bf16(rng.standard_normal((4, k)))
    at = [0, (1 << 17) - 1, 1 << 17, n - 1]
    for r, v in zip(at, rows):
        w[r] = dev_bf16(v)
    codes = torch.zeros(n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(n, k // 32, dtype=torch.bfloat16, device="cuda")
    zeros = torch.zeros(n, k // 32, dtype=torch.uint8, device="cuda")
    w4_quantize(w, codes, scales, zeros)
    want = ref.quantize(rows, 32, True)
    for got, v in zip((codes, scales, zeros), want):
        got = got[at]
        assert np.array_equal(host(got) if got.dtype == torch.bfloat16 else got.cpu().numpy(), v)
    w.fill_(7.0)
    w4_dequantize(codes, scales, zeros, w)
    assert np.array_equal(host(w[at]), ref.bf16(ref.values(*want)))
    assert torch.count_nonzero(w[5:105]) == 0


def test_experts_behind_2_to_the_31_bytes_of_codes():
    """The last of 80 experts of 4096 x 14336, by the small kernels and by the tile
    kernels, against its product in 64 bits."""
    import torch
    from persistent_megakernel_sm_gb300 import W4Experts
    E, d, f, group = 80, 4096, 14336, 128
    g = torch.Generator(device="cuda").manual_seed(5)

    def matrix(rows, cols):
        codes = torch.randint(0, 256, (E, rows, cols // 2), dtype=torch.uint8, device="cuda", generator=g)
        scales = (0.5 + torch.rand(E, rows, cols // group, device="cuda", generator=g)) / (4.6 * cols ** 0.5)
        return codes, scales.bfloat16(), None

    def last(m):
        q = torch.stack((m[0][-1] & 15, m[0][-1] >> 4), -1).flatten(1).double() - 8
        return q * m[1][-1].double().repeat_interleave(group, 1)

    gate, up, down = matrix(f, d), matrix(f, d), matrix(d, f)
    experts = W4Experts(d, f, E, 1, group=group)
    experts.reserve(720)
    experts.set_weights(gate, up, down)
    for T in (2, 720):
        x = torch.randn(T, d, device="cuda", generator=g).bfloat16()
        idx = torch.full((T, 1), E - 1, dtype=torch.int32, device="cuda")
        w = torch.ones(T, 1, device="cuda")
        out = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
        experts.forward(x, idx, w, out)
        xd = x.double()
        want = (torch.nn.functional.silu(xd @ last(gate).T) * (xd @ last(up).T)) @ last(down).T
        assert float((out.double() - want).norm() / want.norm()) <= ref.EXPERTS_NORM
    experts.check()


# --------------------------------------------- the ways a batch can be run

@pytest.mark.parametrize("group,zeros", [(32, False), (32, True), (64, False), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("T", [1, 5, 40, 90])
def test_every_kernel_with_every_group_and_zero_point(T, group, zeros):
    """One token (the fused sums), a few rows (the small kernels), 20 and 45 rows
    an expert (the tile kernels), with rows of 384 and 640 columns: row tiles
    that do not fill a four of them."""
    Case(T, 384, 4, 2, 640, 1, group, zeros, seed=T + group).checked()


@pytest.mark.parametrize("rows", [6, 31, 32, 33, 63, 64, 65, 96, 97, 128, 129, 200])
def test_tiles_with_token_counts_about_their_widths(rows):
    c = Case(rows, 256, 2, 1, 256, 0, 128, False, seed=rows)
    c.idx[:] = 1
    c.idx[rows // 2:rows // 2 + 1] = 0
    c.checked()


def test_uneven_experts_on_the_tile_kernels():
    """One expert has most of the rows, one a single row, one none."""
    c = Case(300, 128, 5, 2, 384, 0, 64, True, seed=77)
    rng = np.random.default_rng(1)
    c.idx[:, 0], c.idx[:, 1] = 3, np.where(rng.random(300) < 0.1, 1, 2)
    c.idx[9, 1] = 0
    c.idx[250:] = -1
    c.w[250:] = 0
    c.checked()


def test_nothing_to_do_writes_zeros():
    for T in (1, 3, 64):
        c = Case(T, 128, 8, 2, 128, 0, 128, False, seed=T)
        c.idx[:] = -1
        layer = c.layer()
        assert np.all(c.run(layer) == 0)
        c.idx[:] = [0, 1]
        c.check(c.run(layer))


def test_largest_batch():
    """T = 1024, k = 16: 16384 slots, listed in 16 rounds."""
    c = Case(1024, 128, 64, 16, 128, 0, 128, False, seed=91)
    got = c.run()
    rows = np.r_[0:8, 511:515, 1016:1024]
    want, off = ref.experts(c.x[rows], c.idx[rows], c.w[rows].astype(np.float64), c.gate, c.up, c.down, 64, 0)
    assert np.all(np.abs(got[rows] - want) <= off)
    assert np.all(np.isfinite(got))


def test_two_layers_at_once_on_two_streams():
    import torch
    a, b = Case(1, 512, 8, 2, 1024, 0, 128, False, seed=95), Case(64, 512, 8, 2, 1024, 0, 64, True, seed=96)
    la, lb = a.layer(), b.layer()
    want = [a.run(la), b.run(lb)]
    ins = [(dev_bf16(c.x), dev(c.idx), dev(c.w), torch.empty(c.shape[0], 512, dtype=torch.bfloat16, device="cuda"))
           for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(30):
        for layer, i, s in zip((la, lb), ins, streams):
            with torch.cuda.stream(s):
                layer.forward(*i)
    torch.cuda.synchronize()
    for i, w in zip(ins, want):
        assert np.array_equal(host(i[3]), w)
    la.check(), lb.check()


def test_magnitudes_at_the_ends_of_the_range():
    """x of 2^40 and 2^-40, scales of 2^-60: h and out far from one."""
    for T in (3, 24):
        c = Case(T, 128, 2, 1, 128, 0, 128, False, seed=5)
        c.x = c.x * 2.0 ** np.where(np.arange(T) % 2, -20, 20)[:, None]
        c.down = (c.down[0], c.down[1] * 2.0 ** -60, None)
        c.checked()


@pytest.mark.parametrize("T", [2, 40])
@pytest.mark.parametrize("zeros", [False, True])
def test_magnitudes_within_rows(T, zeros):
    """Scales 2^20 apart within a weight row and 2^6 between rows, values 2^16
    apart within a token row and 2^8 between rows, a row of zeros and one of
    subnormal numbers.  |gate|, |up| are under 2^(14 + 12 + 3), so h is in the
    range that the operator takes (2^64)."""
    c = Case(T, 256, 2, 1, 384, 0, 32, zeros, seed=T)
    rng = np.random.default_rng(T)
    for name in ("gate", "up", "down"):
        codes, scales, z = getattr(c, name)
        scales = scales * 2.0 ** rng.integers(-10, 11, scales.shape)
        scales = scales * 2.0 ** rng.integers(-3, 4, scales.shape[:-1])[..., None]
        setattr(c, name, (codes, ref.bf16(scales), z))
    c.x = c.x * 2.0 ** rng.integers(-8, 9, c.x.shape) * 2.0 ** rng.integers(-4, 5, (T, 1))
    if T > 2:
        c.x[3] = 0.0
        c.x[4] = 2.0 ** -133 * rng.integers(-100, 101, 256)
    c.x = ref.bf16(c.x)
    got = c.run()
    want, off = ref.experts(c.x, c.idx, c.w.astype(np.float64), c.gate, c.up, c.down, 2, 0)
    assert np.all(np.abs(got - want) <= off + 2.0 ** -60)


@pytest.mark.parametrize("bad", [np.inf, np.nan])
@pytest.mark.parametrize("T", [3, 40])
def test_a_row_that_is_not_finite_stays_its_own(T, bad):
    c = Case(T, 256, 2, 1, 128, 1, 64, False, seed=T)
    c.x[1, 77] = bad
    got = c.run()
    assert np.all(~np.isfinite(got[1]))
    keep = np.arange(T) != 1
    want, off = ref.experts(c.x[keep], c.idx[keep], c.w[keep].astype(np.float64), c.gate, c.up, c.down, 2, 1)
    assert np.all(np.abs(got[keep] - want) <= off)


def test_weights_replaced():
    import torch
    a, b = Case(9, 128, 4, 2, 256, 0, 64, True, seed=1), Case(9, 128, 4, 2, 256, 0, 64, False, seed=2)
    layer = a.layer()
    a.check(a.run(layer))
    second = [(dev(c), dev_bf16(s), dev(z)) for c, s, z in (b.gate, b.up, b.down)]
    layer.set_weights(*second)
    for _, s, _ in second:
        s.zero_()                       # copied: later changes are not seen
    b.check(b.run(layer))
    layer.reserve(50)                   # a larger workspace keeps them
    b.check(b.run(layer))
    torch.cuda.synchronize()
