"""The layer for a few tokens against its definition in 64 bits; and a decode step as it would be used."""
import numpy as np
import pytest

import _block_ref as br

pytestmark = pytest.mark.gpu

U16 = 2.0 ** -8


def dev(a, kind="bfloat16"):
    import torch
    if a is None:
        return None
    if a.dtype == np.int32:
        return torch.from_numpy(a).cuda()
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(getattr(torch, kind)).cuda()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


class Case:
    def __init__(self, T, d, E, k, f, S=0, bias=False, seed=0):
        rng = self.rng = np.random.default_rng(seed + T + d + E + f)
        self.shape = (T, d, E, k, f, S)
        n = E + S
        small = lambda *s: br.bf16(rng.standard_normal(s, dtype=np.float32) * s[-1] ** -0.5)  # noqa: E731
        self.gate, self.up, self.down, self.router = small(n, f, d), small(n, f, d), small(n, d, f), small(E, d)
        self.bias = (0.3 * rng.standard_normal(E)).astype(np.float32).astype(np.float64) if bias else None
        self.x = br.bf16(rng.standard_normal((T, d)))
        for _ in range(50):  # no two of the compared logits nearer than their sums' roundings
            logits = -np.sort(-(self.x @ self.router.T + (0 if self.bias is None else self.bias)), axis=1)[:, :k + 1]
            bad = (logits[:, :-1] - logits[:, 1:] < 1e-4).any(1)
            if not bad.any():
                break
            self.x[bad] = br.bf16(rng.standard_normal((bad.sum(), d)))
        self.idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
        self.w = rng.random((T, k)).astype(np.float32).astype(np.float64)

    def weights(self):
        return [dev(m) for m in (self.gate, self.up, self.down)]

    def make(self, T_max=None):
        from persistent_megakernel_sm_gb300 import MoEDecode
        T, d, E, k, f, S = self.shape
        n = MoEDecode(d, f, E, k, shared_experts=S)
        n.reserve(T_max or T)
        return n

    def forward(self, layer=None, weights=None, x=None):
        import torch
        x = dev(self.x if x is None else x)
        T, k = len(x), self.shape[3]
        out = torch.full((T + 1, x.shape[1]), 5.0, dtype=torch.bfloat16, device="cuda")
        idx = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
        w = torch.full((T, k), 77.0, device="cuda")
        n = layer or self.make()
        n.forward(x, dev(self.router), *(weights or self.weights()), out[:T], bias=dev(self.bias, "float32"), idx=idx, w=w)
        n.check()
        assert torch.all(out[T] == 5)
        return host(out[:T]), idx.cpu().numpy(), host(w)

    def routed(self, layer=None, weights=None, idx=None, w=None, x=None):
        import torch
        x = dev(self.x if x is None else x)
        out = torch.full((len(x) + 1, x.shape[1]), 5.0, dtype=torch.bfloat16, device="cuda")
        n = layer or self.make()
        n.forward_routed(x, dev(self.idx if idx is None else idx), dev(self.w if w is None else w, "float32"),
                         *(weights or self.weights()), out[:len(x)])
        n.check()
        assert torch.all(out[len(x)] == 5)
        return host(out[:len(x)])

    def check_out(self, got, idx, w, x=None):
        want, err = br.experts(self.x if x is None else x, idx, w, self.gate, self.up, self.down, self.shape[5])
        assert np.all(np.abs(got - want) <= U16 * np.abs(want) + (1 + U16) * err)
        return want

    def check_choice(self, idx, w, x=None):
        want_idx, want_w = br.choice(self.x if x is None else x, self.router, self.bias, self.shape[3])
        assert np.array_equal(idx, want_idx)
        # a logit is off by 128 roundings of its terms' sum, a weight by twice that, relative
        size = (np.abs(self.x if x is None else x) @ np.abs(self.router).T).max()
        assert np.all(np.abs(w - want_w) <= (2 * 128 * br.U32 * (size + 1) + 16 * br.U32) * want_w)


SHAPES = [(1, 128, 1, 1, 128, 0), (1, 256, 8, 2, 512, 0), (4, 2048, 16, 4, 768, 0), (16, 256, 8, 2, 384, 1),
          (9, 1024, 64, 6, 256, 1), (8, 256, 256, 16, 128, 0), (13, 384, 40, 3, 1408, 1), (5, 32768, 3, 2, 128, 0),
          (2, 128, 3, 2, 32768, 1), (7, 7168, 5, 5, 128, 0)]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_own_router(shape, bias):
    c = Case(*shape, bias=bias)
    out, idx, w = c.forward()
    c.check_choice(idx, w)
    c.check_out(out, idx, w)


@pytest.mark.parametrize("shape", SHAPES)
def test_given_routing(shape):
    c = Case(*shape)
    c.check_out(c.routed(), c.idx, c.w)


def test_every_number_of_tokens():
    c = Case(16, 512, 24, 4, 256, 1)
    n, weights = c.make(16), c.weights()
    for T in range(1, 17):
        out, idx, w = c.forward(n, weights, c.x[:T])
        c.check_choice(idx, w, c.x[:T])
        c.check_out(out, idx, w, c.x[:T])
        c.check_out(c.routed(n, weights, c.idx[:T], c.w[:T], c.x[:T]), c.idx[:T], c.w[:T], c.x[:T])


def test_h_keeps_sixteen_bits():
    """The output's own rounding alone is 1.66e-3 of its norm (a bf16 step over sqrt(12), over the binade); with h
    rounded to bf16 too it would be at least 2.2e-3."""
    c = Case(16, 2048, 4, 2, 512)
    got = c.routed()
    want, _ = br.experts(c.x, c.idx, c.w, c.gate, c.up, c.down, 0)
    assert np.linalg.norm(got - want) <= 1.85e-3 * np.linalg.norm(want)


def test_slots_without_an_expert():
    for S in (0, 1):
        c = Case(6, 256, 8, 3, 256, S)
        c.idx[1], c.idx[2, 1], c.idx[3, 0], c.idx[4] = -1, -1, 8, [5, 5, 2]
        c.idx[5] = 1 << 30
        c.w[1] = np.nan  # of slots that choose nothing
        got = c.routed()
        c.check_out(got, c.idx, c.w)
        if not S:
            assert np.all(got[1] == 0) and np.all(got[5] == 0)
        c.idx[:] = -1
        got = c.routed()
        c.check_out(got, c.idx, c.w)
        assert S or np.all(got == 0)


def test_masked_experts_and_ties():
    c = Case(5, 256, 12, 4, 128, bias=True)
    c.bias[:] = 0
    c.bias[[0, 3, 4, 5, 6, 8, 9, 10, 11]] = -np.inf  # three are left for four slots
    out, idx, w = c.forward()
    c.check_choice(idx, w)
    assert np.all(idx[:, 3] == -1) and np.all(w[:, 3] == 0) and np.all(np.isin(idx[:, :3], (1, 2, 7)))
    c.check_out(out, idx, w)
    c.bias[:] = 0
    c.x[2] = 0  # every logit alike: the first experts, evenly
    out, idx, w = c.forward()
    assert np.array_equal(idx[2], [0, 1, 2, 3]) and np.all(w[2] == 0.25) and np.all(out[2] == 0)
    c.bias[:] = -np.inf
    out, idx, w = c.forward()
    assert np.all(idx == -1) and np.all(w == 0) and np.all(out == 0)


def test_what_is_not_finite_stays_where_it_was_chosen():
    c = Case(6, 256, 8, 2, 256)
    c.idx[:] = [[0, 1], [1, 2], [2, 3], [4, 5], [5, 6], [6, 4]]
    clean = c.routed()
    c.gate[3, 7, 5], c.down[3, 2, 9], c.down[7], c.up[7] = np.nan, np.inf, np.nan, np.inf  # 3: token 2 alone; 7: none
    c.x[5, 3] = np.inf
    got = c.routed()
    for t in (0, 1, 3, 4):
        assert np.array_equal(got[t], clean[t]), t
    assert np.all(np.isnan(got[2])) and np.all(np.isnan(got[5]))


def test_offsets_beyond_32_bits():
    """More than 2^31 weights a matrix: the last expert's output is right."""
    import torch
    from persistent_megakernel_sm_gb300 import MoEDecode
    d, f, E = 4096, 4096, 132
    m = [torch.zeros(E, f, d, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    rng = np.random.default_rng(0)
    part = [br.bf16(rng.standard_normal((2, f, d), dtype=np.float32) / 64) for _ in range(3)]
    for a, b in zip(m, part):
        a[0], a[E - 1] = dev(b)[0], dev(b)[1]
    x, w = br.bf16(rng.standard_normal((3, d))), np.full((3, 2), 0.5)
    idx = np.array([[0, E - 1], [E - 1, 4], [E - 1, 0]], dtype=np.int32)
    n = MoEDecode(d, f, E, 2)
    n.reserve(3)
    out = torch.empty(3, d, dtype=torch.bfloat16, device="cuda")
    n.forward_routed(dev(x), dev(idx), dev(w, "float32"), *m, out)
    n.check()
    near = np.where(idx == E - 1, 1, np.where(idx == 0, 0, -1)).astype(np.int32)
    want, err = br.experts(x, near, w, *part, 0)
    assert np.all(np.abs(host(out) - want) <= U16 * np.abs(want) + (1 + U16) * err)


def test_captured_passes_on_streams_of_their_own():
    """Two handles' graphs at once, on new tokens in the old tensors: the bits of the eager passes."""
    import torch
    c = Case(5, 512, 16, 4, 256, 1, bias=True)
    weights, router, bias = c.weights(), dev(c.router), dev(c.bias, "float32")
    runs = []
    for i in range(2):
        n, x = c.make(), dev(c.x)
        out, idx, w = torch.empty_like(x), torch.empty(5, 4, dtype=torch.int32, device="cuda"), torch.empty(5, 4, device="cuda")
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            n.forward(x, router, *weights, out, bias=bias, idx=idx, w=w)
            side.synchronize()
            with torch.cuda.graph(graph, stream=side):
                n.forward(x, router, *weights, out, bias=bias, idx=idx, w=w)
        runs.append((n, x, (out, idx, w), side, graph))
    torch.cuda.synchronize()
    for _ in range(3):
        want = []
        for n, x, outs, _, _ in runs:
            x.normal_()
            n.forward(x, router, *weights, outs[0], bias=bias, idx=outs[1], w=outs[2])
            want.append([t.clone() for t in outs])
            for t in outs:
                t.fill_(3)
        torch.cuda.synchronize()
        for _, _, _, side, graph in runs:
            with torch.cuda.stream(side):
                for _ in range(5):
                    graph.replay()
        torch.cuda.synchronize()
        for (n, _, outs, _, _), w in zip(runs, want):
            n.check()
            assert all(torch.equal(a, b) for a, b in zip(outs, w))


def test_reserving_again_and_no_tokens():
    import torch
    from persistent_megakernel_sm_gb300 import MOE_E_INVAL, MOE_E_STATE, MoEDecode, MoEError
    c = Case(4, 256, 8, 2, 128)
    n, weights = c.make(2), c.weights()
    with pytest.raises(MoEError) as err:
        c.routed(n, weights)
    assert err.value.code == MOE_E_INVAL
    n.reserve(16)
    c.check_out(c.routed(n, weights), c.idx, c.w)
    n.reserve(4)
    c.check_out(c.routed(n, weights), c.idx, c.w)
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    n.forward(e, dev(c.router), *weights, e)
    n.forward_routed(e, torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda"), *weights, e)
    n.check()
    with pytest.raises(MoEError) as err:
        c.routed(MoEDecode(256, 128, 8, 2), weights)
    assert err.value.code == MOE_E_STATE


@pytest.mark.parametrize("S", [0, 1])
def test_the_layer_itself(S):
    """The same tensors through the layer's megakernel: the same choice, and outputs within both roundings."""
    import torch
    from persistent_megakernel_sm_gb300 import MoELayer
    c = Case(8, 512, 16, 4, 256, S, bias=True)
    out, idx, w = c.forward()
    layer = MoELayer(512, 256, 16, 4, S)
    layer.reserve(8)
    weights = c.weights()
    bias = dev(c.bias, "float32")
    layer.set_router_bias(bias)
    got = torch.empty(8, 512, dtype=torch.bfloat16, device="cuda")
    layer.forward(dev(c.x), dev(c.router), *weights, got)
    layer.check()
    li = torch.empty(8, 4, dtype=torch.int32, device="cuda")
    layer.get_routing(idx=li)
    assert np.array_equal(np.sort(li.cpu().numpy(), 1), np.sort(idx, 1))
    # the layer rounds h and y to bf16: what it is held to against 64 bits
    assert np.all(np.abs(host(got) - out) <= 1e-2 + 1e-2 * np.abs(out))


def test_a_decode_step_of_a_block():
    """Norm, the layer for a few tokens on the routing operator's choice, gate, residual add and the next norm: each on
    what the one before it wrote."""
    import torch
    from persistent_megakernel_sm_gb300 import MoEBlockNorm, MoEDecode, MoERouter
    T, d, E, k, f, S = 6, 512, 32, 4, 256, 1
    c = Case(T, d, E, k, f, S)
    bf = torch.bfloat16
    first = MoEBlockNorm(d, pre="rms")
    after = MoEBlockNorm(d, pre="rms", post="rms", gate="channel", scale=0.5)
    router = MoERouter(E, k, score="sigmoid", groups=4, groups_kept=2, scale=2.5)
    layer = c.make()
    rng = np.random.default_rng(4)
    gains = [br.bf16(1 + 0.2 * rng.standard_normal(d)) for _ in range(3)]
    gate = br.bf16(0.5 + 0.2 * rng.standard_normal(d))
    r = br.bf16(rng.standard_normal((T, d)))
    residual, n0, y, n1 = dev(r), *(torch.empty(T, d, dtype=bf, device="cuda") for _ in range(3))
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    first.forward(residual, None, None, n0, pre_gain=dev(gains[0]))
    logits = n0.float() @ dev(c.router).float().t()
    router.forward(logits, idx, w)
    layer.forward_routed(n0, idx, w, *c.weights(), y)
    out = residual.clone()
    after.forward(out, y, out, n1, pre_gain=dev(gains[1]), post_gain=dev(gains[2]), gate=dev(gate))
    layer.check()
    conf = dict(pre="rms", post="rms", gate="channel", eps=1e-6, scale=0.5, one=0.0)
    p = dict(pre_gain=gains[0], pre_shift=None, post_gain=gains[2], post_shift=None)
    want, _, _, size = br.normed(conf, r, p)
    assert np.all(np.abs(host(n0) - want) <= U16 * np.abs(want) + 33 * br.U32 * size)
    c.check_out(host(y), idx.cpu().numpy(), host(w), host(n0))
    want, _, _, size = br.summed(conf, r, host(y), p, gate)
    assert np.all(np.abs(host(out) - want) <= U16 * np.abs(want) + 33 * br.U32 * size)
    want, _, _, size = br.normed(conf, host(out), dict(p, pre_gain=gains[1]))
    assert np.all(np.abs(host(n1) - want) <= U16 * np.abs(want) + 33 * br.U32 * size)
