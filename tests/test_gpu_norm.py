"""The norms about a block and their gradient, against their definitions in 64 bits."""
import numpy as np
import pytest

import _block_ref as br

pytestmark = pytest.mark.gpu

U16 = 2.0 ** -8  # half a step of bf16, relative to the value
# fp32 roundings of a value that is a few products and sums of terms, and of the
# statistics in it: a thread's 8 terms, five exchanges in a warp, four warps a lane
# and five exchanges more (22 roundings), the root, and less than ten of its own.
# The sums of the backward pass go through one more such chain.
C32 = 32 * br.U32
B32 = 64 * br.U32


def dev(a, kind="float32"):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(getattr(torch, kind)).cuda()


def host(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


class Wide:
    """Rows as columns of a wider buffer, with marks around them."""

    def __init__(self, T, d, kind, pad):
        import torch
        self.mark = 5.0
        self.all = torch.full((T + 1, d + pad), self.mark, dtype=getattr(torch, kind), device="cuda")
        self.rows = self.all[:T, pad // 2:pad // 2 + d]
        self.T, self.d, self.pad = T, d, pad

    def fill(self, a, kind):
        self.rows.copy_(dev(a, kind))
        return self

    def untouched(self):
        a, lo = host(self.all), self.pad // 2
        return np.all(a[self.T] == self.mark) and np.all(a[:, :lo] == self.mark) and np.all(a[:, lo + self.d:] == self.mark)


class Case:
    def __init__(self, T, d, pre="rms", post="none", gate="none", res="bfloat16", par="bfloat16", offset=False, scale=1.0,
                 group=128, pad=0, eps=1e-6, seed=0, level=0.5):
        self.c = dict(pre=pre, post=post, gate=gate, eps=eps, scale=np.float32(scale).item(), one=1.0 if offset else 0.0)
        self.T, self.d, self.res, self.par, self.group, self.pad, self.offset = T, d, res, par, group, pad, offset
        rng = self.rng = np.random.default_rng(seed + 1000 * T + d)
        normal = rng.standard_normal
        self.residual = br.as_type(normal((T, d)) + level * normal(d), res)
        self.y = br.bf16(0.7 * normal((T, d)) + 0.2)
        gain = lambda: br.as_type(0.2 * normal(d) + (0 if offset else 1), par)  # noqa: E731
        shift = lambda: br.as_type(0.1 * normal(d), par)  # noqa: E731
        self.p = dict(pre_gain=gain() if pre != "none" else None, pre_shift=shift() if pre == "layer" else None,
                      post_gain=gain() if post != "none" else None, post_shift=shift() if post == "layer" else None)
        self.gate = {"none": None, "channel": br.as_type(0.5 + 0.3 * normal(d), par),
                     "token": normal(T).astype(np.float32).astype(np.float64),
                     "element": br.bf16(0.5 + 0.3 * normal((T, d)))}[gate]

    def make(self):
        from persistent_megakernel_sm_gb300 import MoEBlockNorm
        c = self.c
        return MoEBlockNorm(self.d, pre=c["pre"], post=c["post"], gate=c["gate"], eps=c["eps"], scale=c["scale"],
                            unit_offset=self.offset, group=self.group)

    def params(self):
        out = {n: dev(v, self.par) for n, v in self.p.items()}
        kind = {"channel": self.par, "token": "float32", "element": "bfloat16"}.get(self.c["gate"])
        if self.c["gate"] == "element":
            out["gate"] = Wide(self.T, self.d, kind, self.pad).fill(self.gate, kind).rows
        else:
            out["gate"] = dev(self.gate, kind) if kind else None
        return out

    def held(self):
        import torch
        n = -(-self.d // self.group)
        return (torch.full((self.T, self.d), 9, dtype=torch.int8, device="cuda"),
                torch.full((self.T, n), 9.0, dtype=torch.bfloat16, device="cuda"))

    def forward(self, save=False, in_place=False, stats=True):
        import torch
        T, d = self.T, self.d
        r = Wide(T, d, self.res, self.pad).fill(self.residual, self.res)
        y = Wide(T, d, "bfloat16", self.pad).fill(self.y, "bfloat16")
        out = r if in_place else Wide(T, d, self.res, self.pad)
        norm = Wide(T, d, "bfloat16", self.pad) if self.c["pre"] != "none" else None
        st = torch.full((T, 4), 9.0, device="cuda") if stats else None
        out8, y8 = (self.held(), self.held()) if save else (None, None)
        n = self.make()
        n.forward(r.rows, y.rows, out.rows, norm.rows if norm else None, **self.params(), stats=st, out8=out8, y8=y8)
        torch.cuda.synchronize()
        assert out.untouched() and (norm is None or norm.untouched())
        return dict(out=host(out.rows), norm=host(norm.rows) if norm else None, stats=host(st), out8=out8, y8=y8)

    def check_forward(self, **how):
        got = self.forward(**how)
        want, my, ry, size = br.summed(self.c, self.residual, self.y, self.p, self.gate)
        half = U16 if self.res == "bfloat16" else br.U32
        assert np.all(np.abs(got["out"] - want) <= half * np.abs(want) + C32 * size)
        m, r = np.zeros((self.T, 1)), np.ones((self.T, 1))
        if got["norm"] is not None:  # of the rounded sum
            want, m, r, size = br.normed(self.c, got["out"], self.p)
            assert np.all(np.abs(got["norm"] - want) <= U16 * np.abs(want) + (1 + U16) * C32 * size)
        if got["stats"] is not None:
            s = got["stats"]
            for i, (mean, rstd, x) in enumerate(((my, ry, self.y), (m, r, got["out"]))):
                most = np.abs(x).mean(1)
                assert np.all(np.abs(s[:, 2 * i] - mean[:, 0]) <= C32 * most)
                # what x - m loses is relative to x and the mean, and rstd has half of it
                assert np.all(np.abs(s[:, 2 * i + 1] / rstd[:, 0] - 1) <= C32 * (1 + np.abs(mean[:, 0]) * rstd[:, 0]))
        if how.get("save"):
            for name, v, kind in (("out8", got["out"], self.res), ("y8", self.y, "bfloat16")):
                codes, scales = got[name]
                want_codes, want_scales = br.rows8(v, self.group, kind)
                assert np.array_equal(codes.cpu().numpy(), want_codes)
                assert np.array_equal(host(scales), want_scales)
        return got

    def backward(self, save=False, drop=(), in_place=False):
        """Gradients from inputs of their own; `drop`: names of gradients that are not given or not wanted."""
        import torch
        T, d, c = self.T, self.d, self.c
        rng = np.random.default_rng(7 + T + d)
        out, my, ry, _ = br.summed(c, self.residual, self.y, self.p, self.gate)
        out = br.as_type(out, self.res)
        m, r = br.moments(out, c["pre"], c["eps"])
        stats = np.concatenate((my, ry, m, r), 1).astype(np.float32).astype(np.float64)
        go = None if "grad_out" in drop else br.as_type(rng.standard_normal((T, d)), self.res)
        gn = None if "grad_norm" in drop or c["pre"] == "none" else br.bf16(rng.standard_normal((T, d)))
        need_y = "y" not in drop and (c["post"] != "none" or c["gate"] != "none")
        kept_out, kept_y = out, self.y
        wide = lambda a, kind: Wide(T, d, kind, self.pad).fill(a, kind).rows  # noqa: E731
        if save:
            held = []
            for v, kind in ((out, self.res), (self.y, "bfloat16")):
                codes, scales = br.rows8(v, self.group, kind)
                held.append((torch.from_numpy(codes).cuda(), dev(scales, "bfloat16")))
            t_out, t_y = held
            kept_out, kept_y = (br.rows8_values(h[0].cpu().numpy(), host(h[1]), self.group) for h in held)
        else:
            t_out, t_y = wide(out, self.res), wide(self.y, "bfloat16")
        want = br.backward(c, self.p, self.gate, stats, go, gn, kept_out if gn is not None else None, kept_y if need_y else None)
        params = self.params()
        grads = {"grad_" + n: torch.full((d,), 9.0, device="cuda") for n, v in self.p.items()
                 if v is not None and n in want and n not in drop}
        gate = None
        if self.gate is not None and "gate" in want and "gate" not in drop:
            gate = Wide(T, d, "bfloat16", self.pad) if c["gate"] == "element" else torch.full(
                (T if c["gate"] == "token" else d,), 9.0, device="cuda")
        tgo = None if go is None else Wide(T, d, self.res, self.pad).fill(go, self.res)
        gr = None if "residual" in drop else tgo if in_place else Wide(T, d, self.res, self.pad)
        gy = None if "y" in drop or ("y" not in want) else Wide(T, d, "bfloat16", self.pad)
        n = self.make()
        n.reserve()
        n.backward(None if tgo is None else tgo.rows, None if gn is None else wide(gn, "bfloat16"),
                   None if gr is None else gr.rows, None if gy is None else gy.rows,
                   stats=dev(stats), out=t_out if gn is not None else None, y=t_y if need_y else None, **params,
                   grad_gate=gate.rows if isinstance(gate, Wide) else gate, **grads)
        torch.cuda.synchronize()
        got = {k[5:]: host(v) for k, v in grads.items()}
        for name, t in (("residual", gr), ("y", gy), ("gate", gate)):
            if t is not None:
                got[name] = host(t.rows if isinstance(t, Wide) else t)
                assert not isinstance(t, Wide) or t.untouched()
        return got, want

    def check_backward(self, **how):
        got, want = self.backward(**how)
        for name, v in got.items():
            w, size = want[name]
            half = U16 if name == "y" or (name == "gate" and self.c["gate"] == "element") or (
                name == "residual" and self.res == "bfloat16") else br.U32
            # a sum over rows adds up to T roundings, those of a team and of the teams
            steps = B32 + (self.T * br.U32 if v.ndim == 1 and not (name == "gate" and self.c["gate"] == "token") else 0)
            assert np.all(np.abs(v - w) <= half * np.abs(w) + (1 + half) * steps * size), name
        return got


KINDS = [("rms", "none"), ("layer", "none"), ("rms", "rms"), ("layer", "layer"), ("none", "rms"), ("none", "layer"),
         ("layer", "rms"), ("none", "none")]
GATES = ["none", "channel", "token", "element"]


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("pre,post", KINDS)
def test_forward_kinds(pre, post, gate):
    for i, (T, d, pad) in enumerate(((5, 200, 0), (3, 77, 3))):
        Case(T, d, pre, post, gate, res=("bfloat16", "float32")[i], par=("float32", "bfloat16")[i], offset=bool(i),
             scale=0.5, pad=pad).check_forward(save=gate == "element")


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("pre,post", KINDS)
def test_backward_kinds(pre, post, gate):
    for i, (T, d, pad) in enumerate(((5, 200, 0), (3, 77, 3))):
        Case(T, d, pre, post, gate, res=("float32", "bfloat16")[i], par=("bfloat16", "float32")[i], offset=bool(i),
             scale=0.5, pad=pad).check_backward(save=gate in ("token", "element"))


WIDTHS = [1, 7, 8, 31, 64, 256, 264, 1000, 2047, 2048, 4096, 4097, 4104, 7168, 8200, 16384, 20000, 32768, 32767]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_widths(d, kind):
    for T, save in ((1, False), (3, True)):
        c = Case(T, d, kind, kind, "element" if d % 3 else "channel", res="float32" if d % 2 else "bfloat16", scale=0.3)
        c.check_forward(save=save)
        c.check_backward(save=save)


@pytest.mark.parametrize("T", [2, 151, 153, 700, 3000])
@pytest.mark.parametrize("d,pad", [(64, 0), (520, 8), (4104, 0), (333, 5)])
def test_rows_in_numbers(T, d, pad):
    c = Case(T, d, "rms", "layer", "token", pad=pad, group=32)
    c.check_forward(save=True, in_place=True)
    c.check_backward(in_place=True)


def test_a_large_mean_costs_a_layer_norm_nothing():
    """Squares about the mean are not taken from sums of squares: a level of 3000 deviations."""
    c = Case(4, 3000, "layer", "layer", res="float32")
    c.residual = (c.residual + 3000).astype(np.float32).astype(np.float64)
    c.y = br.bf16(0.5 * c.rng.integers(-1, 2, (4, 3000)) + 100)
    c.check_forward()


def test_rows_of_zeros_and_of_one_value():
    c = Case(3, 520, "layer", "rms", eps=1e-5)
    c.residual[0] = c.y[0] = 0
    c.residual[1], c.y[1] = 2.0, 0
    got = c.check_forward(save=True)
    assert np.all(np.isfinite(got["norm"]))
    c.check_backward()


@pytest.mark.parametrize("d", [520, 333, 4104])
def test_rows_that_are_not_finite_keep_to_themselves(d):
    c = Case(4, d, "layer", "rms", res="bfloat16")
    clean = c.forward(save=True)
    c.residual[1, d - 1], c.y[2, 0], c.residual[3, 5] = np.nan, np.inf, -np.inf
    got = c.forward(save=True)
    assert np.array_equal(got["norm"][0], clean["norm"][0]) and np.array_equal(got["out"][0], clean["out"][0])
    assert np.all(np.isnan(got["norm"][1:]))
    assert np.isnan(got["out"][1, d - 1]) and np.all(np.isfinite(got["out"][1, :d - 1]))
    scales = host(got["out8"][1])
    assert np.all(np.isfinite(scales[0])) and np.isnan(scales[1, -1]) and np.all(np.isfinite(scales[1, :-1]))


def test_the_first_blocks_norm_alone():
    import torch
    c = Case(9, 1000, "rms", "none")
    n, norm = c.make(), Wide(9, 1000, "bfloat16", 0)
    p = c.params()
    stats = torch.empty(9, 4, device="cuda")
    held = c.held()
    n.forward(dev(c.residual, "bfloat16"), None, None, norm.rows, **p, stats=stats, out8=held)
    want, m, r, size = br.normed(c.c, c.residual, c.p)
    got = host(norm.rows)
    assert np.all(np.abs(got - want) <= U16 * np.abs(want) + (1 + U16) * C32 * size)
    assert np.array_equal(held[0].cpu().numpy(), br.rows8(c.residual, 128, "bfloat16")[0])
    s = host(stats)
    assert np.all(s[:, 0] == 0) and np.all(s[:, 1] == 1)


@pytest.mark.parametrize("drop", [("grad_out",), ("grad_norm",), ("y",), ("residual",), ("pre_gain", "post_gain", "gate"),
                                  ("pre_shift", "post_shift")])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
def test_gradients_that_are_not_given_or_not_wanted(drop, gate):
    if "y" in drop:
        gate = "none"
    for d, pad in ((264, 0), (77, 3)):
        Case(6, d, "layer", "none" if "y" in drop else "layer", gate, pad=pad).check_backward(drop=drop)


def test_gradients_against_differences():
    """The reference's gradient is that of the forward pass in 64 bits."""
    for pre, post, gate in (("rms", "rms", "channel"), ("layer", "layer", "element"), ("layer", "rms", "token")):
        c = Case(3, 12, pre, post, gate, scale=0.7, offset=True, eps=1e-3)
        go, gn = c.rng.standard_normal((2, 3, 12))

        def loss(residual, y, p, g):
            out = br.summed(c.c, residual, y, p, g)[0]
            return (go * out).sum() + (gn * br.normed(c.c, out, p)[0]).sum()

        out, my, ry, _ = br.summed(c.c, c.residual, c.y, c.p, c.gate)
        stats = np.concatenate((my, ry, *br.moments(out, pre, 1e-3)), 1)
        want = br.backward(c.c, c.p, c.gate, stats, go, gn, out, c.y)
        base = dict(residual=c.residual, y=c.y, gate=c.gate, **c.p)
        for name, v in base.items():
            if v is None:
                continue
            for at in list(np.ndindex(v.shape))[::5]:
                diff = 0.0
                for sign in (1, -1):
                    w = v.copy()
                    w[at] += sign * 1e-5
                    b = {**base, name: w}
                    diff += sign * loss(b["residual"], b["y"], {n: b[n] for n in c.p}, b["gate"])
                assert abs(want[name][0][at] - diff / 2e-5) <= 1e-6 * (1 + np.abs(want[name][0]).max()), (name, at)


def test_the_same_bits_again_and_on_another_stream():
    import torch
    c = Case(400, 1000, "layer", "layer", "channel")
    first, _ = c.backward()
    again, _ = c.backward()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other, _ = c.backward()
    for k in first:
        assert np.array_equal(first[k], again[k]) and np.array_equal(first[k], other[k]), k


@pytest.mark.parametrize("d,res", [(1000, "bfloat16"), (77, "float32"), (7168, "bfloat16")])
def test_captured_passes(d, res):
    """Forward and backward in one graph, on new values in the old tensors: the bits of the eager passes."""
    import torch
    T = 40
    c = Case(T, d, "rms", "rms", "channel", res=res)
    n = c.make()
    n.reserve()
    dtype = getattr(torch, res)
    r, y = dev(c.residual, res), dev(c.y, "bfloat16")
    p = c.params()
    empty = lambda kind: torch.empty(T, d, dtype=kind, device="cuda")  # noqa: E731
    out, norm, stats, out8, y8 = empty(dtype), empty(torch.bfloat16), torch.empty(T, 4, device="cuda"), c.held(), c.held()
    go, gn = empty(dtype).normal_(), empty(torch.bfloat16).normal_()
    gr, gy = empty(dtype), empty(torch.bfloat16)
    grads = {k: torch.empty(d, device="cuda") for k in ("grad_pre_gain", "grad_post_gain", "grad_gate")}

    def step():
        n.forward(r, y, out, norm, **p, stats=stats, out8=out8, y8=y8)
        n.backward(go, gn, gr, gy, stats=stats, out=out8, y=y8, **p, **grads)

    every = [out, norm, stats, *out8, *y8, gr, gy, *grads.values()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        r.normal_(), y.normal_(), go.normal_()
        step()
        want = [t.clone() for t in every]
        for t in every:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(every, want))


def test_no_rows():
    import torch
    c = Case(0, 96, "layer", "layer", "channel")
    n = c.make()
    n.reserve()
    e = torch.empty(0, 96, dtype=torch.bfloat16, device="cuda")
    st = torch.empty(0, 4, device="cuda")
    p = c.params()
    n.forward(e, e, e, e, **p, stats=st)
    g = {k: torch.full((96,), 9.0, device="cuda") for k in ("grad_pre_gain", "grad_pre_shift", "grad_post_gain",
                                                            "grad_post_shift", "grad_gate")}
    n.backward(e, e, e, e, stats=st, out=e, y=e, **p, **g)
    assert all(torch.all(t == 0) for t in g.values())


def test_backward_needs_its_workspace():
    import torch
    from persistent_megakernel_sm_gb300 import MOE_E_STATE, MoEError
    c = Case(4, 64)
    n = c.make()
    t = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    st, p = torch.zeros(4, 4, device="cuda"), c.params()
    with pytest.raises(MoEError) as err:
        n.backward(t, t, t, None, stats=st, out=t, **p, grad_pre_gain=torch.empty(64, device="cuda"))
    assert err.value.code == MOE_E_STATE
    n.backward(t, t, torch.empty_like(t), None, stats=st, out=t, **p)  # none is used
    torch.cuda.synchronize()


def test_offsets_beyond_32_bits():
    """Rows whose elements are more than 2^31 into their tensors."""
    import torch
    from persistent_megakernel_sm_gb300 import MoEBlockNorm
    d, T = 512, 5
    stride = (1 << 31) // 4 + 8
    wide = torch.zeros(T, stride, dtype=torch.bfloat16, device="cuda")
    n = MoEBlockNorm(d, pre="rms")
    g = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    r = torch.randn(T, d, device="cuda").to(torch.bfloat16)
    y = torch.randn(T, d, device="cuda").to(torch.bfloat16)
    want = [torch.empty_like(r) for _ in range(2)]
    n.forward(r, y, *want, pre_gain=g)
    wide[:, :d], wide[:, d:2 * d] = r, y
    n.forward(wide[:, :d], wide[:, d:2 * d], wide[:, 2 * d:3 * d], wide[:, 3 * d:4 * d], pre_gain=g)
    assert torch.equal(wide[:, 2 * d:3 * d], want[0]) and torch.equal(wide[:, 3 * d:4 * d], want[1])


@pytest.mark.parametrize("d,pad", [(264, 0), (77, 3), (4104, 0)])
@pytest.mark.parametrize("post,gate", [("rms", "none"), ("layer", "token"), ("none", "element")])
def test_the_residuals_gradient_needs_nothing_of_the_block(d, pad, post, gate):
    """Without y: the gradients that go on through the residual stream, and the pre norm's."""
    got = Case(6, d, "layer", post, gate, pad=pad).check_backward(drop=("y", "gate"))
    assert set(got) == {"residual", "pre_gain", "pre_shift"}


def test_a_first_call_may_be_captured():
    """Kernels that no call has used before, in a graph at once."""
    import torch
    c = Case(5, 72, "layer", "rms", "element", res="float32", offset=True)
    want = c.forward()
    fresh = Case(5, 70, "layer", "layer", "token", res="float32", offset=True, pad=2, seed=3)
    n = fresh.make()
    n.reserve()
    p = fresh.params()
    r, y = Wide(5, 70, "float32", 2).fill(fresh.residual, "float32"), Wide(5, 70, "bfloat16", 2).fill(fresh.y, "bfloat16")
    out, norm, stats = Wide(5, 70, "float32", 2), Wide(5, 70, "bfloat16", 2), torch.empty(5, 4, device="cuda")
    gr, gain = Wide(5, 70, "float32", 2), torch.empty(70, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        n.forward(r.rows, y.rows, out.rows, norm.rows, **p, stats=stats)
        n.backward(out.rows, norm.rows, gr.rows, None, stats=stats, out=out.rows, y=y.rows, **p, grad_pre_gain=gain)
    graph.replay()
    torch.cuda.synchronize()
    got = [host(t) for t in (out.rows, norm.rows, gr.rows, gain)]
    for t in (out.rows, norm.rows, gr.rows, gain):
        t.zero_()
    n.forward(r.rows, y.rows, out.rows, norm.rows, **p, stats=stats)
    n.backward(out.rows, norm.rows, gr.rows, None, stats=stats, out=out.rows, y=y.rows, **p, grad_pre_gain=gain)
    assert all(np.array_equal(a, host(b)) for a, b in zip(got, (out.rows, norm.rows, gr.rows, gain)))
    assert np.all(np.isfinite(want["norm"]))


@pytest.mark.parametrize("d", [64, 1000, 4104])
def test_two_streams_share_a_handle_forward(d):
    """The handle holds settings alone in the forward pass: calls at once on two streams have their own rows' results."""
    import torch
    cases = [Case(300, d, "layer", "rms", "channel", seed=i) for i in range(2)]
    n = cases[0].make()
    p = cases[0].params()
    ins = [[dev(c.residual, "bfloat16"), dev(c.y, "bfloat16")] for c in cases]
    want = []
    for r, y in ins:
        want.append([torch.empty_like(r) for _ in range(2)])
        n.forward(r, y, *want[-1], **p)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.empty_like(t) for t in w] for w in want]
    for _ in range(20):
        for s, (r, y), g in zip(streams, ins, got):
            n.forward(r, y, *g, **p, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))


@pytest.mark.parametrize("d,pad", [(4104, 0), (8200, 0), (16392, 0), (32768, 0), (9001, 3)])
@pytest.mark.parametrize("pre,post,gate,res", [("rms", "rms", "channel", "bfloat16"), ("layer", "layer", "element", "float32")])
def test_wide_rows_of_long_batches(d, pad, pre, post, gate, res):
    """Rows enough for a lane to hold two eights, and so wide that a cluster shares each."""
    c = Case(310, d, pre, post, gate, res=res, pad=pad, scale=0.5, group=64)
    c.check_forward(save=d == 8200)
    c.check_backward(save=d == 8200)
