"""The routing operators' and 4-bit experts' refusals, on CPU: settings and
pointers that the C entries refuse before any launch, and tensors that the
binding refuses before any C call."""
import numpy as np
import pytest
import torch

import _ops_ref as ref
import persistent_megakernel_sm_gb300 as pkg
from persistent_megakernel_sm_gb300 import binding
from persistent_megakernel_sm_gb300 import build as cuda_build


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return pkg.load_library()


@pytest.mark.parametrize("args,ok", [
    # E, k, score, groups, kept, group score, renormalise, scale
    ((256, 8, 1, 8, 4, 1, 1, 2.5), True),
    ((1, 1, 0, 1, 1, 0, 0, 1.0), True),
    ((60, 16, 0, 1, 1, 0, 1, 1.0), True),
    ((257, 8, 0, 1, 1, 0, 1, 1.0), False),    # E > 256
    ((64, 17, 0, 1, 1, 0, 1, 1.0), False),    # k > 16
    ((4, 5, 0, 1, 1, 0, 1, 1.0), False),      # k > E
    ((64, 0, 0, 1, 1, 0, 1, 1.0), False),
    ((64, 8, 2, 1, 1, 0, 1, 1.0), False),     # no such score
    ((64, 8, 0, 7, 2, 0, 1, 1.0), False),     # groups do not divide E
    ((64, 1, 0, 64, 2, 0, 1, 1.0), False),    # over 32 groups
    ((64, 8, 0, 8, 9, 0, 1, 1.0), False),     # more groups kept than there are
    ((64, 8, 0, 8, 0, 0, 1, 1.0), False),
    ((64, 9, 0, 8, 1, 0, 1, 1.0), False),     # k > the kept groups' experts
    ((64, 8, 0, 8, 4, 2, 1, 1.0), False),     # no such group score
    ((64, 8, 0, 8, 4, 0, 2, 1.0), False),
    ((64, 8, 0, 8, 4, 0, 1, float("inf")), False),
    ((64, 8, 0, 8, 4, 0, 1, float("nan")), False),
])
def test_router_create_validates(lib, args, ok):
    h = lib.moe_router_create(*args)
    assert bool(h) == ok
    if ok:
        lib.moe_router_destroy(h)
    else:
        assert lib.moe_last_error()
    lib.moe_router_destroy(None)


def test_router_calls_validate(lib):
    h = lib.moe_router_create(64, 8, 0, 1, 1, 0, 1, 1.0)
    bad = pkg.MOE_E_INVAL
    try:
        fwd, bwd = lib.moe_router_forward, lib.moe_router_backward
        assert fwd(None, 4, 16, 0, 64, None, 16, 16, None, None) == bad
        assert fwd(h, -1, 16, 0, 64, None, 16, 16, None, None) == bad
        assert fwd(h, 4, 16, 2, 64, None, 16, 16, None, None) == bad      # type
        assert fwd(h, 4, None, 0, 64, None, 16, 16, None, None) == bad
        assert fwd(h, 4, 18, 0, 64, None, 16, 16, None, None) == bad      # alignment
        assert fwd(h, 4, 17, 1, 64, None, 16, 16, None, None) == bad
        assert fwd(h, 4, 16, 0, 63, None, 16, 16, None, None) == bad      # rows overlap
        assert fwd(h, 4, 16, 0, 64, None, None, 16, None, None) == bad
        assert fwd(h, 4, 16, 0, 64, None, 16, None, None, None) == bad
        assert fwd(h, 4, 16, 0, 64, 18, 16, 16, None, None) == bad
        assert fwd(h, 0, None, 0, 64, None, None, None, None, None) == pkg.MOE_OK
        assert bwd(None, 4, 16, 0, 64, 16, 16, 16, 64, None) == bad
        assert bwd(h, 4, 16, 0, 64, None, 16, 16, 64, None) == bad
        assert bwd(h, 4, 16, 0, 64, 16, None, 16, 64, None) == bad
        assert bwd(h, 4, 16, 0, 64, 16, 16, None, 64, None) == bad
        assert bwd(h, 4, 16, 0, 64, 16, 16, 18, 64, None) == bad
        assert bwd(h, 4, 16, 0, 64, 16, 16, 16, 63, None) == bad
        assert bwd(h, 0, None, 0, 64, None, None, None, 64, None) == pkg.MOE_OK
    finally:
        lib.moe_router_destroy(h)


def test_w4_conversion_validates(lib):
    for f in (lib.moe_w4_quantize, lib.moe_w4_dequantize):
        assert f(4, 256, 48, 16, 16, 16, None, None) == pkg.MOE_E_INVAL     # group
        assert f(4, 192, 128, 16, 16, 16, None, None) == pkg.MOE_E_INVAL    # cols % group
        assert f(-1, 256, 32, 16, 16, 16, None, None) == pkg.MOE_E_INVAL
        assert f(4, 256, 32, None, 16, 16, None, None) == pkg.MOE_E_INVAL
        assert f(4, 256, 32, 16, None, 16, None, None) == pkg.MOE_E_INVAL
        assert f(4, 256, 32, 16, 16, None, None, None) == pkg.MOE_E_INVAL
        assert f(4, 256, 32, 24, 16, 16, None, None) == pkg.MOE_E_INVAL     # alignment
        assert f(0, 256, 32, None, None, None, None, None) == pkg.MOE_OK
        assert f(4, 0, 32, None, None, None, None, None) == pkg.MOE_OK


@pytest.mark.parametrize("args,ok", [
    ((4096, 14336, 8, 2, 0, 128), True),
    ((2048, 768, 128, 8, 1, 32), True),
    ((100, 512, 8, 2, 0, 128), False),
    ((256, 200, 8, 2, 0, 128), False),
    ((256, 512, 300, 2, 0, 128), False),
    ((256, 512, 8, 9, 0, 128), False),
    ((256, 512, 8, 2, 2, 128), False),
    ((256, 512, 8, 2, 0, 256), False),
    ((32896, 512, 8, 2, 0, 128), False),
    ((256, 32896, 8, 2, 0, 128), False),
])
def test_w4_create_validates(lib, args, ok):
    h = lib.moe_w4_create(*args)
    assert bool(h) == ok
    if not ok:
        assert lib.moe_last_error()
    lib.moe_w4_destroy(h)


def test_w4_calls_validate(lib):
    h = lib.moe_w4_create(256, 512, 8, 2, 0, 128)
    try:
        assert lib.moe_w4_workspace_bytes(h, 0) >= 0
        assert lib.moe_w4_workspace_bytes(h, 256) >= 256 * 2 * 512 * 2
        assert lib.moe_w4_workspace_bytes(h, 1025) == -1
        assert lib.moe_w4_workspace_bytes(None, 4) == -1
        assert lib.moe_w4_reserve(h, 0, None) == pkg.MOE_E_INVAL
        assert lib.moe_w4_reserve(h, 1025, None) == pkg.MOE_E_INVAL
        assert lib.moe_w4_forward(h, 1, 16, 16, 16, 16, None) == pkg.MOE_E_STATE  # before reserve
        m = lambda *p: binding.ctypes.byref(binding._W4Weight(*p))  # noqa: E731
        good, zero = m(16, 16, None), m(16, 16, 16)
        assert lib.moe_w4_set_weights(h, good, good, good, None) == pkg.MOE_E_STATE  # before reserve
        assert lib.moe_w4_set_weights(h, good, good, zero, None) == pkg.MOE_E_INVAL  # some with zero points
        assert lib.moe_w4_set_weights(h, good, good, None, None) == pkg.MOE_E_INVAL
        assert lib.moe_w4_set_weights(h, m(None, 16, None), good, good, None) == pkg.MOE_E_INVAL
        assert lib.moe_w4_set_weights(h, m(16, 8, None), good, good, None) == pkg.MOE_E_INVAL
        assert lib.moe_w4_forward(None, 1, 16, 16, 16, 16, None) == pkg.MOE_E_INVAL
    finally:
        lib.moe_w4_destroy(h)
    lib.moe_w4_destroy(None)


def test_routed_forward_validates(lib):
    h = lib.moe_layer_create(2048, 768, 128, 8, 0)
    try:
        f, ptrs = lib.moe_layer_forward_routed, [16] * 4
        assert f(h, 1, 16, None, 16, *ptrs, None) == pkg.MOE_E_INVAL
        assert f(h, 1, 16, 16, None, *ptrs, None) == pkg.MOE_E_INVAL
        assert f(h, 1, 16, 18, 16, *ptrs, None) == pkg.MOE_E_INVAL
        assert f(h, 1, 16, 16, 17, *ptrs, None) == pkg.MOE_E_INVAL
        assert f(h, 1, 16, 16, 16, *ptrs, None) == pkg.MOE_E_STATE  # before reserve
        assert f(None, 1, 16, 16, 16, *ptrs, None) == pkg.MOE_E_INVAL
    finally:
        lib.moe_layer_destroy(h)


# ---- the binding's checks, with the library replaced by a recorder

class _OnDevice(torch.Tensor):
    """A host tensor that reports itself as a CUDA tensor (test stand-in)."""

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return 0


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 1 if name.endswith("_create") else 0
        return call


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder()
    monkeypatch.setattr(binding, "lib", r)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    yield r


def _dev(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnDevice)


def test_router_binding_passes_and_refuses(rec):
    r = binding.MoERouter(64, 6, score="sigmoid", groups=8, groups_kept=4)
    idx, w = _dev(5, 6, dtype=torch.int32), _dev(5, 6)
    wide = _dev(5, 80)
    r.forward(_dev(5, 64), idx, w, stream=0)
    r.forward(wide[:, :64], idx, w, bias=_dev(64), counts=_dev(64, dtype=torch.int32), stream=0)
    r.forward(_dev(0, 64, dtype=torch.bfloat16), idx[:0], w[:0], stream=0)
    r.backward(wide[:, 16:], idx, w, _dev(5, 64), stream=0)
    assert rec.calls.count("moe_router_forward") == 3 and "moe_router_backward" in rec.calls
    before = list(rec.calls)
    bad = [
        lambda: r.forward(_dev(5, 64, dtype=torch.float16), idx, w, stream=0),
        lambda: r.forward(_dev(5, 63), idx, w, stream=0),
        lambda: r.forward(_dev(64, 5).t(), idx, w, stream=0),
        lambda: r.forward(_dev(1, 64).expand(5, 64), idx, w, stream=0),
        lambda: r.forward(torch.zeros(5, 64), idx, w, stream=0),
        lambda: r.forward(_dev(5, 64), idx.long(), w, stream=0),
        lambda: r.forward(_dev(5, 64), idx[:4], w, stream=0),
        lambda: r.forward(_dev(5, 64), idx, _dev(5, 12)[:, ::2], stream=0),
        lambda: r.forward(_dev(5, 64), idx, w, bias=_dev(64, dtype=torch.bfloat16), stream=0),
        lambda: r.forward(_dev(5, 64), idx, w, counts=_dev(64), stream=0),
        lambda: r.backward(_dev(5, 64), idx, w, _dev(5, 64, dtype=torch.bfloat16), stream=0),
        lambda: r.backward(_dev(5, 64), idx, w, _dev(4, 64), stream=0),
        lambda: r.backward(_dev(5, 64), idx, w[:4], _dev(5, 64), stream=0),
    ]
    for call in bad:
        with pytest.raises(binding.MoEError) as err:
            call()
        assert err.value.code == binding.MOE_E_INVAL
    with pytest.raises(binding.MoEError):
        binding.MoERouter(64, 6, score="tanh")
    assert rec.calls == before
    r.close()


def test_routed_binding_passes_and_refuses(rec):
    bf = torch.bfloat16
    layer = binding.MoELayer(256, 384, 8, 2, 1)
    gate, down, x = _dev(9, 384, 256, dtype=bf), _dev(9, 256, 384, dtype=bf), _dev(5, 256, dtype=bf)
    idx, w = _dev(5, 2, dtype=torch.int32), _dev(5, 2)
    layer.forward_routed(x, idx, w, gate, gate, down, x, stream=0)
    assert "moe_layer_forward_routed" in rec.calls
    before = list(rec.calls)
    for args in ((x, idx.long(), w, gate, gate, down, x), (x, idx[:4], w, gate, gate, down, x),
                 (x, idx, w.to(bf), gate, gate, down, x), (x, idx, w, down, gate, down, x),
                 (x, idx, w, gate, gate, gate, x), (x.float(), idx, w, gate, gate, down, x),
                 (x, idx, w, gate, gate, down, x[:4])):
        with pytest.raises(binding.MoEError) as err:
            layer.forward_routed(*args, stream=0)
        assert err.value.code == binding.MOE_E_INVAL
    assert rec.calls == before
    layer.close()


def test_w4_binding_passes_and_refuses(rec):
    u8, bf = torch.uint8, torch.bfloat16
    mat = lambda n, rows, cols, g=32, z=True: (_dev(n, rows, cols // 2, dtype=u8), _dev(n, rows, cols // g, dtype=bf),  # noqa: E731
                                               _dev(n, rows, cols // g, dtype=u8) if z else None)
    c, s, z = mat(3, 8, 256)
    w = _dev(3, 8, 256, dtype=bf)
    binding.w4_quantize(w, c, s, z, stream=0)
    binding.w4_quantize(w[0], c[0], s[0], stream=0)
    binding.w4_dequantize(c, s, None, w, stream=0)
    e = binding.W4Experts(256, 384, 3, 2, shared_experts=1, group=32)
    gate, down = mat(4, 384, 256), mat(4, 256, 384)
    e.set_weights(gate, gate, down, stream=0)
    x, idx, wt = _dev(7, 256, dtype=bf), _dev(7, 2, dtype=torch.int32), _dev(7, 2)
    e.forward(x, idx, wt, _dev(7, 256, dtype=bf), stream=0)
    assert "moe_w4_forward" in rec.calls and rec.calls.count("moe_w4_quantize") == 2
    before = list(rec.calls)
    bad = [
        lambda: binding.w4_quantize(w.float(), c, s, stream=0),
        lambda: binding.w4_quantize(w, c[:2], s, stream=0),
        lambda: binding.w4_quantize(w, c, _dev(3, 8, 16, dtype=bf), stream=0),       # groups of 16
        lambda: binding.w4_quantize(w, c, _dev(3, 8, 3, dtype=bf), stream=0),
        lambda: binding.w4_quantize(w, c, s.float(), stream=0),
        lambda: binding.w4_quantize(w.transpose(1, 2), c, s, stream=0),
        lambda: binding.w4_dequantize(c, s, z.int(), w, stream=0),
        lambda: e.set_weights(down, gate, down, stream=0),
        lambda: e.set_weights(gate, gate, mat(3, 256, 384), stream=0),
        lambda: e.set_weights(mat(4, 384, 256, 64), gate, down, stream=0),
        lambda: e.forward(x.float(), idx, wt, x, stream=0),
        lambda: e.forward(x, idx.long(), wt, x, stream=0),
        lambda: e.forward(x, idx, wt[:6], x, stream=0),
        lambda: e.forward(x, idx, wt, x[:6], stream=0),
        lambda: e.forward(x, idx, wt, torch.zeros(7, 256, dtype=bf), stream=0),
    ]
    for call in bad:
        with pytest.raises(binding.MoEError) as err:
            call()
        assert err.value.code == binding.MOE_E_INVAL
    assert rec.calls == before
    e.close()


# ---- the references themselves

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_reference_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    r = dict(E=12, k=4, score=score, groups=1, groups_kept=1, group_score="max", renormalise=renorm, scale=1.5)
    l = rng.standard_normal((3, 12))
    idx, _ = ref.route(l, r)
    gw = rng.standard_normal((3, 4))
    grad, size = ref.route_grad(l, r, idx, gw)
    assert np.all(np.abs(grad) <= size + 1e-12)
    for e in range(12):
        step = np.zeros_like(l)
        step[:, e] = 1e-5
        # the choice stays as it was: a weight of the differences is that of the same experts
        hi, lo = (_weights_of(l + q, r, idx) for q in (step, -step))
        diff = ((hi - lo) * gw).sum(1) / 2e-5
        assert np.allclose(grad[:, e], diff, atol=1e-8)


def _weights_of(l, r, idx):
    s = np.take_along_axis(ref.scores(l, r["score"]), idx.astype(np.int64), 1)
    return r["scale"] * (s / s.sum(1, keepdims=True) if r["renormalise"] else s)


@pytest.mark.parametrize("zeros", [False, True])
def test_reference_conversion_is_within_half_a_step(zeros):
    rng = np.random.default_rng(5)
    w = ref.bf16(rng.standard_normal((16, 256)))
    codes, s, z = ref.quantize(w, 64, zeros)
    step = np.repeat(s, 64, -1)
    # half a step, and where the scale was rounded down the ends of the range
    # lie up to 15 (7) steps x 2^-8 beyond the last code; the zero point's
    # rounding moves the range by up to half a step more
    slack = (0.5 + (0.5 if zeros else 0.0) + 15 * ref.U16) * step
    assert np.all(np.abs(ref.values(codes, s, z) - w) <= slack)
