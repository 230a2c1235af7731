"""The refusals of the norms about a block, 8-bit rows and the layer for a few
tokens, on CPU: what the C entries refuse before any launch, and tensors that the
binding refuses before any C call; and the references themselves."""
import ctypes

import numpy as np
import pytest
import torch

import _block_ref as br
import persistent_megakernel_sm_gb300 as pkg
from persistent_megakernel_sm_gb300 import binding
from persistent_megakernel_sm_gb300 import build as cuda_build
from test_ops_host import _dev, rec  # noqa: F401

BAD = pkg.MOE_E_INVAL
bf, f32, i8 = torch.bfloat16, torch.float32, torch.int8


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return pkg.load_library()


# ------------------------------------------------------------------- 8-bit rows

def test_rows8_calls_validate(lib):
    for f in (lib.moe_rows8_quantize, lib.moe_rows8_dequantize):
        assert f(4, 100, 1, 48, 16, 16, 16, None) == BAD         # group
        assert f(4, 100, 2, 32, 16, 16, 16, None) == BAD         # type
        assert f(-1, 100, 1, 32, 16, 16, 16, None) == BAD
        assert f(4, -1, 1, 32, 16, 16, 16, None) == BAD
        assert f(4, 100, 1, 32, None, 16, 16, None) == BAD
        assert f(4, 100, 1, 32, 16, None, 16, None) == BAD
        assert f(4, 100, 1, 32, 16, 16, None, None) == BAD
        assert f((1 << 38) + 1, 1, 1, 32, 16, 16, 16, None) == BAD
        assert f(1 << 37, 1, 1, 32, 16, 16, 16, None) == BAD     # more blocks than a grid has
        assert f(1, (1 << 30) + 1, 1, 32, 16, 16, 16, None) == BAD
        assert f(0, 100, 1, 32, None, None, None, None) == pkg.MOE_OK
        assert f(4, 0, 1, 32, None, None, None, None) == pkg.MOE_OK
    assert lib.moe_rows8_quantize(4, 100, 0, 32, 18, 16, 16, None) == BAD    # alignment
    assert lib.moe_rows8_quantize(4, 100, 1, 32, 17, 16, 16, None) == BAD
    assert lib.moe_rows8_quantize(4, 100, 1, 32, 16, 16, 17, None) == BAD


def test_counts_beyond_the_c_calls_ints_are_refused(rec):  # noqa: F811
    """A C int would take 2^32 + 4 for 4."""
    many = (1 << 32) + 4
    wide = torch.zeros(1, dtype=bf).expand(1, many).as_subclass(type(_dev(1)))
    tall = torch.zeros(1, 64, dtype=bf).expand(many, 64).as_subclass(type(_dev(1)))
    n = binding.MoEBlockNorm(64)
    for call in (lambda: binding.rows8_quantize(wide, wide, wide, stream=0), lambda: n.forward(tall, None, None, tall, stream=0),
                 lambda: n.backward(tall, None, tall, None, stream=0)):
        with pytest.raises(binding.MoEError) as err:
            call()
        assert err.value.code == BAD
    assert not [c for c in rec.calls if "quantize" in c or "ward" in c]
    n.close()


def test_rows8_binding_passes_and_refuses(rec):  # noqa: F811
    v, c, s = _dev(3, 5, 100, dtype=bf), _dev(3, 5, 100, dtype=i8), _dev(3, 5, 4, dtype=bf)
    binding.rows8_quantize(v, c, s, group=32, stream=0)
    binding.rows8_dequantize(c, s, v.float(), group=32, stream=0)
    binding.rows8_quantize(_dev(0, 64, dtype=bf), _dev(0, 64, dtype=i8), _dev(0, 1, dtype=bf), stream=0)
    assert rec.calls.count("moe_rows8_quantize") == 2 and "moe_rows8_dequantize" in rec.calls
    before = list(rec.calls)
    for call in (lambda: binding.rows8_quantize(v.half(), c, s, group=32, stream=0),
                 lambda: binding.rows8_quantize(v, c, s, group=64, stream=0),
                 lambda: binding.rows8_quantize(v, c, s, group=33, stream=0),
                 lambda: binding.rows8_quantize(v, c[:2], s, group=32, stream=0),
                 lambda: binding.rows8_quantize(v, c.to(torch.uint8), s, group=32, stream=0),
                 lambda: binding.rows8_quantize(v, c, s.float(), group=32, stream=0),
                 lambda: binding.rows8_quantize(v.transpose(0, 1), c.transpose(0, 1), s, group=32, stream=0),
                 lambda: binding.rows8_quantize(torch.zeros(3, 5, 100, dtype=bf), c, s, group=32, stream=0),
                 lambda: binding.rows8_quantize(v[0, 0, 0], c, s, group=32, stream=0),
                 lambda: binding.rows8_dequantize(c, s, v[:, :, :50], group=32, stream=0)):
        with pytest.raises(binding.MoEError) as err:
            call()
        assert err.value.code == BAD
    assert rec.calls == before


# ------------------------------------------------------------------------ norms

@pytest.mark.parametrize("args,ok", [
    # d, pre, post, gate, eps, scale, unit offset, group
    ((4096, 1, 1, 1, 1e-6, 1.0, 0, 128), True),
    ((1, 0, 0, 0, 0.0, -2.0, 1, 32), True),
    ((32768, 2, 2, 3, 1e-5, 0.0, 0, 64), True),
    ((0, 1, 0, 0, 1e-6, 1.0, 0, 128), False),
    ((32769, 1, 0, 0, 1e-6, 1.0, 0, 128), False),
    ((64, 3, 0, 0, 1e-6, 1.0, 0, 128), False),
    ((64, 1, -1, 0, 1e-6, 1.0, 0, 128), False),
    ((64, 1, 0, 4, 1e-6, 1.0, 0, 128), False),
    ((64, 1, 0, 0, -1e-6, 1.0, 0, 128), False),
    ((64, 1, 0, 0, float("nan"), 1.0, 0, 128), False),
    ((64, 1, 0, 0, float("inf"), 1.0, 0, 128), False),
    ((64, 1, 0, 0, 1e-6, float("inf"), 0, 128), False),
    ((64, 1, 0, 0, 1e-6, 1.0, 2, 128), False),
    ((64, 1, 0, 0, 1e-6, 1.0, 0, 48), False),
])
def test_norm_create_validates(lib, args, ok):
    h = lib.moe_norm_create(*args)
    assert bool(h) == ok
    if ok:
        assert lib.moe_norm_workspace_bytes(h) >= args[0] * 16
    else:
        assert lib.moe_last_error()
    lib.moe_norm_destroy(h)
    assert lib.moe_norm_workspace_bytes(None) == -1
    assert lib.moe_norm_reserve(None, None) == BAD


def _params(**v):
    p = binding._NormParams()
    p.type = 1
    for n, x in v.items():
        setattr(p, n, x)
    return ctypes.byref(p)


def _fwd(lib, h, T=4, kind=1, r=64, rs=64, y=64, ys=64, p=None, out=128, os=64, n=64, ns=64, st=None, out8=None, y8=None):
    return lib.moe_norm_forward(h, T, kind, r, rs, y, ys, p or _params(pre_gain=16), out, os, n, ns, st, out8, y8, None)


def test_norm_forward_validates(lib):
    rms, layer = lib.moe_norm_create(64, 1, 0, 0, 1e-6, 1.0, 0, 128), lib.moe_norm_create(64, 2, 2, 3, 1e-6, 1.0, 0, 128)
    none = lib.moe_norm_create(64, 0, 0, 0, 1e-6, 1.0, 0, 128)
    held = lambda c, s: ctypes.byref(binding._Rows8(c, s))  # noqa: E731
    try:
        bad = [dict(T=-1), dict(T=(1 << 30) + 1), dict(rs=1 << 31), dict(kind=2), dict(r=None), dict(rs=63), dict(ys=63), dict(os=63), dict(ns=63), dict(r=17),
               dict(r=18, kind=0), dict(y=17), dict(n=17), dict(y=None), dict(out=None), dict(n=None), dict(st=8),
               dict(out8=held(None, 16)), dict(out8=held(16, None)), dict(y8=held(16, 18)), dict(out=64, os=72),
               dict(y=None, out=None, y8=held(16, 16)), dict(p=_params(pre_gain=17)), dict(p=_params(pre_shift=16)),
               dict(p=_params(post_gain=16)), dict(p=_params(gate=16)), dict(p=_params(type=2))]
        for how in bad:
            assert _fwd(lib, rms, **how) == BAD, how
        assert _fwd(lib, None) == BAD
        assert lib.moe_norm_forward(rms, 4, 1, 64, 64, 64, 64, None, 128, 64, 64, 64, None, None, None, None) == BAD
        for p in (_params(), _params(gate=16, gate_stride=63), _params(gate=17, gate_stride=64)):
            assert _fwd(lib, layer, p=p) == BAD
        assert _fwd(lib, layer, p=_params(gate=16, gate_stride=64), y=None, out=None) == BAD
        assert _fwd(lib, none) == BAD                                       # a norm that it does not have
        assert _fwd(lib, none, p=_params(), n=None, y=None, out=None) == BAD  # nothing to do
        assert _fwd(lib, rms, T=0, r=None, y=None, out=None, n=None) == pkg.MOE_OK
    finally:
        for h in (rms, layer, none):
            lib.moe_norm_destroy(h)


def _bwd(lib, h, T=4, kind=1, go=64, gos=64, gn=64, gns=64, p=None, kept=None, gr=128, grs=64, gy=128, gys=64, grads=None):
    k = binding._NormKept()
    for n, v in (kept if kept is not None else dict(out=64, out_stride=64, y=64, y_stride=64, stats=64)).items():
        setattr(k, n, v)
    g = binding._NormGrads()
    for n, v in (grads or {}).items():
        setattr(g, n, v)
    return lib.moe_norm_backward(h, T, kind, go, gos, gn, gns, p or _params(pre_gain=16), ctypes.byref(k), gr, grs, gy, gys,
                                 ctypes.byref(g), None)


def test_norm_backward_validates(lib):
    rms, layer = lib.moe_norm_create(64, 1, 0, 0, 1e-6, 1.0, 0, 128), lib.moe_norm_create(64, 2, 2, 3, 1e-6, 1.0, 0, 128)
    none = lib.moe_norm_create(64, 0, 0, 0, 1e-6, 1.0, 0, 128)
    held = ctypes.addressof(binding._Rows8(16, 16))
    half = binding._Rows8(16, None)
    full = dict(out=64, out_stride=64, y=64, y_stride=64, stats=64)
    lp = _params(pre_gain=16, gate=16, gate_stride=64)
    try:
        bad = [dict(T=-1), dict(T=(1 << 30) + 1), dict(gos=1 << 31), dict(kind=2), dict(go=None, gn=None), dict(gos=63), dict(gns=63), dict(grs=63), dict(gys=63),
               dict(go=17), dict(gn=17), dict(gr=17), dict(gy=17), dict(go=128, gos=72), dict(gr=None, gy=None),
               dict(kept=dict(full, out=None)), dict(kept=dict(full, stats=None)), dict(kept=dict(full, stats=8)),
               dict(kept=dict(full, out_stride=63)), dict(kept=dict(full, out8=ctypes.addressof(half))),
               dict(grads=dict(post_gain=16)), dict(grads=dict(pre_shift=16)), dict(grads=dict(gate=16)),
               dict(grads=dict(pre_gain=18))]
        for how in bad:
            assert _bwd(lib, rms, **how) == BAD, how
        del held
        assert _bwd(lib, None) == BAD
        assert lib.moe_norm_backward(rms, 4, 1, 64, 64, 64, 64, _params(), None, 64, 64, 64, 64, None, None) == BAD
        assert _bwd(lib, rms, grads=dict(pre_gain=16)) == pkg.MOE_E_STATE   # before reserve
        assert _bwd(lib, layer, p=lp, kept=dict(full, y=None)) == BAD       # grad_y through the post norm needs y
        assert _bwd(lib, layer, p=lp, gy=None, kept=dict(full, y=None), grads=dict(gate=16, gate_stride=64)) == BAD
        assert _bwd(lib, layer, p=lp, grads=dict(gate=16, gate_stride=63)) == BAD
        assert _bwd(lib, layer, p=lp, gn=None, grads=dict(pre_gain=16)) in (BAD, pkg.MOE_E_STATE)
        assert _bwd(lib, none, p=_params()) == BAD                          # the gradient of a norm that it does not have
        assert _bwd(lib, rms, T=0) == pkg.MOE_OK
    finally:
        for h in (rms, layer, none):
            lib.moe_norm_destroy(h)


def test_norm_binding_passes_and_refuses(rec):  # noqa: F811
    n = binding.MoEBlockNorm(64, pre="layer", post="rms", gate="element", group=32)
    T = 5
    t = lambda dtype=bf, w=64: _dev(T, w, dtype=dtype)  # noqa: E731
    g = _dev(64, dtype=bf)
    held = (t(i8), _dev(T, 2, dtype=bf))
    n.forward(t(), t(), t(), t(), pre_gain=g, pre_shift=g, post_gain=g, gate=t(w=80)[:, :64], stats=_dev(T, 4), out8=held,
              y8=held, stream=0)
    n.forward(t(f32), t(), t(f32), t(), pre_gain=_dev(64), gate=t(), stream=0)
    n.reserve(stream=0)
    n.backward(t(), t(), t(), t(), stats=_dev(T, 4), out=t(), y=t(), pre_gain=g, post_gain=g, gate=t(), grad_gate=t(),
               grad_pre_gain=_dev(64), grad_post_gain=_dev(64), stream=0)
    n.backward(t(f32), t(), t(f32), t(), stats=_dev(T, 4), out=held, y=held, gate=t(), stream=0)
    n.backward(None, t(), None, t(), stats=_dev(T, 4), out=held, y=held, gate=t(), stream=0)
    assert rec.calls.count("moe_norm_forward") == 2 and rec.calls.count("moe_norm_backward") == 3
    before = list(rec.calls)
    ok = dict(pre_gain=g, gate=t(), stream=0)
    bad = [
        lambda: n.forward(t(torch.float16), t(), t(torch.float16), t(), **ok),
        lambda: n.forward(t(), t(f32), t(), t(), **ok),
        lambda: n.forward(t(), t(), t(f32), t(), **ok),
        lambda: n.forward(t(), t(), t(), t(f32), **ok),
        lambda: n.forward(t(), t(w=63), t(), t(), **ok),
        lambda: n.forward(t(), t()[:4], t(), t(), **ok),
        lambda: n.forward(_dev(64, T, dtype=bf).t(), t(), t(), t(), **ok),
        lambda: n.forward(_dev(1, 64, dtype=bf).expand(T, 64), t(), t(), t(), **ok),
        lambda: n.forward(torch.zeros(T, 64, dtype=bf), t(), t(), t(), **ok),
        lambda: n.forward(t(), t(), t(), t(), pre_gain=g, post_gain=_dev(64), gate=t(), stream=0),   # types differ
        lambda: n.forward(t(), t(), t(), t(), pre_gain=_dev(63, dtype=bf), gate=t(), stream=0),
        lambda: n.forward(t(), t(), t(), t(), pre_gain=g, gate=t(f32), stream=0),
        lambda: n.forward(t(), t(), t(), t(), stats=_dev(T, 3), **ok),
        lambda: n.forward(t(), t(), t(), t(), stats=_dev(T, 4, dtype=bf), **ok),
        lambda: n.forward(t(), t(), t(), t(), out8=(t(i8), _dev(T, 1, dtype=bf)), **ok),
        lambda: n.forward(t(), t(), t(), t(), y8=(t(torch.uint8), _dev(T, 2, dtype=bf)), **ok),
        lambda: n.backward(None, None, t(), t(), **ok),
        lambda: n.backward(t(), t(), t(f32), t(), stats=_dev(T, 4), out=t(), y=t(), **ok),
        lambda: n.backward(t(), t(f32), t(), t(), stats=_dev(T, 4), out=t(), y=t(), **ok),
        lambda: n.backward(t(), t(), t(), t(), stats=_dev(T, 4), out=t(f32), y=t(), **ok),
        lambda: n.backward(t(), t(), t(), t(), stats=_dev(T, 4), out=t(), y=t(), grad_pre_gain=_dev(64, dtype=bf), **ok),
        lambda: n.backward(t(), t(), t(), t(), stats=_dev(T, 4), out=t(), y=t(), grad_gate=t(f32), **ok),
    ]
    for call in bad:
        with pytest.raises(binding.MoEError) as err:
            call()
        assert err.value.code == BAD
    for kw in (dict(pre="mean"), dict(post="batch"), dict(gate="row")):
        with pytest.raises(binding.MoEError):
            binding.MoEBlockNorm(64, **kw)
    with pytest.raises(binding.MoEError):
        binding.MoEBlockNorm(64).forward(t(), t(), t(), t(), gate=g, stream=0)   # it has none
    assert [c for c in rec.calls if c in ("moe_norm_forward", "moe_norm_backward")] == [
        c for c in before if c in ("moe_norm_forward", "moe_norm_backward")]
    n.close()


# ------------------------------------------------------- the layer for a few tokens

@pytest.mark.parametrize("args,ok", [
    ((4096, 14336, 8, 2, 0), True),
    ((2048, 768, 128, 8, 1), True),
    ((32768, 32768, 1, 1, 0), True),
    ((100, 512, 8, 2, 0), False),
    ((256, 200, 8, 2, 0), False),
    ((256, 512, 300, 2, 0), False),
    ((256, 512, 8, 9, 0), False),
    ((256, 512, 64, 17, 0), False),
    ((256, 512, 8, 0, 0), False),
    ((256, 512, 8, 2, 2), False),
    ((32896, 512, 8, 2, 0), False),
    ((256, 32896, 8, 2, 0), False),
])
def test_decode_create_validates(lib, args, ok):
    h = lib.moe_decode_create(*args)
    assert bool(h) == ok
    if not ok:
        assert lib.moe_last_error()
    lib.moe_decode_destroy(h)


def test_decode_calls_validate(lib):
    h = lib.moe_decode_create(256, 512, 8, 2, 1)
    try:
        assert lib.moe_decode_workspace_bytes(h, 16) >= 16 * 3 * 512 * 4
        assert lib.moe_decode_workspace_bytes(h, 17) == -1 and lib.moe_decode_workspace_bytes(None, 1) == -1
        assert lib.moe_decode_reserve(h, 0, None) == BAD and lib.moe_decode_reserve(h, 17, None) == BAD
        assert lib.moe_decode_reserve(None, 1, None) == BAD
        own, routed = lib.moe_decode_forward, lib.moe_decode_forward_routed
        assert own(None, 1, 16, 16, None, 16, 16, 16, 16, None, None, None) == BAD
        assert routed(None, 1, 16, 16, 16, 16, 16, 16, 16, None) == BAD
        assert own(h, 1, 16, 16, None, 16, 16, 16, 16, None, None, None) == pkg.MOE_E_STATE  # before reserve
        assert routed(h, 1, 16, 16, 16, 16, 16, 16, 16, None) == pkg.MOE_E_STATE
        assert lib.moe_decode_status(None, None) == BAD and lib.moe_decode_status(h, None) == pkg.MOE_E_STATE
    finally:
        lib.moe_decode_destroy(h)
    lib.moe_decode_destroy(None)


def test_decode_binding_passes_and_refuses(rec):  # noqa: F811
    n = binding.MoEDecode(256, 384, 8, 2, 1)
    n.reserve(16, stream=0)
    gate, down, x = _dev(9, 384, 256, dtype=bf), _dev(9, 256, 384, dtype=bf), _dev(5, 256, dtype=bf)
    r, idx, w = _dev(8, 256, dtype=bf), _dev(5, 2, dtype=torch.int32), _dev(5, 2)
    n.forward(x, r, gate, gate, down, x, stream=0)
    n.forward(x, r, gate, gate, down, x, bias=_dev(8), idx=idx, w=w, stream=0)
    n.forward_routed(x, idx, w, gate, gate, down, x, stream=0)
    assert rec.calls.count("moe_decode_forward") == 2 and "moe_decode_forward_routed" in rec.calls
    before = list(rec.calls)
    own = lambda *a, **k: (lambda: n.forward(*a, **k, stream=0))  # noqa: E731
    routed = lambda *a: (lambda: n.forward_routed(*a, stream=0))  # noqa: E731
    for call in (own(x.float(), r, gate, gate, down, x), own(x, r[:7], gate, gate, down, x), own(x, r, down, gate, down, x),
                 own(x, r, gate, gate[:8], down, x), own(x, r, gate, gate, gate, x), own(x, r, gate, gate, down, x[:4]),
                 own(x, r, gate, gate, down, torch.zeros(5, 256, dtype=bf)),
                 own(x, r, gate, gate, down, x, bias=_dev(8, dtype=bf)), own(x, r, gate, gate, down, x, idx=idx.long()),
                 own(x, r, gate, gate, down, x, w=w[:4]), routed(x, idx.long(), w, gate, gate, down, x),
                 routed(x, idx, w.to(bf), gate, gate, down, x), routed(x, idx[:4], w, gate, gate, down, x),
                 routed(x, idx, _dev(5, 4)[:, ::2], gate, gate, down, x)):
        with pytest.raises(binding.MoEError) as err:
            call()
        assert err.value.code == BAD
    assert rec.calls == before
    n.close()


# ---------------------------------------------------------- the references themselves

def test_reference_rows_are_within_half_a_step():
    rng = np.random.default_rng(5)
    v = br.bf16(rng.standard_normal((16, 200)))
    codes, s = br.rows8(v, 64, "bfloat16")
    # half a step, and where the scale was rounded down the largest value lies up to
    # 127 steps x 2^-8 beyond the last code
    assert np.all(np.abs(br.rows8_values(codes, s, 64) - v) <= (0.5 + 127 * 2.0 ** -8) * np.repeat(s, 64, 1)[:, :200])


@pytest.mark.parametrize("pre,post,gate", [("rms", "rms", "channel"), ("layer", "layer", "element"), ("layer", "rms", "token")])
def test_reference_gradient_is_within_its_size(pre, post, gate):
    rng = np.random.default_rng(2)
    T, d = 4, 20
    c = dict(pre=pre, post=post, gate=gate, eps=1e-6, scale=0.5, one=0.0)
    r, y, go, gn = rng.standard_normal((4, T, d))
    p = dict(pre_gain=rng.standard_normal(d), pre_shift=None, post_gain=rng.standard_normal(d), post_shift=rng.standard_normal(d))
    g = {"channel": rng.standard_normal(d), "token": rng.standard_normal(T), "element": rng.standard_normal((T, d))}[gate]
    out, my, ry, size = br.summed(c, r, y, p, g)
    assert np.all(np.abs(out) <= size * (1 + 1e-12))
    stats = np.concatenate((my, ry, *br.moments(out, pre, 1e-6)), 1)
    for name, (v, size) in br.backward(c, p, g, stats, go, gn, out, y).items():
        assert np.all(np.abs(v) <= size * (1 + 1e-12)), name
