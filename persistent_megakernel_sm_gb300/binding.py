"""ctypes binding of include/moe.h: argument marshalling only.

Each C entry point is exposed under its own name on ``lib`` (a ``ctypes.CDLL``
with argument and return types set from the header).  ``MoELayer`` wraps a
handle for callers holding torch tensors: it passes ``data_ptr()`` values and
the current CUDA stream, and turns non-zero status codes into ``MoEError``.
Every step of the layer runs in the library's kernels.  ``MoERouter``,
``w4_quantize`` / ``w4_dequantize`` and ``W4Experts`` do the same for the
routing operator and the 4-bit experts.
"""
from __future__ import annotations

import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libmoe.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "moe.h")

MOE_OK, MOE_E_INVAL, MOE_E_CUDA, MOE_E_TIMEOUT, MOE_E_DEVICE, MOE_E_NOMEM, MOE_E_STATE = range(7)
MOE_MODE_PERSISTENT, MOE_MODE_MULTIKERNEL, MOE_MODE_STATIC = 0, 1, 2

OPTIONS = {
    "mode": 1, "timeout_ns": 2, "mover_ctas": 3, "grid_ctas": 4, "split_k": 5,
    "tokens_per_tile": 6, "fault_drop_task": 7, "route_tokens": 8, "claim_ahead": 9,
    "trace": 10, "release": 11, "prefetch": 12, "bands": 13, "route_splits": 14, "l2_prefetch": 15,
    "pair": 16, "front_split": 17, "fault_drop_type": 18, "fault_corrupt_count": 19,
    "fault_repush": 20, "debug_claims": 21, "fold_gather": 22,
}
STATS = {"mover_ctas": 1, "tasks": 2, "grid": 3, "gemm_tasks": 4, "mover_tasks": 5, "stolen": 6,
         "ahead": 7, "trace_records": 8, "tile_tokens": 9, "split_k": 10, "bands": 11, "y_bytes": 12,
         "combine_tokens": 13, "pair": 14}
SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_SCORES = {"max": 0, "top2": 1}
TASK_TYPES = {1: "route", 2: "gather", 3: "gateup", 4: "down", 5: "combine", 6: "plan"}

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong

_SIGNATURES = {
    "moe_layer_create": ([_i32, _i32, _i32, _i32, _i32], _vp),
    "moe_layer_reserve": ([_vp, _i32, _vp], _i32),
    "moe_layer_set_router_bias": ([_vp, _vp], _i32),
    "moe_layer_forward": ([_vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "moe_layer_forward_host": ([_vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "moe_layer_forward_noalloc": ([_vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "moe_layer_forward_residual_norm": ([_vp, _i32] + [_vp] * 7 + [ctypes.c_float, _vp, _vp, _vp],
                                        _i32),
    "moe_layer_forward_routed": ([_vp, _i32] + [_vp] * 8, _i32),
    "moe_layer_calibrate": ([_vp, _i32] + [_vp] * 6 + [_i32, _vp, _vp], _i32),
    "moe_layer_get_routing": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    "moe_layer_status": ([_vp, _vp], _i32),
    "moe_layer_set_option": ([_vp, _i32, _i64], _i32),
    "moe_layer_get_stat": ([_vp, _i32], _i64),
    "moe_layer_workspace_bytes": ([_vp, _i32], _i64),
    "moe_layer_get_trace": ([_vp, _vp, _i32, _vp], _i32),
    "moe_layer_destroy": ([_vp], None),
    "moe_router_create": ([_i32] * 7 + [ctypes.c_float], _vp),
    "moe_router_forward": ([_vp, _i32, _vp, _i32, _i64, _vp, _vp, _vp, _vp, _vp], _i32),
    "moe_router_backward": ([_vp, _i32, _vp, _i32, _i64, _vp, _vp, _vp, _i64, _vp], _i32),
    "moe_router_destroy": ([_vp], None),
    "moe_w4_quantize": ([_i64, _i32, _i32] + [_vp] * 5, _i32),
    "moe_w4_dequantize": ([_i64, _i32, _i32] + [_vp] * 5, _i32),
    "moe_w4_create": ([_i32] * 6, _vp),
    "moe_w4_reserve": ([_vp, _i32, _vp], _i32),
    "moe_w4_workspace_bytes": ([_vp, _i32], _i64),
    "moe_w4_set_weights": ([_vp] * 5, _i32),
    "moe_w4_forward": ([_vp, _i32, _vp, _vp, _vp, _vp, _vp], _i32),
    "moe_w4_status": ([_vp, _vp], _i32),
    "moe_w4_destroy": ([_vp], None),
    "moe_last_error": ([], ctypes.c_char_p),
}


class MoEError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"moe error {code}: {msg}")
        self.code = code


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmoe.so (raises OSError if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError(f"{path} is missing: build it with persistent_megakernel_sm_gb300.build")
    dll = ctypes.CDLL(path)
    for name, (args, res) in _SIGNATURES.items():
        fn = getattr(dll, name)
        fn.argtypes = args
        fn.restype = res
    _lib = dll
    return dll


class _LazyLib:
    def __getattr__(self, name):
        return getattr(load_library(), name)


lib = _LazyLib()


def header_symbols(header: str = HEADER) -> list[str]:
    """Names of the functions include/moe.h declares."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))


def _err(code: int):
    if code != MOE_OK:
        raise MoEError(code, (lib.moe_last_error() or b"").decode())


def _stream_ptr(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(getattr(stream, "cuda_stream", stream))


def _check_tensor(name, t, dtype, shape, rows_at_least=False):
    """Refuse a tensor the kernels would read or write out of its bounds: wrong
    dtype or shape, not contiguous, or not on a CUDA device.  ``shape`` is the
    exact shape, except that with ``rows_at_least`` the first dimension may be
    larger (an output buffer with room for more rows)."""
    if t.dtype != dtype:
        raise MoEError(MOE_E_INVAL, f"{name}: dtype {t.dtype}, expected {dtype}")
    got = tuple(t.shape)
    ok = (len(got) == len(shape) and got[1:] == tuple(shape[1:]) and
          (got[0] >= shape[0] if rows_at_least else got[0] == shape[0]))
    if not ok:
        want = ("[>=%d, %s]" % (shape[0], ", ".join(map(str, shape[1:])))
                if rows_at_least else str(list(shape)))
        raise MoEError(MOE_E_INVAL, f"{name}: shape {list(got)}, expected {want}")
    if not t.is_contiguous():
        raise MoEError(MOE_E_INVAL, f"{name}: not contiguous")
    if not t.is_cuda:
        raise MoEError(MOE_E_INVAL, f"{name}: not a CUDA tensor")


class MoELayer:
    """One MoE layer handle (d, f, E, k, shared experts).

    The tensor-taking methods check each tensor's dtype (bf16; the bias fp32),
    shape, contiguity and device before the C call, so that a mismatched
    tensor raises ``MoEError`` instead of being read out of bounds."""

    def __init__(self, d: int, f: int, E: int, k: int, shared_experts: int = 0):
        h = lib.moe_layer_create(d, f, E, k, shared_experts)
        if not h:
            raise MoEError(MOE_E_INVAL, (lib.moe_last_error() or b"").decode())
        self.h = ctypes.c_void_p(h)
        self.d, self.f, self.E, self.k, self.S = d, f, E, k, shared_experts
        self._bias = None

    def reserve(self, T_max: int, stream=None):
        _err(lib.moe_layer_reserve(self.h, T_max, _stream_ptr(stream)))

    def _check_weights(self, router_w, w_gate, w_up, w_down):
        import torch
        bf, n = torch.bfloat16, self.E + self.S
        _check_tensor("router_w", router_w, bf, (self.E, self.d))
        _check_tensor("w_gate", w_gate, bf, (n, self.f, self.d))
        _check_tensor("w_up", w_up, bf, (n, self.f, self.d))
        _check_tensor("w_down", w_down, bf, (n, self.d, self.f))

    def _check_rows(self, T, **rows):
        import torch
        for name, t in rows.items():
            _check_tensor(name, t, torch.bfloat16, (T, self.d), rows_at_least=name != "x")

    def set_router_bias(self, bias):
        if bias is not None:
            import torch
            _check_tensor("bias", bias, torch.float32, (self.E,))
        self._bias = bias  # keep the tensor alive while the library holds its pointer
        _err(lib.moe_layer_set_router_bias(self.h, None if bias is None else bias.data_ptr()))

    def set_option(self, key, value: int):
        _err(lib.moe_layer_set_option(self.h, OPTIONS.get(key, key), int(value)))

    def forward(self, x, router_w, w_gate, w_up, w_down, out, stream=None):
        T = x.shape[0]
        self._check_weights(router_w, w_gate, w_up, w_down)
        self._check_rows(T, x=x, out=out)
        _err(lib.moe_layer_forward(self.h, T, x.data_ptr(), router_w.data_ptr(),
                                   w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
                                   out.data_ptr(), _stream_ptr(stream)))
        return out

    def forward_routed(self, x, idx, w, w_gate, w_up, w_down, out, stream=None):
        """moe_layer_forward_routed: the forward pass on a given routing, idx [T, k]
        int32 and w [T, k] fp32 (MoERouter.forward's, without slots of -1: a token's
        k experts are in [0, E) and distinct, or the pass ends in MOE_E_DEVICE)."""
        import torch
        T, n = x.shape[0], self.E + self.S
        _check_tensor("w_gate", w_gate, torch.bfloat16, (n, self.f, self.d))
        _check_tensor("w_up", w_up, torch.bfloat16, (n, self.f, self.d))
        _check_tensor("w_down", w_down, torch.bfloat16, (n, self.d, self.f))
        self._check_rows(T, x=x, out=out)
        _check_tensor("idx", idx, torch.int32, (T, self.k))
        _check_tensor("w", w, torch.float32, (T, self.k))
        _err(lib.moe_layer_forward_routed(self.h, T, x.data_ptr(), idx.data_ptr(), w.data_ptr(),
                                          w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
                                          out.data_ptr(), _stream_ptr(stream)))
        return out

    def forward_residual_norm(self, x, router_w, w_gate, w_up, w_down, residual, gamma, eps,
                              out, norm_out, stream=None):
        """moe_layer_forward_residual_norm: out = residual + layer(x), norm_out =
        RMSNorm(out) * gamma, fused into the combine."""
        import torch
        T = x.shape[0]
        self._check_weights(router_w, w_gate, w_up, w_down)
        self._check_rows(T, x=x, out=out, residual=residual, norm_out=norm_out)
        _check_tensor("gamma", gamma, torch.bfloat16, (self.d,))
        _err(lib.moe_layer_forward_residual_norm(
            self.h, T, x.data_ptr(), router_w.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(),
            w_down.data_ptr(), residual.data_ptr(), gamma.data_ptr(), float(eps), out.data_ptr(),
            norm_out.data_ptr(), _stream_ptr(stream)))
        return out, norm_out

    def calibrate(self, x, router_w, w_gate, w_up, w_down, out, reps: int = 3, stream=None):
        """moe_layer_calibrate: time candidate tile sizes, K splits and d bands
        on these inputs and keep the fastest as options; returns the best mean
        time in microseconds."""
        T = x.shape[0]
        self._check_weights(router_w, w_gate, w_up, w_down)
        self._check_rows(T, x=x, out=out)
        best = ctypes.c_float(0.0)
        _err(lib.moe_layer_calibrate(self.h, T, x.data_ptr(), router_w.data_ptr(),
                                     w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
                                     out.data_ptr(), int(reps), ctypes.byref(best),
                                     _stream_ptr(stream)))
        return best.value

    def forward_noalloc(self, x, router_w, w_gate, w_up, w_down, out, stream=None):
        """moe_layer_forward_noalloc: the same pass on the library's fixed scratch,
        allocating nothing (for callers that cannot allocate device memory)."""
        T = x.shape[0]
        self._check_weights(router_w, w_gate, w_up, w_down)
        self._check_rows(T, x=x, out=out)
        _err(lib.moe_layer_forward_noalloc(self.h, T, x.data_ptr(), router_w.data_ptr(),
                                          w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
                                          out.data_ptr(), _stream_ptr(stream)))
        return out

    def forward_host(self, T, x_host_ptr, router_w, w_gate, w_up, w_down, out_host_ptr,
                     stream=None):
        """moe_layer_forward_host: x and out are host addresses of T x d bf16
        values each (pinned memory for asynchronous copies)."""
        self._check_weights(router_w, w_gate, w_up, w_down)
        _err(lib.moe_layer_forward_host(self.h, T, x_host_ptr, router_w.data_ptr(),
                                        w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
                                        out_host_ptr, _stream_ptr(stream)))

    def status(self, stream=None) -> int:
        return lib.moe_layer_status(self.h, _stream_ptr(stream))

    def check(self, stream=None):
        _err(self.status(stream))

    def get_routing(self, idx=None, w=None, counts=None, offsets=None, perm=None, pos=None,
                    stream=None):
        ptr = (lambda t: None if t is None else t.data_ptr())
        _err(lib.moe_layer_get_routing(self.h, ptr(idx), ptr(w), ptr(counts), ptr(offsets),
                                       ptr(perm), ptr(pos), _stream_ptr(stream)))

    def stat(self, key) -> int:
        return lib.moe_layer_get_stat(self.h, STATS.get(key, key))

    def trace(self, cap: int = 1 << 16, stream=None):
        """Task records of the last forward as a numpy array of dicts-of-arrays:
        cta, task id, type, t_claim, t_start, t_end (ns, %globaltimer)."""
        import numpy as np
        buf = np.zeros((cap, 4), dtype=np.uint64)
        n = lib.moe_layer_get_trace(self.h, buf.ctypes.data, cap, _stream_ptr(stream))
        if n < 0:
            raise MoEError(MOE_E_CUDA, (lib.moe_last_error() or b"").decode())
        buf = buf[:n]
        task = (buf[:, 0] & 0xffffffff).astype(np.int64)
        return {"cta": (buf[:, 0] >> 32).astype(np.int64), "task": task,
                "type": task >> 28, "t_claim": buf[:, 1].astype(np.int64),
                "t_start": buf[:, 2].astype(np.int64), "t_end": buf[:, 3].astype(np.int64)}

    def workspace_bytes(self, T_max: int) -> int:
        return lib.moe_layer_workspace_bytes(self.h, T_max)

    def close(self):
        if self.h:
            lib.moe_layer_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _on_device(name, t, device, dtype, shape):
    """_check_tensor for the operators: the exact shape, on ``device`` (the
    current CUDA device's index, on which the call's stream is).  A call of a few
    microseconds makes several of these checks, so what is right costs four
    comparisons; a host tensor's device is -1."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == device:
        return
    _check_tensor(name, t, dtype, shape)
    raise MoEError(MOE_E_INVAL, f"{name}: on device {t.get_device()}, the current one is {device}")


class _Torch:
    """What the operators' calls need of torch, looked up once."""

    def __init__(self):
        import torch
        self.f32, self.bf16, self.i32, self.u8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
        self.current_device = torch.cuda.current_device
        # the current stream's handle without a Stream object around it
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)


_torch_names = None


def _torch():
    global _torch_names
    if _torch_names is None:
        _torch_names = _Torch()
    return _torch_names


def _current_device():
    return _torch().current_device()


def _stream_on(stream, device):
    """The handle of ``stream``, or of the current stream of ``device``."""
    return _torch().raw_stream(device) if stream is None else getattr(stream, "cuda_stream", stream)


class MoERouter:
    """Routing of tokens to experts from their logits (moe_router_* of
    include/moe.h): ``score`` "softmax" or "sigmoid", an optional balance bias
    that selects only, ``groups`` of consecutive experts of which the best
    ``groups_kept`` (by "max" or "top2") stay in the choice, top-k, weights
    renormalised or not and scaled.  The handle holds settings alone."""

    def __init__(self, E: int, k: int, score: str = "softmax", groups: int = 1, groups_kept: int = 1,
                 group_score: str = "top2", renormalise: bool = True, scale: float = 1.0):
        self.h = None
        if score not in SCORES or group_score not in GROUP_SCORES:
            raise MoEError(MOE_E_INVAL, f"score is one of {list(SCORES)}, group_score of {list(GROUP_SCORES)}")
        h = lib.moe_router_create(E, k, SCORES[score], groups, groups_kept, GROUP_SCORES[group_score],
                                  int(bool(renormalise)), scale)
        if not h:
            raise MoEError(MOE_E_INVAL, (lib.moe_last_error() or b"").decode())
        self.h = ctypes.c_void_p(h)
        self.E, self.k = E, k
        self._c_forward, self._c_backward = lib.moe_router_forward, lib.moe_router_backward

    def _check_logits(self, name, t, device):
        """Rows of E values, fp32 or bf16, that may be columns of a wider
        buffer; returns the type code and the row stride."""
        tt = _torch()
        if t.dtype is tt.f32:
            kind = 0
        elif t.dtype is tt.bf16:
            kind = 1
        else:
            raise MoEError(MOE_E_INVAL, f"{name}: dtype {t.dtype}, expected torch.float32 or torch.bfloat16")
        if t.dim() != 2 or t.shape[1] != self.E:
            raise MoEError(MOE_E_INVAL, f"{name}: shape {list(t.shape)}, expected [T, {self.E}]")
        rows, step = t.stride()
        if t.shape[0] <= 1:  # a single row's stride is anything
            rows = max(rows, self.E)
        if t.shape[0] and ((step != 1 and self.E > 1) or rows < self.E):
            raise MoEError(MOE_E_INVAL, f"{name}: strides {[rows, step]}, rows of consecutive values are needed")
        if not t.is_cuda:
            raise MoEError(MOE_E_INVAL, f"{name}: not a CUDA tensor")
        if t.get_device() != device:
            raise MoEError(MOE_E_INVAL, f"{name}: on device {t.get_device()}, the current one is {device}")
        return kind, rows

    def forward(self, logits, idx, w, bias=None, counts=None, stream=None):
        """logits [T, E] -> idx [T, k] int32, w [T, k] fp32 and, if given, counts
        [E] int32 (each expert's tokens).  ``bias`` [E] fp32 selects only."""
        tt, dev = _torch(), _current_device()
        kind, row = self._check_logits("logits", logits, dev)
        T = logits.shape[0]
        _on_device("idx", idx, dev, tt.i32, (T, self.k))
        _on_device("w", w, dev, tt.f32, (T, self.k))
        if bias is not None:
            _on_device("bias", bias, dev, tt.f32, (self.E,))
        if counts is not None:
            _on_device("counts", counts, dev, tt.i32, (self.E,))
        _err(self._c_forward(self.h, T, logits.data_ptr(), kind, row,
                             None if bias is None else bias.data_ptr(), idx.data_ptr(),
                             w.data_ptr(), None if counts is None else counts.data_ptr(),
                             _stream_on(stream, dev)))
        return idx, w

    def backward(self, logits, idx, grad_w, grad_logits, stream=None):
        """grad_w [T, k] fp32 -> grad_logits [T, E], of the logits' dtype."""
        tt, dev = _torch(), _current_device()
        kind, row = self._check_logits("logits", logits, dev)
        out_kind, out_row = self._check_logits("grad_logits", grad_logits, dev)
        T = logits.shape[0]
        if out_kind != kind or grad_logits.shape[0] != T:
            raise MoEError(MOE_E_INVAL, "grad_logits: dtype and rows must be those of logits")
        _on_device("idx", idx, dev, tt.i32, (T, self.k))
        _on_device("grad_w", grad_w, dev, tt.f32, (T, self.k))
        _err(self._c_backward(self.h, T, logits.data_ptr(), kind, row, idx.data_ptr(),
                              grad_w.data_ptr(), grad_logits.data_ptr(), out_row,
                              _stream_on(stream, dev)))
        return grad_logits

    def close(self):
        if self.h:
            lib.moe_router_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _check_w4(w, codes, scales, zeros):
    """Shapes of a bf16 matrix (any leading dimensions) and its 4-bit form;
    returns rows, columns, the group and the device."""
    tt, dev = _torch(), _current_device()
    shape = tuple(w.shape)
    if len(shape) < 2 or scales.dim() != len(shape) or shape[-1] % 2 != 0:
        raise MoEError(MOE_E_INVAL, f"weights {list(shape)} and scales {list(scales.shape)}: expected "
                                    "[..., rows, cols] and [..., rows, cols / group]")
    cols, n = shape[-1], scales.shape[-1]
    group = cols // n if n else 0
    if group not in (32, 64, 128) or group * n != cols:
        raise MoEError(MOE_E_INVAL, f"{cols} columns and {n} scales a row: groups of 32, 64 or 128 are needed")
    _on_device("weights", w, dev, tt.bf16, shape)
    _on_device("codes", codes, dev, tt.u8, shape[:-1] + (cols // 2,))
    _on_device("scales", scales, dev, tt.bf16, shape[:-1] + (n,))
    if zeros is not None:
        _on_device("zeros", zeros, dev, tt.u8, shape[:-1] + (n,))
    return w.numel() // cols, cols, group, dev


def w4_quantize(w, codes, scales, zeros=None, stream=None):
    """moe_w4_quantize: bf16 w [..., rows, cols] -> codes uint8 [..., rows,
    cols / 2], scales bf16 [..., rows, cols / group] and, if given, zeros uint8
    of the scales' shape.  The shape of ``scales`` sets the group (32, 64, 128)."""
    rows, cols, group, dev = _check_w4(w, codes, scales, zeros)
    _err(lib.moe_w4_quantize(rows, cols, group, w.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                             None if zeros is None else zeros.data_ptr(), _stream_on(stream, dev)))
    return codes, scales, zeros


def w4_dequantize(codes, scales, zeros, w, stream=None):
    """moe_w4_dequantize: the 4-bit weights' values as bf16 into w."""
    rows, cols, group, dev = _check_w4(w, codes, scales, zeros)
    _err(lib.moe_w4_dequantize(rows, cols, group, codes.data_ptr(), scales.data_ptr(),
                               None if zeros is None else zeros.data_ptr(), w.data_ptr(),
                               _stream_on(stream, dev)))
    return w


class _W4Weight(ctypes.Structure):
    _fields_ = [("codes", _vp), ("scales", _vp), ("zeros", _vp)]


class W4Experts:
    """The experts' SwiGLU product on 4-bit weights for decode batches, given
    the routing (moe_w4_* of include/moe.h)."""

    def __init__(self, d: int, f: int, E: int, k: int, shared_experts: int = 0, group: int = 128):
        self.h = None
        h = lib.moe_w4_create(d, f, E, k, shared_experts, group)
        if not h:
            raise MoEError(MOE_E_INVAL, (lib.moe_last_error() or b"").decode())
        self.h = ctypes.c_void_p(h)
        self.d, self.f, self.E, self.k, self.S, self.group = d, f, E, k, shared_experts, group
        self._weights = self._device = None
        self._c_forward = lib.moe_w4_forward

    def reserve(self, T_max: int, stream=None):
        _err(lib.moe_w4_reserve(self.h, T_max, _stream_ptr(stream)))
        self._device = _current_device()

    def workspace_bytes(self, T_max: int) -> int:
        return lib.moe_w4_workspace_bytes(self.h, T_max)

    def set_weights(self, gate, up, down, stream=None):
        """After reserve.  Each of gate, up, down: (codes, scales, zeros or None), codes uint8
        [E + S, rows, cols / 2], scales bf16 and zeros uint8 [E + S, rows, cols /
        group]; rows, cols are f, d for gate and up and d, f for down.
        The codes are read where they are, the scales and zeros copied now."""
        tt, dev = _torch(), _current_device()
        self._check_device(dev)
        n, args = self.E + self.S, []
        for name, m, rows, cols in (("gate", gate, self.f, self.d), ("up", up, self.f, self.d),
                                    ("down", down, self.d, self.f)):
            codes, scales, zeros = m
            _on_device(name + " codes", codes, dev, tt.u8, (n, rows, cols // 2))
            _on_device(name + " scales", scales, dev, tt.bf16, (n, rows, cols // self.group))
            if zeros is not None:
                _on_device(name + " zeros", zeros, dev, tt.u8, (n, rows, cols // self.group))
            args.append(_W4Weight(codes.data_ptr(), scales.data_ptr(),
                                  None if zeros is None else zeros.data_ptr()))
        _err(lib.moe_w4_set_weights(self.h, *(ctypes.byref(a) for a in args), _stream_on(stream, dev)))
        self._weights = (tuple(gate), tuple(up), tuple(down))  # alive while the library holds their pointers

    def _check_device(self, dev):
        if dev != self._device and self._device is not None:
            raise MoEError(MOE_E_INVAL, f"the workspace is on device {self._device}, the current one is {dev}")

    def forward(self, x, idx, w, out, stream=None):
        """x [T, d] bf16, idx [T, k] int32 and w [T, k] fp32 (MoERouter.forward's)
        -> out [T, d] bf16; slots with idx outside [0, E) add nothing."""
        tt, dev = _torch(), _current_device()
        self._check_device(dev)
        T = x.shape[0]
        _on_device("x", x, dev, tt.bf16, (T, self.d))
        _on_device("idx", idx, dev, tt.i32, (T, self.k))
        _on_device("w", w, dev, tt.f32, (T, self.k))
        _on_device("out", out, dev, tt.bf16, (T, self.d))
        _err(self._c_forward(self.h, T, x.data_ptr(), idx.data_ptr(), w.data_ptr(), out.data_ptr(),
                             _stream_on(stream, dev)))
        return out

    def status(self, stream=None) -> int:
        return lib.moe_w4_status(self.h, _stream_ptr(stream))

    def check(self, stream=None):
        """Synchronise and raise if a wait inside the kernels ran out."""
        _err(self.status(stream))

    def close(self):
        if self.h:
            lib.moe_w4_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
