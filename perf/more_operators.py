"""The norms about a block, 8-bit rows and the layer for a few tokens, as cases to be measured.

Each case names one call of a user's program; `run` makes it, either in its
plain form (elementary torch operations in 32 bits) or, with `own` set, through
this package's entry points.  `exact` gives the same outputs in 64 bits."""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode step, between the layer and the next block: residual add, then the next block's norm
        dict(name="norm_one_token", op="norm", T=1, d=2048, pre="rms", post="none", gate="none", res="bfloat16",
             par="bfloat16", offset=False, scale=1.0, save=0, pad=0),
        # a decode batch of 256 sequences, norms on both sides of the block, a gate for each token
        dict(name="norm_decode_256", op="norm", T=256, d=4096, pre="rms", post="rms", gate="token", res="bfloat16",
             par="bfloat16", offset=True, scale=1.0, save=0, pad=0),
        # the prefill batch of a training step: a gate for each channel, what the backward pass needs kept in 8 bits
        # (and, to be looked at, read back)
        dict(name="norm_train_8k", op="norm", T=8192, d=7168, pre="rms", post="rms", gate="channel", res="bfloat16",
             par="float32", offset=False, scale=0.5, save=128, pad=0),
        # an odd width in wider buffers, layer norms, a gate for each value, the residual stream in 32 bits
        dict(name="norm_odd_layer", op="norm", T=4099, d=2047, pre="layer", post="layer", gate="element", res="float32",
             par="float32", offset=False, scale=1.0, save=0, pad=5),
        # the backward pass of a small batch, sums and outputs kept in bf16
        dict(name="norm_grad_512", op="norm_grad", T=512, d=4096, pre="rms", post="none", gate="none", res="bfloat16",
             par="bfloat16", offset=False, scale=1.0, save=0, pad=0),
        # the backward pass at the prefill batch, from what was kept in 8 bits
        dict(name="norm_grad_train_8k", op="norm_grad", T=8192, d=7168, pre="rms", post="rms", gate="channel",
             res="bfloat16", par="float32", offset=False, scale=0.5, save=128, pad=0),
        # the backward pass of the odd width
        dict(name="norm_grad_odd_layer", op="norm_grad", T=4099, d=2047, pre="layer", post="layer", gate="element",
             res="float32", par="float32", offset=False, scale=1.0, save=0, pad=5),
        # an odd activation to 8 bits and back
        dict(name="rows8_odd", op="rows8", T=1021, d=1411, group=32, type="float32"),
        # the experts' activations of the skewed batch (4096 tokens in 6 experts each) kept in 8 bits and fetched back
        dict(name="rows8_experts", op="rows8", T=24576, d=1408, group=128, type="bfloat16"),
        # decode of one token: the whole fine-grained layer, its own router with a bias
        dict(name="decode_fine_1", op="decode", T=1, d=2048, E=128, k=8, f=768, S=0, bias=True, routed=False, padded=0),
        # speculative decode of 4 tokens: the whole eight-expert layer
        dict(name="decode_eight_4", op="decode", T=4, d=4096, E=8, k=2, f=14336, S=0, bias=False, routed=False, padded=0),
        # a padded batch of 13 rows, 3 of them padding, routed before the call, with a shared expert
        dict(name="decode_padded_13", op="decode", T=13, d=7168, E=32, k=8, f=2048, S=1, bias=False, routed=True, padded=3),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "norm", "norm_grad", "rows8", "decode", "decode"])
    if op in ("norm", "norm_grad"):
        T = _log_int(rng, 1, 32768)
        d = _log_int(rng, 16, min(16384, (1 << 26) // T))
        if rng.random() < 0.6:  # most widths are multiples of 64
            d = max(64, d // 64 * 64)
        pre, post = rng.choice(["rms", "rms", "layer"]), rng.choice(["none", "rms", "layer"])
        return dict(op=op, T=T, d=d, pre=pre, post=post, gate=rng.choice(["none", "channel", "token", "element"]),
                    res=rng.choice(["bfloat16", "float32"]), par=rng.choice(["bfloat16", "float32"]),
                    offset=rng.random() < 0.3, scale=rng.choice([1.0, 0.5, 0.22]), save=rng.choice([0, 0, 32, 64, 128]),
                    pad=rng.choice([0, 0, 8, 3]))
    if op == "rows8":
        T = _log_int(rng, 1, 65536)
        return dict(op=op, T=T, d=_log_int(rng, 1, min(32768, (1 << 26) // T)), group=rng.choice([32, 64, 128]),
                    type=rng.choice(["bfloat16", "float32"]))
    while True:
        d, f = 128 * _log_int(rng, 2, 56), 128 * _log_int(rng, 2, 112)
        E, S = _log_int(rng, 4, 256), rng.choice([0, 0, 1])
        if 3 * (E + S) * d * f <= 1 << 30:
            break
    T, routed = _log_int(rng, 1, 16), rng.random() < 0.4
    return dict(op=op, T=T, d=d, E=E, k=rng.randint(1, min(8, E)), f=f, S=S, bias=not routed and rng.random() < 0.5,
                routed=routed, padded=rng.choice([0, T // 4]) if routed else 0)


def work(case):
    c = case
    T, d = c["T"], c["d"]
    if c["op"] == "decode":
        rows = T - c["padded"]
        active = c["E"] * (1 - (1 - c["k"] / c["E"]) ** rows) + c["S"]  # experts that at least one row is expected to choose
        return {"bytes": active * 6 * d * c["f"] + (0 if c["routed"] else 2 * c["E"] * d) + T * (4 * d + 8 * c["k"]),
                "flops": 6 * d * c["f"] * rows * (c["k"] + c["S"]) + (0 if c["routed"] else 2 * T * c["E"] * d)}
    if c["op"] == "rows8":
        size = 2 if c["type"] == "bfloat16" else 4
        return {"bytes": T * d * (2 * size + 2 + 4 / c["group"]), "flops": 6 * T * d}
    res = 2 if c["res"] == "bfloat16" else 4
    gate = T * d * 2 if c["gate"] == "element" else T * 4 if c["gate"] == "token" else 0
    kept = 2 if c["save"] == 0 else 1 + 2 / c["save"]
    norms = (1 if c["pre"] != "none" else 0) + (1 if c["post"] != "none" else 0)
    if c["op"] == "norm":
        read_back = 2 * (2 * (1 + 2 / c["save"]) + 2) if c["save"] else 0  # both kept ones written, read and written as bf16
        return {"bytes": T * d * (2 * res + 2 + 2 + read_back) + gate + T * 16, "flops": T * d * (4 + 4 * norms)}
    kept_out = res if c["save"] == 0 else kept
    kept_y = kept if c["post"] != "none" or c["gate"] != "none" else 0
    return {"bytes": T * d * (2 * res + 2 + 2 + kept_out + kept_y) + 2 * gate + T * 16, "flops": T * d * (6 + 10 * norms)}


# ----------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, g, dtype=F32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _rows(v, pad):
    """v as columns of a wider buffer."""
    if not pad:
        return v
    wide = torch.zeros(v.shape[0], v.shape[1] + pad, dtype=v.dtype, device="cuda")
    wide[:, : v.shape[1]] = v
    return wide[:, : v.shape[1]]


def _empty(c, dtype):
    return torch.empty(c["T"], c["d"] + c["pad"], dtype=dtype, device="cuda")[:, : c["d"]]


def _codes(c, rows, group):
    return (torch.empty(rows, c["d"], dtype=torch.int8, device="cuda"),
            torch.empty(rows, -(-c["d"] // group), dtype=BF16, device="cuda"))


def _prepare_norm(c, seed):
    g, T, d = _gen(seed), c["T"], c["d"]
    res, par = getattr(torch, c["res"]), getattr(torch, c["par"])
    level = 0.4 + 0.6 * _normal(d, g)  # a residual stream's channels have levels of their own, a few of them large
    level[torch.rand(d, generator=g, device="cuda") < 0.003] *= 20
    s = dict(case=c, residual=_rows((_normal((T, d), g) + level).to(res), c["pad"]),
             y=_rows((0.7 * _normal((T, d), g) + 0.2).to(BF16), c["pad"]))

    def gain():
        return (0.2 * _normal(d, g) + (0.0 if c["offset"] else 1.0)).to(par)

    s["params"] = dict(pre_gain=gain(), post_gain=gain() if c["post"] != "none" else None,
                       pre_shift=(0.1 * _normal(d, g)).to(par) if c["pre"] == "layer" else None,
                       post_shift=(0.1 * _normal(d, g)).to(par) if c["post"] == "layer" else None)
    s["gate"] = (None if c["gate"] == "none" else (0.5 + 0.3 * _normal(d, g)).to(par) if c["gate"] == "channel"
                 else torch.sigmoid(_normal(T, g)) if c["gate"] == "token"
                 else _rows((0.5 + 0.3 * _normal((T, d), g)).to(BF16), c["pad"]))
    if c["op"] == "norm":
        s.update(out=_empty(c, res), norm=_empty(c, BF16), stats=torch.empty(T, 4, device="cuda"))
        if c["save"]:
            s.update(out8=_codes(c, T, c["save"]), y8=_codes(c, T, c["save"]), out_back=torch.empty(T, d, dtype=BF16, device="cuda"),
                     y_back=torch.empty(T, d, dtype=BF16, device="cuda"))
    else:
        kept = _plain_norm(c, s)
        s.update(stats=kept["stats"], kept_out=_rows(kept["out"], c["pad"]), kept_y=s["y"],
                 grad_norm=_rows((0.01 * _normal((T, d), g)).to(BF16), c["pad"]),
                 grad_out=_rows((0.01 * _normal((T, d), g)).to(res), c["pad"]),
                 grad_residual=_empty(c, res), grad_y=_empty(c, BF16))
        if c["save"]:
            s["kept_out"], s["kept_y"] = _plain_rows8(kept["out"], c["save"]), _plain_rows8(s["y"], c["save"])
        s["grads"] = {n: torch.empty(d, device="cuda") for n, p in s["params"].items() if p is not None}
        s["grad_gate"] = (None if c["gate"] == "none" else torch.empty(d, device="cuda") if c["gate"] == "channel"
                          else torch.empty(T, device="cuda") if c["gate"] == "token" else _empty(c, BF16))
        if c["post"] == "none" and c["gate"] == "none":
            s["kept_y"] = None
        del s["residual"], s["y"]
    if own:
        from persistent_megakernel_sm_gb300 import MoEBlockNorm
        s["block"] = MoEBlockNorm(d, pre=c["pre"], post=c["post"], gate=c["gate"], scale=c["scale"], eps=1e-6,
                                  unit_offset=c["offset"], group=c["save"] or 128)
        if c["op"] == "norm_grad":
            s["block"].reserve()
    return s


def _prepare_decode(c, seed):
    g = _gen(seed)
    T, d, f, E, k, S = (c[n] for n in ("T", "d", "f", "E", "k", "S"))
    weights = [_normal(shape, g, BF16).mul_(shape[-1] ** -0.5) for shape in ((E + S, f, d), (E + S, f, d), (E + S, d, f))]
    s = dict(case=c, x=_normal((T, d), g, BF16), weights=weights, out=torch.empty(T, d, dtype=BF16, device="cuda"))
    if c["routed"]:
        idx = torch.rand(T, E, generator=g, device="cuda").argsort(-1, descending=True)[:, :k].to(torch.int32)
        w = torch.softmax(_normal((T, k), g), -1)
        if c["padded"]:  # the rows behind the batch's sequences choose nothing
            idx[T - c["padded"]:] = -1
            w[T - c["padded"]:] = 0
        s.update(idx=idx.contiguous(), w=w.contiguous())
    else:
        s["router_w"] = _normal((E, d), g, BF16).mul_(d ** -0.5)
        s["bias"] = 0.3 * _normal(E, g) if c["bias"] else None
        for _ in range(50):  # rows whose choice hangs on the last bits of a sum are drawn again
            top = s["x"].double() @ s["router_w"].double().t() + (s["bias"].double() if c["bias"] else 0)
            top = top.sort(-1, descending=True).values[:, : k + 1]
            rows = ((top[:, :-1] - top[:, 1:]) < 1e-3).any(1).nonzero()[:, 0]
            if not len(rows):
                break
            s["x"][rows] = _normal((len(rows), d), g, BF16)
        s.update(idx=torch.empty(T, k, dtype=torch.int32, device="cuda"), w=torch.empty(T, k, device="cuda"))
    if own:
        from persistent_megakernel_sm_gb300 import MoEDecode
        s["layer"] = MoEDecode(d, f, E, k, shared_experts=S)
        s["layer"].reserve(T)
    return s


def prepare(case, seed):
    c = case
    if c["op"] in ("norm", "norm_grad"):
        return _prepare_norm(c, seed)
    if c["op"] == "decode":
        return _prepare_decode(c, seed)
    g, dtype = _gen(seed), getattr(torch, c["type"])
    # activations behind a gate: most near zero, a few large
    v = _normal((c["T"], c["d"]), g) * torch.sigmoid(2 * _normal((c["T"], c["d"]), g))
    return dict(case=c, v=v.to(dtype), held=_codes(c, c["T"], c["group"]),
                back=torch.empty(c["T"], c["d"], dtype=dtype, device="cuda"))


# ------------------------------------------------------------------ plain forms

def _plain_rows8(v, group):
    """Codes and scales of rows, a scale for each group of consecutive columns (the last one may be short)."""
    T, d = v.shape
    n = -(-d // group)
    x = torch.zeros(T, n * group, device=v.device)
    x[:, :d] = v.float()
    x = x.view(T, n, group)
    scales = (x.abs().amax(-1) / 127).to(BF16)
    step = torch.where(scales == 0, 1.0, scales.float())
    codes = torch.round(x / step.unsqueeze(-1)).clamp(-127, 127).to(torch.int8)
    return codes.view(T, n * group)[:, :d].contiguous(), scales


def _plain_values8(held, group):
    codes, scales = held
    T, d = codes.shape
    x = torch.zeros(T, scales.shape[1] * group, device=codes.device)
    x[:, :d] = codes.float()
    return (x.view(T, -1, group) * scales.float().unsqueeze(-1)).view(T, -1)[:, :d]


def _plain_stats(x, kind):
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    return mean, 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + 1e-6)


def _gains(c, s):
    one = 1.0 if c["offset"] else 0.0
    return [None if p is None else p.float() + (one if "gain" in n else 0.0) for n, p in s["params"].items()]


def _gate(c, s):
    g = s["gate"]
    return 1.0 if g is None else g.float().unsqueeze(1) if c["gate"] == "token" else g.float()


def _plain_norm(c, s):
    pre_gain, post_gain, pre_shift, post_shift = _gains(c, s)
    y = s["y"].float()
    mean_y, rstd_y = torch.zeros_like(y[:, :1]), torch.ones_like(y[:, :1])
    p = y
    if c["post"] != "none":
        mean_y, rstd_y = _plain_stats(y, c["post"])
        p = (y - mean_y) * rstd_y * post_gain + (0.0 if post_shift is None else post_shift)
    out = (s["residual"].float() + c["scale"] * (_gate(c, s) * p)).to(s["residual"].dtype)
    x = out.float()  # the norm is of what is kept
    mean, rstd = _plain_stats(x, c["pre"])
    norm = (x - mean) * rstd * pre_gain + (0.0 if pre_shift is None else pre_shift)
    return dict(out=out, norm=norm.to(BF16), stats=torch.cat((mean_y, rstd_y, mean, rstd), 1))


def _back(gn, xhat, rstd, kind):
    """The gradient through a norm: gn of its output before gain, xhat that output."""
    along = xhat * (gn * xhat).mean(1, keepdim=True)
    return rstd * (gn - (gn.mean(1, keepdim=True) + along if kind == "layer" else along))


def _plain_norm_grad(c, s):
    pre_gain, post_gain, pre_shift, post_shift = _gains(c, s)
    mean_y, rstd_y, mean, rstd = s["stats"].split(1, 1)
    x = _plain_values8(s["kept_out"], c["save"]) if c["save"] else s["kept_out"].float()
    gn = s["grad_norm"].float()
    xhat = (x - mean) * rstd
    grads = dict(pre_gain=(gn * xhat).sum(0))
    if pre_shift is not None:
        grads["pre_shift"] = gn.sum(0)
    gr = s["grad_out"].float() + _back(gn * pre_gain, xhat, rstd, c["pre"])
    gp = c["scale"] * gr
    grad_gate = None
    gate = _gate(c, s)
    if s["kept_y"] is not None:
        y = _plain_values8(s["kept_y"], c["save"]) if c["save"] else s["kept_y"].float()
        yhat = (y - mean_y) * rstd_y
        p = yhat if post_gain is None else yhat * post_gain + (0.0 if post_shift is None else post_shift)
        if c["gate"] != "none":
            grad_gate = gp * p
            grad_gate = (grad_gate.sum(0) if c["gate"] == "channel" else grad_gate.sum(1) if c["gate"] == "token"
                         else grad_gate.to(BF16))
    gp = gp * gate
    if post_gain is not None:
        grads["post_gain"] = (gp * yhat).sum(0)
        if post_shift is not None:
            grads["post_shift"] = gp.sum(0)
        gp = _back(gp * post_gain, yhat, rstd_y, c["post"])
    return dict(residual=gr.to(s["grad_out"].dtype), y=gp.to(BF16), gate=grad_gate, **grads)


def _plain_route(c, s):
    logits = s["x"].float() @ s["router_w"].float().t()
    if s["bias"] is not None:
        logits = logits + s["bias"]
    top, idx = logits.sort(dim=1, descending=True, stable=True)
    e = torch.exp(top[:, : c["k"]] - top[:, :1])
    return idx[:, : c["k"]].to(torch.int32), e / e.sum(1, keepdim=True)


def _plain_decode(c, s):
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    idx, w = (s["idx"], s["w"]) if c["routed"] else _plain_route(c, s)
    x = s["x"].float()
    live = idx >= 0
    at = idx.clamp_min(0).long()
    wl = torch.where(live, w, 0.0)
    if T * k <= E:  # few slots: each one's own expert's weights
        gate, up, down = (m[at.view(-1)].float() for m in s["weights"])
        rows = x.repeat_interleave(k, 0).unsqueeze(-1)
        z = gate @ rows
        y = down @ (z / (1 + torch.exp(-z)) * (up @ rows))
        out = (y.view(T, k, -1) * wl.unsqueeze(-1)).sum(1)
    else:  # many: every expert on every row, weighted (by zero where it was not chosen)
        gate, up, down = (m[:E].float() for m in s["weights"])
        z = gate @ x.t()
        h = z / (1 + torch.exp(-z)) * (up @ x.t())
        full = torch.zeros(T, E, device=x.device).scatter_add_(1, at, wl)
        out = (down @ (h * full.t().unsqueeze(1))).sum(0).t()
    if S:
        gate, up, down = (m[E].float() for m in s["weights"])
        z = x @ gate.t()
        out = out + (z / (1 + torch.exp(-z)) * (x @ up.t())) @ down.t()
    return out.to(BF16) if c["routed"] else (out.to(BF16), idx, w)


def run(state):
    s, c = state, state["case"]
    if c["op"] == "norm":
        if own:
            s["block"].forward(s["residual"], s["y"], s["out"], s["norm"], **s["params"], gate=s["gate"], stats=s["stats"],
                               out8=s.get("out8"), y8=s.get("y8"))
            got = dict(out=s["out"], norm=s["norm"], stats=s["stats"])
            if c["save"]:
                from persistent_megakernel_sm_gb300 import rows8_dequantize
                got["out8"] = rows8_dequantize(*s["out8"], s["out_back"], group=c["save"])
                got["y8"] = rows8_dequantize(*s["y8"], s["y_back"], group=c["save"])
            return got
        got = _plain_norm(c, s)
        if c["save"]:
            got["out8"] = _plain_values8(_plain_rows8(got["out"], c["save"]), c["save"]).to(BF16)
            got["y8"] = _plain_values8(_plain_rows8(s["y"], c["save"]), c["save"]).to(BF16)
        return got
    if c["op"] == "norm_grad":
        if own:
            s["block"].backward(s["grad_out"], s["grad_norm"], s["grad_residual"], s["grad_y"], stats=s["stats"],
                                out=s["kept_out"], y=s["kept_y"], **s["params"], gate=s["gate"], grad_gate=s["grad_gate"],
                                **{"grad_" + n: t for n, t in s["grads"].items()})
            return dict(residual=s["grad_residual"], y=s["grad_y"], gate=s["grad_gate"], **s["grads"])
        return _plain_norm_grad(c, s)
    if c["op"] == "rows8":
        if own:
            from persistent_megakernel_sm_gb300 import rows8_dequantize, rows8_quantize
            codes, scales = rows8_quantize(s["v"], *s["held"], group=c["group"])
            return rows8_dequantize(codes, scales, s["back"], group=c["group"]), scales
        held = _plain_rows8(s["v"], c["group"])
        return _plain_values8(held, c["group"]).to(s["v"].dtype), held[1]
    if own:
        if c["routed"]:
            return s["layer"].forward_routed(s["x"], s["idx"], s["w"], *s["weights"], s["out"])
        s["layer"].forward(s["x"], s["router_w"], *s["weights"], s["out"], bias=s["bias"], idx=s["idx"], w=s["w"])
        return s["out"], s["idx"], s["w"]
    return _plain_decode(c, s)


# ---------------------------------------------------------------- in 64 bits

def _exact_values8(held, group):
    codes, scales = held
    at = torch.arange(codes.shape[1], device=codes.device) // group
    return codes.double() * scales.double()[:, at]


def _exact_rows8(v, group):
    """What the rows are held as, by the definition: the scale itself is a bf16 number."""
    v = v.double()
    out, scales = torch.empty_like(v), []
    for lo in range(0, v.shape[1], group):
        part = v[:, lo : lo + group]
        by = (part.abs().max(1, keepdim=True).values / 127).float().to(BF16).double()
        out[:, lo : lo + group] = (part / torch.where(by > 0, by, torch.ones_like(by))).round().clamp(-127, 127) * by
        scales.append(by)
    return out, torch.cat(scales, 1)


def _exact_moments(x, kind):
    if kind == "none":
        return torch.zeros(len(x), dtype=F64, device="cuda"), torch.ones(len(x), dtype=F64, device="cuda")
    mean = x.sum(1) / x.shape[1] if kind == "layer" else torch.zeros(len(x), dtype=F64, device="cuda")
    return mean, ((x - mean[:, None]).square().sum(1) / x.shape[1] + 1e-6).rsqrt()


def _exact_gains(c, s):
    d = c["d"]
    one, none = torch.ones(d, dtype=F64, device="cuda"), torch.zeros(d, dtype=F64, device="cuda")
    p = s["params"]

    def gain(name):
        return one if p[name] is None else p[name].double() + float(c["offset"])

    def shift(name):
        return none if p[name] is None else p[name].double()

    g = s["gate"]
    gate = one if g is None else g.double()[:, None] if c["gate"] == "token" else g.double()
    return gain("pre_gain"), shift("pre_shift"), gain("post_gain"), shift("post_shift"), gate


def _exact_norm(c, s):
    a, b, ap, bp, gate = _exact_gains(c, s)
    y = s["y"].double()
    my, ry = _exact_moments(y, c["post"])
    out = s["residual"].double() + gate * c["scale"] * (ap * (y - my[:, None]) * ry[:, None] + bp)
    kept = out.to(s["residual"].dtype)  # the norm is of what is kept
    x = kept.double()
    m, r = _exact_moments(x, c["pre"])
    got = dict(out=out, norm=a * ((x - m[:, None]) * r[:, None]) + b, stats=torch.stack((my, ry, m, r), 1))
    if c["save"]:
        got["out8"], got["y8"] = _exact_rows8(kept, c["save"])[0], _exact_rows8(s["y"], c["save"])[0]
    return got


def _exact_norm_grad(c, s):
    """Each norm's Jacobian (I - 1 1' / d - u u' / d) / sigma applied to the gradient, u the normalised row (a root mean
    square has no 1 1' in it)."""
    a, _, ap, bp, gate = _exact_gains(c, s)
    d, stats = c["d"], s["stats"].double()
    held = (lambda t: _exact_values8(t, c["save"])) if c["save"] else (lambda t: t.double())
    u = (held(s["kept_out"]) - stats[:, 2:3]) * stats[:, 3:4]
    gn = s["grad_norm"].double()
    t = gn * a
    through = t - u * ((t * u).sum(1) / d)[:, None] - (t.sum(1)[:, None] / d if c["pre"] == "layer" else 0)
    gr = s["grad_out"].double() + through * stats[:, 3:4]
    got = dict(residual=gr, y=c["scale"] * gate * gr, gate=None, pre_gain=torch.einsum("td,td->d", gn, u))
    if s["params"]["pre_shift"] is not None:
        got["pre_shift"] = torch.einsum("td->d", gn)
    if s["kept_y"] is not None:
        v = (held(s["kept_y"]) - stats[:, 0:1]) * stats[:, 1:2]
        if c["gate"] != "none":
            each = c["scale"] * gr * (v * ap + bp)
            got["gate"] = each.sum(0) if c["gate"] == "channel" else each.sum(1) if c["gate"] == "token" else each
        if c["post"] != "none":
            t = got["y"]
            got["post_gain"] = torch.einsum("td,td->d", t, v)
            if s["params"]["post_shift"] is not None:
                got["post_shift"] = torch.einsum("td->d", t)
            t = t * ap
            got["y"] = stats[:, 1:2] * (t - v * ((t * v).sum(1) / d)[:, None] - (t.sum(1)[:, None] / d if c["post"] == "layer" else 0))
    return got


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "norm":
        return _exact_norm(c, s)
    if c["op"] == "norm_grad":
        return _exact_norm_grad(c, s)
    if c["op"] == "rows8":
        return _exact_rows8(s["v"], c["group"])
    T, E, S, k = c["T"], c["E"], c["S"], c["k"]
    x, out = s["x"].double(), torch.zeros(T, c["d"], dtype=F64, device="cuda")
    idx, w = s["idx"], s["w"].double()
    if not c["routed"]:
        logits = torch.einsum("td,ed->te", x, s["router_w"].double()) + (0 if s["bias"] is None else s["bias"].double())
        idx = logits.argsort(dim=1, descending=True, stable=True)[:, :k]
        w = torch.softmax(logits, 1).gather(1, idx)
        w = w / w.sum(1, keepdim=True)
    for e in range(E + S):
        rows = (idx == e).any(1).nonzero()[:, 0] if e < E else torch.arange(T, device="cuda")
        if not len(rows):
            continue
        weight = (w * (idx == e)).sum(1)[rows, None] if e < E else 1.0
        z = x[rows] @ s["weights"][0][e].double().t()
        h = z * torch.sigmoid(z) * (x[rows] @ s["weights"][1][e].double().t())
        out[rows] += weight * (h @ s["weights"][2][e].double().t())
    return out if c["routed"] else (out, idx.to(torch.int32), w)
