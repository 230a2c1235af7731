"""The routing operators and the 4-bit experts, as cases to be measured.

Each case names one call of a user's program; `run` makes it, either in its
plain form (elementary torch operations in 32 bits) or, with `own` set, through
this package's entry points.  `exact` gives the same outputs in 64 bits."""
import math

import numpy as np
import torch

own = False

BF16 = torch.bfloat16


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode step: 256 experts in 8 groups, sigmoid scores with a balance bias
        dict(name="route_one_token", op="route", T=1, E=256, k=8, score="sigmoid", bias=True, groups=8, kept=4,
             group_score="top2", renorm=True, scale=2.5, dtype="float32", pad=0, masked=False),
        # a training or prefill step of 8192 tokens over the same experts
        dict(name="route_grouped_8k", op="route", T=8192, E=256, k=8, score="sigmoid", bias=True, groups=8, kept=4,
             group_score="top2", renorm=True, scale=2.5, dtype="float32", pad=0, masked=False),
        # plain softmax routing on bf16 logits, exact ties among them; some experts are masked out of each
        # row, some rows (padding) of all of them
        dict(name="route_softmax_masked", op="route", T=32768, E=64, k=6, score="softmax", bias=False, groups=1, kept=1,
             group_score="max", renorm=False, scale=1.0, dtype="bfloat16", pad=0, masked=True),
        # the backward pass of a training step's softmax router, logits a view into a wider buffer
        dict(name="route_grad_softmax", op="route_grad", T=4099, E=60, k=6, score="softmax", bias=False, groups=1, kept=1,
             group_score="max", renorm=False, scale=1.0, dtype="bfloat16", pad=4, masked=False),
        # the backward pass of the grouped sigmoid router, at the longest batch of the layer
        dict(name="route_grad_sigmoid_32k", op="route_grad", T=32768, E=256, k=8, score="sigmoid", bias=True, groups=8,
             kept=4, group_score="top2", renorm=True, scale=2.5, dtype="float32", pad=0, masked=False),
        # converting one layer's fine-grained gate projections, with zero points, and reading them back
        dict(name="quantize_fine_zeros", op="quantize", N=16 * 768, K=2048, group=32, zeros=True),
        # converting all down projections of the eight-expert layer and reading them back (the step from bf16
        # weights to 4-bit ones and, for long prompts, back)
        dict(name="quantize_down", op="quantize", N=8 * 4096, K=14336, group=128, zeros=False),
        # decode of one token: the fine-grained layer, the smallest call
        dict(name="experts_fine_1", op="experts", T=1, d=2048, E=128, k=8, f=768, S=0, group=32, zeros=False, padded=0),
        # decode of one token: the eight-expert layer
        dict(name="experts_eight_1", op="experts", T=1, d=4096, E=8, k=2, f=14336, S=0, group=128, zeros=False, padded=0),
        # a padded decode batch (13 rows, 3 of them padding) on zero-point weights with a shared expert
        dict(name="experts_padded_13", op="experts", T=13, d=4096, E=64, k=6, f=1408, S=1, group=64, zeros=True, padded=3),
        # a decode batch of 64 sequences on the fine-grained layer: every expert is read, a few rows each
        dict(name="experts_fine_64", op="experts", T=64, d=2048, E=128, k=8, f=768, S=0, group=128, zeros=False, padded=0),
        # the decode workload's batch: 256 sequences, 64 rows per expert
        dict(name="experts_eight_256", op="experts", T=256, d=4096, E=8, k=2, f=14336, S=0, group=128, zeros=False, padded=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "quantize", "experts", "experts"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 4, 8])
        E = _log_int(rng, 8, 256) if groups == 1 else groups * rng.randint(2, 256 // groups)
        kept = 1 if groups == 1 else rng.randint(2, groups)
        k = rng.randint(1, min(16, E // groups * kept))
        return dict(op=op, T=_log_int(rng, 1, 32768), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, kept=kept, group_score=rng.choice(["max", "top2"]),
                    renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["float32", "bfloat16"]),
                    pad=rng.choice([0, 0, 3, 8]), masked=rng.random() < 0.4)
    group = rng.choice([32, 64, 128])
    if op == "quantize":
        K = group * _log_int(rng, 1, 14336 // group)
        return dict(op=op, N=_log_int(rng, 64, min(1 << 17, (1 << 28) // K)), K=K, group=group, zeros=rng.random() < 0.5)
    while True:
        d, f = 128 * _log_int(rng, 2, 56), 128 * _log_int(rng, 2, 112)
        E, S = _log_int(rng, 4, 256), rng.choice([0, 0, 1])
        if 3 * (E + S) * d * f <= 1 << 30:
            break
    T = _log_int(rng, 1, 256)
    return dict(op=op, T=T, d=d, E=E, k=rng.randint(1, min(8, E)), f=f, S=S, group=group, zeros=rng.random() < 0.5,
                padded=rng.choice([0, 0, T // 5]))


def work(case):
    c = case
    if c["op"] in ("route", "route_grad"):
        size = 4 if c["dtype"] == "float32" else 2
        slots = c["T"] * c["k"] * 8
        if c["op"] == "route":
            return {"bytes": c["T"] * c["E"] * size + slots + c["E"] * (8 if c["bias"] else 4), "flops": 8 * c["T"] * c["E"]}
        return {"bytes": 2 * c["T"] * c["E"] * size + slots, "flops": 8 * c["T"] * c["E"]}
    per = 0.5 + (2 + (1 if c["zeros"] else 0)) / c["group"]
    if c["op"] == "quantize":
        return {"bytes": c["N"] * c["K"] * 2 * (2 + per), "flops": 6 * c["N"] * c["K"]}
    rows = c["T"] - c["padded"]
    active = c["E"] * (1 - (1 - c["k"] / c["E"]) ** rows) + c["S"]  # experts that at least one row is expected to choose
    return {"bytes": active * 3 * c["d"] * c["f"] * per + c["T"] * (4 * c["d"] + 8 * c["k"]),
            "flops": 6 * c["d"] * c["f"] * rows * (c["k"] + c["S"])}


# ----------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _draw_logits(c, rows, offsets, g):
    """Logits as a router's product gives them: unit normal about an expert's own level."""
    v = torch.randn(rows, c["E"], generator=g, device="cuda") + offsets
    if c["masked"]:
        v.masked_fill_(torch.rand(rows, c["E"], generator=g, device="cuda") < 0.2, -math.inf)
        v.masked_fill_(torch.rand(rows, 1, generator=g, device="cuda") < 0.02, -math.inf)
    return v.to(getattr(torch, c["dtype"]))


def _near(c, logits, bias):
    """Rows in which two compared sums of scores (not logits: those are compared as they are) come within a few
    roundings in 32 bits of one another, so that the choice would not be defined by the formula."""
    x = logits.double()
    s = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(x, -1))
    v = (s + bias.double() if bias is not None else s).masked_fill(x == -math.inf, -math.inf)
    bad = torch.zeros(len(x), dtype=torch.bool, device="cuda")

    def close(sorted_values):
        d = sorted_values[:, :-1] - sorted_values[:, 1:]
        return ((d < 4e-6) & torch.isfinite(d)).any(1)

    if c["groups"] > 1 and (c["group_score"] == "top2" or bias is not None):
        top = v.view(len(x), c["groups"], -1).topk(2, -1).values
        level = top[..., 0]
        if c["group_score"] == "top2":
            level = level + torch.where(top[..., 1] == -math.inf, 0.0, top[..., 1])
        level, order = level.sort(-1, descending=True)
        bad |= close(level[:, c["kept"] - 1 : c["kept"] + 1])
        lost = torch.ones_like(level, dtype=torch.bool).scatter_(1, order[:, : c["kept"]], False)
        v = v.view(len(x), c["groups"], -1).masked_fill(lost[..., None], -math.inf).view(len(x), -1)
    if bias is not None:
        bad |= close(v.sort(-1, descending=True).values[:, : c["k"] + 1])
    return bad


def _logits(c, seed):
    g = _gen(seed)
    offsets = 0.3 * torch.randn(c["E"], generator=g, device="cuda")
    bias = 0.05 * torch.randn(c["E"], generator=g, device="cuda") if c["bias"] else None
    logits = _draw_logits(c, c["T"], offsets, g)
    for _ in range(50):
        rows = _near(c, logits, bias).nonzero()[:, 0]
        if not len(rows):
            break
        logits[rows] = _draw_logits(c, len(rows), offsets, g)
    if c["pad"]:  # columns of a wider buffer
        wide = torch.zeros(c["T"], c["E"] + c["pad"], dtype=logits.dtype, device="cuda")
        wide[:, : c["E"]] = logits
        logits = wide[:, : c["E"]]
    return logits, bias, g


def _codes(rows, cols, group, zeros, sigma, g):
    """4-bit weights as the conversion of normal ones gives them: codes, two to a byte, and their groups' scales."""
    out = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // cols)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        q = torch.randn(n, cols, generator=g, device="cuda").mul_(2.7).add_(8).round_().clamp_(0, 15).to(torch.uint8)
        out[r : r + n] = q[:, 0::2] | (q[:, 1::2] << 4)
    scales = ((0.8 + 0.4 * torch.rand(rows, cols // group, generator=g, device="cuda")) * sigma / 2.7).to(BF16)
    z = torch.randint(6, 11, (rows, cols // group), generator=g, device="cuda").to(torch.uint8) if zeros else None
    return out, scales, z


def prepare(case, seed):
    c = case
    if c["op"] in ("route", "route_grad"):
        logits, bias, g = _logits(c, seed)
        T, k = c["T"], c["k"]
        s = dict(case=c, logits=logits, bias=bias)
        if c["op"] == "route":
            s.update(idx=torch.empty(T, k, dtype=torch.int32, device="cuda"), w=torch.empty(T, k, device="cuda"),
                     counts=torch.empty(c["E"], dtype=torch.int32, device="cuda"))
        else:
            s.update(idx=_plain_route(c, logits, bias)[0], grad_w=torch.randn(T, k, generator=g, device="cuda"),
                     grad=torch.empty(T, c["E"], dtype=logits.dtype, device="cuda"))
        if own:
            from persistent_megakernel_sm_gb300 import MoERouter
            s["router"] = MoERouter(c["E"], k, score=c["score"], groups=c["groups"], groups_kept=c["kept"],
                                    group_score=c["group_score"], renormalise=c["renorm"], scale=c["scale"])
        return s
    g = _gen(seed)
    if c["op"] == "quantize":
        N, K, n = c["N"], c["K"], c["K"] // c["group"]
        weight = torch.empty(N, K, dtype=BF16, device="cuda")
        step = max(1, (1 << 27) // K)
        for r in range(0, N, step):
            weight[r : r + step] = torch.randn(min(step, N - r), K, generator=g, device="cuda") / math.sqrt(K)
        return dict(case=c, weight=weight, codes=torch.empty(N, K // 2, dtype=torch.uint8, device="cuda"),
                    scales=torch.empty(N, n, dtype=BF16, device="cuda"),
                    zeros=torch.empty(N, n, dtype=torch.uint8, device="cuda") if c["zeros"] else None,
                    back=torch.empty(N, K, dtype=BF16, device="cuda"))
    T, d, f, E, k, S = (c[n] for n in ("T", "d", "f", "E", "k", "S"))
    weights = []
    for rows, cols in ((f, d), (f, d), (d, f)):
        parts = _codes((E + S) * rows, cols, c["group"], c["zeros"], cols ** -0.5, g)
        weights.append(tuple(None if p is None else p.view(E + S, rows, -1) for p in parts))
    score = torch.rand(T, E, generator=g, device="cuda")
    idx = score.argsort(-1, descending=True)[:, :k].to(torch.int32)
    w = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), -1)
    if c["padded"]:  # the rows behind the batch's sequences choose nothing
        idx[T - c["padded"]:] = -1
        w[T - c["padded"]:] = 0
    s = dict(case=c, x=torch.randn(T, d, generator=g, device="cuda").to(BF16), idx=idx, w=w, weights=weights,
             out=torch.empty(T, d, dtype=BF16, device="cuda"))
    if own:
        from persistent_megakernel_sm_gb300 import W4Experts
        s["experts"] = W4Experts(d, f, E, k, shared_experts=S, group=c["group"])
        s["experts"].reserve(T)
        s["experts"].set_weights(*weights)
    return s


# ------------------------------------------------------------------ plain forms

def _plain_route(c, logits, bias):
    x = logits.float()
    T, E, k = len(x), c["E"], c["k"]
    dead = x == -math.inf
    if c["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-x))
    else:
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
        s = e / e.sum(1, keepdim=True).clamp_min(1e-38)
    by_sum = bias is not None
    choice = s + bias if by_sum else x
    choice = choice.masked_fill(dead, -math.inf)
    if c["groups"] > 1:
        v = (s if bias is None and c["group_score"] == "top2" else choice).masked_fill(dead, -math.inf)
        v = v.view(T, c["groups"], -1).sort(-1, descending=True).values
        level = v[..., 0]
        if c["group_score"] == "top2" and v.shape[-1] > 1:
            level = level + torch.where(v[..., 1] == -math.inf, 0.0, v[..., 1])
        order = level.sort(dim=1, descending=True, stable=True).indices
        keep = torch.zeros(T, c["groups"], dtype=torch.bool, device=x.device).scatter_(1, order[:, : c["kept"]], True)
        choice = choice.view(T, c["groups"], -1).masked_fill(~keep[..., None], -math.inf).view(T, E)
    value, idx = choice.sort(dim=1, descending=True, stable=True)
    value, idx = value[:, :k], idx[:, :k]
    live = value > -math.inf
    w = torch.where(live, s.gather(1, idx), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-38)
    idx = torch.where(live, idx, -1)
    counts = torch.zeros(E, dtype=torch.int32, device=x.device)
    counts.scatter_add_(0, idx.clamp_min(0).view(-1), live.to(torch.int32).view(-1))
    return idx.to(torch.int32), w * c["scale"], counts


def _plain_route_grad(c, logits, idx, grad_w):
    x = logits.float()
    live = idx >= 0
    at = idx.clamp_min(0).long()
    gw = torch.where(live, grad_w, 0.0) * c["scale"]
    if c["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-x))
    else:
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
        s = e / e.sum(1, keepdim=True).clamp_min(1e-38)
    if c["renorm"]:
        kept = torch.where(live, s.gather(1, at), 0.0)
        total = kept.sum(1, keepdim=True).clamp_min(1e-38)
        gw = torch.where(live, (gw - (gw * kept / total).sum(1, keepdim=True)) / total, 0.0)
    ds = torch.zeros_like(s).scatter_add_(1, at, gw)
    if c["score"] == "sigmoid":
        grad = ds * s * (1 / (1 + torch.exp(x)))
    else:
        grad = s * (ds - (ds * s).sum(1, keepdim=True))
    return grad.to(logits.dtype)


def _plain_values(codes, scales, zeros, group):
    """The weights that codes, scales and zero points stand for, in 32 bits."""
    q = torch.stack((codes & 15, codes >> 4), -1).view(*codes.shape[:-1], -1, group).float()
    q = q - (8 if zeros is None else zeros.unsqueeze(-1))
    return (q * scales.unsqueeze(-1)).view(*codes.shape[:-1], -1)


def _plain_quantize(c, weight):
    v = weight.float().view(c["N"], -1, c["group"])
    if c["zeros"]:
        lo, hi = v.amin(-1).clamp_max(0), v.amax(-1).clamp_min(0)
        scales = ((hi - lo) / 15).to(BF16)
        step = torch.where(scales == 0, 1.0, scales.float())
        zeros = torch.round(-lo / step).clamp(0, 15)
        q = (torch.round(v / step.unsqueeze(-1)) + zeros.unsqueeze(-1)).clamp(0, 15)
    else:
        scales = (v.abs().amax(-1) / 7).to(BF16)
        step = torch.where(scales == 0, 1.0, scales.float())
        zeros = None
        q = torch.round(v / step.unsqueeze(-1)).clamp(-8, 7) + 8
    q = q.to(torch.uint8).view(c["N"], -1)
    codes = q[:, 0::2] | (q[:, 1::2] << 4)
    zeros = None if zeros is None else zeros.to(torch.uint8)
    return _plain_values(codes, scales, zeros, c["group"]).to(BF16), scales, zeros


def _plain_experts(c, s):
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    x = s["x"].float()
    live = s["idx"] >= 0
    w = torch.where(live, s["w"], 0.0)
    at = s["idx"].clamp_min(0).long()
    if T * k <= E:  # few rows: each one's own experts' weights
        pick = at.view(-1)
        gate, up, down = (_plain_values(*(None if p is None else p[:E][pick] for p in m), c["group"]) for m in s["weights"])
        rows = x.repeat_interleave(k, 0).unsqueeze(-1)
        z = gate @ rows
        y = down @ (z / (1 + torch.exp(-z)) * (up @ rows))
        out = (y.view(T, k, -1) * w.unsqueeze(-1)).sum(1)
    else:  # many: every expert on every row, weighted (by zero where it was not chosen)
        gate, up, down = (_plain_values(*(None if p is None else p[:E] for p in m), c["group"]) for m in s["weights"])
        z = gate @ x.t()
        h = z / (1 + torch.exp(-z)) * (up @ x.t())
        full = torch.zeros(T, E, device=x.device).scatter_add_(1, at, w)
        out = (down @ (h * full.t().unsqueeze(1))).sum(0).t()
    if S:
        gate, up, down = (_plain_values(*(None if p is None else p[E] for p in m), c["group"]) for m in s["weights"])
        z = x @ gate.t()
        out = out + (z / (1 + torch.exp(-z)) * (x @ up.t())) @ down.t()
    return out.to(BF16)


def run(state):
    s, c = state, state["case"]
    if c["op"] == "route":
        if own:
            s["router"].forward(s["logits"], s["idx"], s["w"], bias=s["bias"], counts=s["counts"])
            return s["idx"], s["w"], s["counts"]
        return _plain_route(c, s["logits"], s["bias"])
    if c["op"] == "route_grad":
        if own:
            s["router"].backward(s["logits"], s["idx"], s["grad_w"], s["grad"])
            return s["grad"]
        return _plain_route_grad(c, s["logits"], s["idx"], s["grad_w"])
    if c["op"] == "quantize":
        if own:
            from persistent_megakernel_sm_gb300 import w4_dequantize, w4_quantize
            w4_quantize(s["weight"], s["codes"], s["scales"], s["zeros"])
            w4_dequantize(s["codes"], s["scales"], s["zeros"], s["back"])
            return s["back"], s["scales"], s["zeros"]
        return _plain_quantize(c, s["weight"])
    if own:
        s["experts"].forward(s["x"], s["idx"], s["w"], s["out"])
        return s["out"]
    return _plain_experts(c, s)


# ---------------------------------------------------------------- in 64 bits

def _f64(t):
    return t.detach().double().cpu().numpy()


def _exact_scores(c, x):
    with np.errstate(all="ignore"):
        if c["score"] == "sigmoid":
            return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
        top = x.max(1, keepdims=True)
        e = np.exp(x - np.where(np.isfinite(top), top, 0))
        return e / np.maximum(e.sum(1, keepdims=True), 1e-300)


def _exact_route(c, x, bias):
    T, E, k = len(x), c["E"], c["k"]
    s = _exact_scores(c, x)
    sel = x if bias is None else np.where(np.isneginf(x), -np.inf, s + bias)
    if c["groups"] > 1:
        level = sel if bias is not None or c["group_score"] == "max" else np.where(np.isneginf(x), -np.inf, s)
        level = -np.sort(-level.reshape(T, c["groups"], -1), axis=-1)
        second = level[:, :, 1] if c["group_score"] == "top2" and level.shape[2] > 1 else 0.0
        level = level[:, :, 0] + np.where(np.isneginf(second), 0.0, second)
        out = np.argsort(-level, axis=1, kind="stable")[:, c["kept"]:]
        sel = sel.reshape(T, c["groups"], -1).copy()
        np.put_along_axis(sel, out[:, :, None], -np.inf, axis=1)
        sel = sel.reshape(T, E)
    idx = np.argsort(-sel, axis=1, kind="stable")[:, :k]
    gone = np.isneginf(np.take_along_axis(sel, idx, 1))
    w = np.where(gone, 0.0, np.take_along_axis(s, idx, 1))
    if c["renorm"]:
        w = w / np.where(w.sum(1, keepdims=True) > 0, w.sum(1, keepdims=True), 1.0)
    idx = np.where(gone, -1, idx)
    return idx.astype(np.int32), c["scale"] * w, np.bincount(idx[idx >= 0], minlength=E).astype(np.int32)


def _exact_route_grad(c, x, idx, gw):
    """Through the Jacobian, slot by slot: dw_j/dl_e = w_j (d log s_j / dl_e - sum_i (w_i / scale) d log s_i / dl_e)."""
    s = _exact_scores(c, x)
    rows, live = np.arange(len(x)), idx >= 0
    at = np.where(live, idx, 0)
    sk = np.where(live, np.take_along_axis(s, at, 1), 0.0)
    share = sk / np.where(sk.sum(1, keepdims=True) > 0, sk.sum(1, keepdims=True), 1.0)
    w = c["scale"] * (share if c["renorm"] else sk)
    a = np.where(live, gw, 0.0) * w  # the gradient of log s_j, before the sum over all is taken off
    if c["renorm"]:
        a = a - share * a.sum(1, keepdims=True)
    grad = np.zeros_like(x)
    for j in range(c["k"]):
        own_part = a[:, j] * ((1 - s[rows, at[:, j]]) if c["score"] == "sigmoid" else 1.0)
        np.add.at(grad, (rows, at[:, j]), np.where(live[:, j], own_part, 0.0))
    if c["score"] == "softmax":
        grad -= s * a.sum(1, keepdims=True)
    return grad


def _exact_values(codes, scales, zeros, group):
    rows = codes.shape[0]
    q = torch.empty(rows, codes.shape[1] * 2, dtype=torch.float64, device=codes.device)
    q[:, 0::2] = (codes % 16).double()
    q[:, 1::2] = (codes // 16).double()
    z = torch.full_like(scales, 8).double() if zeros is None else zeros.double()
    return (q - z.repeat_interleave(group, 1)) * scales.double().repeat_interleave(group, 1)


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] in ("route", "route_grad"):
        x = _f64(s["logits"])
        if c["op"] == "route":
            return _exact_route(c, x, None if s["bias"] is None else _f64(s["bias"]))
        return _exact_route_grad(c, x, s["idx"].cpu().numpy(), _f64(s["grad_w"]))
    if c["op"] == "quantize":
        back = torch.empty(c["N"], c["K"], dtype=torch.float64, device="cuda")
        scales = torch.empty(c["N"], c["K"] // c["group"], dtype=torch.float64, device="cuda")
        zeros = torch.empty_like(scales) if c["zeros"] else None
        step = max(1, (1 << 26) // c["K"])
        for r in range(0, c["N"], step):
            v = s["weight"][r : r + step].double().unflatten(1, (-1, c["group"]))
            lo = torch.minimum(v.min(-1).values, torch.zeros((), dtype=torch.float64, device="cuda"))
            hi = torch.maximum(v.max(-1).values, torch.zeros((), dtype=torch.float64, device="cuda"))
            by = (hi - lo) / 15 if c["zeros"] else torch.maximum(hi, -lo) / 7
            by = by.to(BF16).double()  # the scale is held in bf16 by definition
            div = torch.where(by > 0, by, torch.ones_like(by))
            z = (-lo / div).round().clamp(0, 15) if c["zeros"] else torch.full_like(by, 8)
            q = ((v / div.unsqueeze(-1)).round() + z.unsqueeze(-1)).clamp(0, 15)
            back[r : r + step] = ((q - z.unsqueeze(-1)) * by.unsqueeze(-1)).flatten(1)
            scales[r : r + step] = by
            if c["zeros"]:
                zeros[r : r + step] = z
        return back, scales, None if zeros is None else zeros.to(torch.uint8)
    T, E, S = c["T"], c["E"], c["S"]
    x, out = s["x"].double(), torch.zeros(T, c["d"], dtype=torch.float64, device="cuda")
    for e in range(E + S):
        weight = (s["w"].double() * (s["idx"] == e)).sum(1) if e < E else torch.ones(T, dtype=torch.float64, device="cuda")
        rows = (s["idx"] == e).any(1).nonzero()[:, 0] if e < E else torch.arange(T, device="cuda")
        if not len(rows):
            continue
        z = x[rows] @ _exact_values(*(None if p is None else p[e] for p in s["weights"][0]), c["group"]).t()
        u = x[rows] @ _exact_values(*(None if p is None else p[e] for p in s["weights"][1]), c["group"]).t()
        h = z * torch.sigmoid(z) * u
        out[rows] += weight[rows, None] * (h @ _exact_values(*(None if p is None else p[e] for p in s["weights"][2]), c["group"]).t())
    return out
