"""The norms about a block, their gradient and 8-bit rows in 64 bits, from their
definitions, with how large the terms are that each value is summed from (what
fp32 roundings are relative to)."""
import numpy as np

import _ops_ref as ref

U32 = 2.0 ** -24


def bf16(a):
    return ref.bf16(np.asarray(a, dtype=np.float64))


def as_type(a, kind):
    return bf16(a) if kind == "bfloat16" else np.asarray(a, dtype=np.float32).astype(np.float64)


# ------------------------------------------------------------------- 8-bit rows

def rows8(v, group, kind):
    """codes int8 and scales: in fp32, as the definition has it."""
    v = np.asarray(v, dtype=np.float32)
    T, d = v.shape
    codes, scales = np.zeros((T, d), dtype=np.int8), np.zeros((T, -(-d // group)))
    with np.errstate(all="ignore"):
        for g, lo in enumerate(range(0, d, group)):
            part = v[:, lo:lo + group]
            most = np.abs(part).max(1)
            s = bf16(most / np.float32(127))
            fine = np.isfinite(most)
            div = np.where(s == 0, 1, s).astype(np.float32)
            q = np.clip(np.rint(part / div[:, None]), -127, 127)
            codes[:, lo:lo + group] = np.where(fine[:, None], q, 0)
            scales[:, g] = np.where(fine, s, np.nan)
    return codes, scales


def rows8_values(codes, scales, group):
    return codes.astype(np.float64) * np.repeat(scales, group, 1)[:, :codes.shape[1]]


# ------------------------------------------------------------------------ norms

def moments(x, kind, eps):
    if kind == "none":
        return np.zeros((len(x), 1)), np.ones((len(x), 1))
    m = x.mean(1, keepdims=True) if kind == "layer" else np.zeros((len(x), 1))
    return m, 1 / np.sqrt(((x - m) ** 2).mean(1, keepdims=True) + eps)


def vec(p, none, plus=0.0):
    return none if p is None else p + plus


def gate_of(c, gate):
    return 1.0 if gate is None else gate[:, None] if c["gate"] == "token" else gate


def summed(c, residual, y, p, gate):
    """out before it is rounded, the post norm's statistics, and the terms' size."""
    m, r = moments(y, c["post"], c["eps"])
    g = c["scale"] * gate_of(c, gate)
    k, b = (1.0, 0.0) if c["post"] == "none" else (vec(p["post_gain"], 1.0, c["one"]), vec(p["post_shift"], 0.0))
    out = residual + g * ((y - m) * r * k + b)
    size = np.abs(residual) + np.abs(g) * ((np.abs(y) + np.abs(m)) * r * np.abs(k) + np.abs(b))
    return out, m, r, size


def normed(c, out, p):
    m, r = moments(out, c["pre"], c["eps"])
    k, b = vec(p["pre_gain"], 1.0, c["one"]), vec(p["pre_shift"], 0.0)
    return (out - m) * r * k + b, m, r, (np.abs(out) + np.abs(m)) * r * np.abs(k) + np.abs(b)


def backward(c, p, gate, stats, grad_out, grad_norm, out, y):
    """The gradients, as {name: (value, size of its terms)}; out, y: what was kept."""
    d = (grad_out if grad_out is not None else grad_norm).shape[1]
    my, ry, m, r = (stats[:, i:i + 1] for i in range(4))
    G = np.zeros_like(grad_norm if grad_out is None else grad_out) if grad_out is None else grad_out
    Gs = np.abs(G)
    got = {}
    if grad_norm is not None:
        u, us = (out - m) * r, (np.abs(out) + np.abs(m)) * r
        t = grad_norm * vec(p["pre_gain"], 1.0, c["one"])
        along, mean = (t * u).sum(1, keepdims=True) / d, t.sum(1, keepdims=True) / d
        back = t - u * along - (mean if c["pre"] == "layer" else 0)
        G = G + r * back
        Gs = Gs + r * (np.abs(t) + us * (np.abs(t) * us).mean(1, keepdims=True) +
                       (np.abs(t).mean(1, keepdims=True) if c["pre"] == "layer" else 0))
        got["pre_gain"] = (grad_norm * u).sum(0), (np.abs(grad_norm) * us).sum(0)
        got["pre_shift"] = grad_norm.sum(0), np.abs(grad_norm).sum(0)
    got["residual"] = G, Gs
    g = c["scale"] * gate_of(c, gate)
    P, Ps = g * G, np.abs(g) * Gs
    v = vs = 0.0
    if y is not None:
        v, vs = (y, np.abs(y)) if c["post"] == "none" else ((y - my) * ry, (np.abs(y) + np.abs(my)) * ry)
        k, b = (1.0, 0.0) if c["post"] == "none" else (vec(p["post_gain"], 1.0, c["one"]), vec(p["post_shift"], 0.0))
        if gate is not None:
            e, es = c["scale"] * G * (v * k + b), np.abs(c["scale"]) * Gs * (vs * np.abs(k) + np.abs(b))
            axis = {"channel": 0, "token": 1}.get(c["gate"])
            got["gate"] = (e, es) if axis is None else (e.sum(axis), es.sum(axis))
        if c["post"] != "none":
            got["post_gain"] = (P * v).sum(0), (Ps * vs).sum(0)
            got["post_shift"] = P.sum(0), Ps.sum(0)
            t, ts = P * k, Ps * np.abs(k)
            layer = c["post"] == "layer"
            P = ry * (t - v * (t * v).mean(1, keepdims=True) - (t.mean(1, keepdims=True) if layer else 0))
            Ps = ry * (ts + vs * (ts * vs).mean(1, keepdims=True) + (ts.mean(1, keepdims=True) if layer else 0))
    got["y"] = P, Ps
    return got


# ------------------------------------------------------- the layer for a few tokens

def choice(x, router_w, bias, k):
    """idx and w of the layer's router: the larger logit first, the lower expert on ties, -1 for what is masked."""
    logits = x @ router_w.T + (0 if bias is None else bias)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    top = np.take_along_axis(logits, idx.astype(np.int64), 1)
    with np.errstate(invalid="ignore"):
        w = np.where(np.isneginf(top), 0.0, np.exp(top - np.where(np.isneginf(top[:, :1]), 0, top[:, :1])))
    idx[np.isneginf(top)] = -1
    total = w.sum(1, keepdims=True)
    return idx, w / np.where(total > 0, total, 1)


def experts(x, idx, w, gate, up, down, shared):
    """out and a bound on what fp32 sums and a 16-bit h lose of it: 128 roundings of the terms' sum for a product (no
    chain of sums has as many), and 2^-16 of h."""
    E = len(gate) - shared
    out, err = np.zeros_like(x), np.zeros_like(x)
    rel = 128 * U32
    slots = [(t, int(e), w[t, j]) for t in range(len(x)) for j, e in enumerate(idx[t]) if 0 <= e < E]
    slots += [(t, E, 1.0) for t in range(len(x)) if shared]
    for t, e, wt in slots:
        z, u = gate[e] @ x[t], up[e] @ x[t]
        ez, eu = rel * (np.abs(gate[e]) @ np.abs(x[t])), rel * (np.abs(up[e]) @ np.abs(x[t]))
        s = z / (1 + np.exp(-z))
        h = s * u
        eh = 1.1 * ez * (np.abs(u) + eu) + np.abs(s) * eu + (2.0 ** -16 + 16 * U32) * np.abs(h)
        out[t] += wt * (down[e] @ h)
        err[t] += np.abs(wt) * (np.abs(down[e]) @ (eh + rel * np.abs(h)))
    return out, err
