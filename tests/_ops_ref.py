"""The routing operators and the 4-bit experts in 64 bits, from their
definitions (numpy, plain loops where they say it best), and the inputs that
their tests share."""
import numpy as np

U32 = 2.0 ** -24     # half a step of fp32, relative
U16 = 2.0 ** -8      # half a step of bf16, relative


def bf16(a):
    """Rounded to bf16 (half to even), as float64."""
    a32 = np.asarray(a, dtype=np.float32)
    u = a32.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32)
    return np.where(np.isnan(a32), np.nan, r.view(np.float32)).astype(np.float64)


# --------------------------------------------------------------------- routing

def scores(l, score):
    l = np.asarray(l, dtype=np.float64)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return np.where(l >= 0, 1 / (1 + np.exp(-l)), np.exp(l) / (1 + np.exp(l)))
        m = np.max(l, axis=1, keepdims=True)
        e = np.exp(l - np.where(np.isneginf(m), 0, m))
        z = e.sum(1, keepdims=True)
        return np.where(z == 0, 0.0, e / np.where(z == 0, 1.0, z))


def order_desc(v):
    """Indices by value, larger first, NaN before all, the lower index on ties."""
    return sorted(range(len(v)), key=lambda i: (0 if np.isnan(v[i]) else 1, 0.0 if np.isnan(v[i]) else -v[i], i))


def levels(c, s, l, r, biased):
    v = c if biased else s if r["group_score"] == "top2" else l
    out = []
    for g in v.reshape(r["groups"], -1):
        top = [g[i] for i in order_desc(g)[:2]]
        add = r["group_score"] == "top2" and len(top) == 2 and not np.isneginf(top[1])
        out.append(top[0] + top[1] if add else top[0])
    return np.array(out)


def route(l, r, bias=None):
    """idx [T, k] and w [T, k] of settings r (a dict of MoERouter's arguments)."""
    l = np.asarray(l, dtype=np.float64)
    T, E = l.shape
    k = r["k"]
    s = scores(l, r["score"])
    idx, w = np.full((T, k), -1, dtype=np.int32), np.zeros((T, k))
    for t in range(T):
        dead = np.isneginf(l[t]) | (np.isneginf(bias) if bias is not None else False)
        c = np.where(dead, -np.inf, s[t] + bias if bias is not None else l[t])
        if r["groups"] > 1:
            lv = levels(c, np.where(dead, -np.inf, s[t]), np.where(dead, -np.inf, l[t]), r, bias is not None)
            for g in order_desc(lv)[r["groups_kept"]:]:
                c[g * (E // r["groups"]):(g + 1) * (E // r["groups"])] = -np.inf
        pick = [e for e in order_desc(c) if not np.isneginf(c[e])][:k]
        idx[t, :len(pick)] = pick
        with np.errstate(all="ignore"):
            if r["renormalise"] and pick:
                x = l[t, pick]
                m = x.max() if r["score"] == "softmax" else min(x.max(), 0.0)
                a = np.exp(x - m) if r["score"] == "softmax" else \
                    np.where(x > 0, 1 / (1 + np.exp(-x)), np.exp(x - m) / (1 + np.exp(x)))
                w[t, :len(pick)] = a / a.sum()
            else:
                w[t, :len(pick)] = s[t, pick]
    return idx, r["scale"] * w


def route_grad(l, r, idx, gw):
    """The gradient and, for each value, the sum of the magnitudes it is made of."""
    l = np.asarray(l, dtype=np.float64)
    s = scores(l, r["score"])
    grad, size = np.zeros_like(l), np.zeros_like(l)
    for t in range(len(l)):
        js = [j for j in range(r["k"]) if 0 <= idx[t, j] < l.shape[1]]
        es, g = [int(idx[t, j]) for j in js], np.array([gw[t, j] for j in js])
        if not js:
            continue
        x = l[t, es]
        if r["renormalise"]:
            m = x.max() if r["score"] == "softmax" else min(x.max(), 0.0)
            a = np.exp(x - m) if r["score"] == "softmax" else \
                np.where(x > 0, 1 / (1 + np.exp(-x)), np.exp(x - m) / (1 + np.exp(x)))
            a = a / a.sum()
            v, mag = a * (g - (g * a).sum()), a * (np.abs(g) + (np.abs(g) * a).sum())
        else:
            v, mag = s[t, es] * g, s[t, es] * np.abs(g)
        if r["score"] == "sigmoid":
            v, mag = v * scores(-x[None], "sigmoid")[0], mag * scores(-x[None], "sigmoid")[0]
        for e, vi, mi in zip(es, v, mag):
            grad[t, e] += vi
            size[t, e] += mi
        if r["score"] == "softmax" and not r["renormalise"]:
            grad[t] -= s[t] * (s[t, es] * g).sum()
            size[t] += s[t] * (s[t, es] * np.abs(g)).sum()
    return r["scale"] * grad, abs(r["scale"]) * size


def clear_logits(rng, T, r, bias, std=1.0, masked=0.0, to=lambda a: a.astype(np.float32).astype(np.float64)):
    """Logits whose choice does not hang on a few fp32 roundings: rows in which
    compared scores come within 4e-6 are drawn again."""
    E = r["E"]
    out = np.empty((T, E))
    for t in range(T):
        while True:
            l = to(rng.standard_normal(E) * std)
            l[rng.random(E) < masked] = -np.inf
            s = scores(l[None], r["score"])[0]
            c = np.where(np.isneginf(l), -np.inf, s + bias if bias is not None else l)
            ok = True
            if r["groups"] > 1:
                v = np.sort(levels(c, np.where(np.isneginf(l), -np.inf, s), l, r, bias is not None))[::-1]
                ok = not (v[r["groups_kept"] - 1] - v[min(r["groups_kept"], r["groups"] - 1)] < 4e-6
                          and r["groups_kept"] < r["groups"])
            if bias is not None:
                v = np.sort(c[~np.isneginf(c)])
                ok = ok and (len(v) < 2 or np.diff(v).min() > 4e-6)
            if ok:
                out[t] = l
                break
    return out


# ---------------------------------------------------------------- 4-bit weights

def values(codes, scales, zeros):
    """codes [.., N, K / 2] uint8, scales [.., N, K / G] -> [.., N, K] float64."""
    codes = np.asarray(codes)
    q = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,))
    q[..., 0::2], q[..., 1::2] = codes & 15, codes >> 4
    group = q.shape[-1] // scales.shape[-1]
    z = np.repeat(8.0 if zeros is None else np.asarray(zeros, dtype=np.float64), group, -1) if zeros is not None else 8.0
    return (q - z) * np.repeat(np.asarray(scales, dtype=np.float64), group, -1)


def quantize(w, group, with_zeros):
    """codes, scales, zeros of bf16 values w [N, K] (finite), by the definition."""
    v = np.asarray(w, dtype=np.float64).reshape(w.shape[0], -1, group)
    lo, hi = np.minimum(v.min(-1), 0), np.maximum(v.max(-1), 0)
    s = bf16(((hi - lo) / 15 if with_zeros else np.maximum(hi, -lo) / 7).astype(np.float32))
    div = np.where(s == 0, 1.0, s)
    z = np.clip(np.round(-lo / div), 0, 15) if with_zeros else np.full(s.shape, 8.0)
    q = np.clip(np.round(v / div[..., None]) + z[..., None], 0, 15).reshape(w.shape).astype(np.uint8)
    return q[:, 0::2] | (q[:, 1::2] << 4), s, z.astype(np.uint8) if with_zeros else None


def make_w4(rng, rows, cols, group, zeros, lead=()):
    codes = rng.integers(0, 256, lead + (rows, cols // 2), dtype=np.uint8)
    scales = bf16((0.5 + rng.random(lead + (rows, cols // group))) / (4.6 * np.sqrt(cols)))
    z = rng.integers(0, 16, lead + (rows, cols // group), dtype=np.uint8) if zeros else None
    return codes, scales, z


def experts(x, idx, w, gate, up, down, E, S):
    """out [T, d] and the bound of each value's error.

    Bound: products of 4-bit values and bf16 are summed in fp32, at most K
    additions a sum, each off by at most one fp32 step (2^-23) of the
    magnitudes' sum; h, the weights' scaled values (where a kernel rounds
    them) and out are rounded to bf16 (2^-8 each); silu is within 8 steps."""
    T, d = x.shape
    out, off = np.zeros((T, d)), np.zeros((T, d))
    G, U, D = values(*gate), values(*up), values(*down)
    f = G.shape[1]
    for t in range(T):
        slots = [(int(e), float(v)) for e, v in zip(idx[t], w[t]) if 0 <= e < E] + ([(E, 1.0)] if S else [])
        for e, v in slots:
            z, u = G[e] @ x[t], U[e] @ x[t]
            az, au = np.abs(G[e]) @ np.abs(x[t]), np.abs(U[e]) @ np.abs(x[t])
            rel = d * 2 * U32 + U16
            silu = z / (1 + np.exp(-z))
            h = silu * u
            dh = 1.1 * az * rel * np.abs(u) + np.abs(silu) * au * rel + np.abs(h) * (U16 + 16 * U32)
            out[t] += v * (D[e] @ h)
            off[t] += abs(v) * (np.abs(D[e]) @ (dh + np.abs(h) * (f * 2 * U32 + U16)))
    return out, off + np.abs(out) * (U16 + 20 * U32) + 1e-30


#: Relative 2-norm of out's error: at most four bf16 roundings lie on a value's
#: way (two of scaled weights, h, out), independent of one another and of the
#: values, each of root mean square at most 2^-8 / sqrt(3).
EXPERTS_NORM = 1.25 * U16
