"""What the 4-bit experts' outputs may be off, by the roundings that each of the
two kinds of kernels makes.

Both hold sums in fp32 and round h and out to bf16.  The kernels for few rows an
expert round no weight: they sum q x and x and put scale and zero point on the
sums, so their sums' error goes with sum scale (q + zero) |x|.  The tile kernels
round each weight, (q - zero) scale, to the 11 bits of fp16."""
import numpy as np

import _ops_ref as ref

U11 = 2.0 ** -11     # half a step of fp16, relative

#: Relative 2-norm of out's error.  Rounding to bf16 is off by at most half a
#: step, evenly spread: 2^-8 / sqrt(3) of the power of two below the value in
#: the root mean square, and sqrt(3 / (8 ln 2)) = 0.7355 of that of the value
#: where its logarithm is spread evenly.  h's rounding and out's are
#: independent, so they add up as squares; the rounding of three factors to 11
#: bits adds 2^-6 of one of them, which is nothing.  A quarter more is for
#: chance among a few hundred values: 2.93e-3.
NORM = 1.25 * np.sqrt(2.0) * np.sqrt(3 / (8 * np.log(2))) * ref.U16 / np.sqrt(3)


def _magnitudes(codes, scales, zeros, rounded):
    """Per weight, what the sums' magnitudes are made of."""
    if rounded:
        return np.abs(ref.values(codes, scales, zeros))
    q = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,))
    q[..., 0::2], q[..., 1::2] = codes & 15, codes >> 4
    group = q.shape[-1] // scales.shape[-1]
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, -1)
    return (q + z) * np.repeat(np.abs(scales), group, -1)


def experts(x, idx, w, gate, up, down, E, S, tiles):
    """out [T, d] in 64 bits and the bound of each value's error, on the tile
    kernels or the others."""
    T, d = x.shape
    out, off = np.zeros((T, d)), np.zeros((T, d))
    val = [ref.values(*m) for m in (gate, up, down)]
    mag = [_magnitudes(*m, tiles) for m in (gate, up, down)]
    f = val[0].shape[1]
    rel = U11 * (1 + U11) if tiles else 0.0
    for t in range(T):
        slots = [(int(e), float(v)) for e, v in zip(idx[t], w[t]) if 0 <= e < E] + ([(E, 1.0)] if S else [])
        for e, v in slots:
            z, u = val[0][e] @ x[t], val[1][e] @ x[t]
            # a product or addition an input at most, each off by a step of fp32
            dz = mag[0][e] @ np.abs(x[t]) * (2 * d * ref.U32) + np.abs(val[0][e]) @ np.abs(x[t]) * rel
            du = mag[1][e] @ np.abs(x[t]) * (2 * d * ref.U32) + np.abs(val[1][e]) @ np.abs(x[t]) * rel
            with np.errstate(over="ignore"):
                silu = z / (1 + np.exp(-z))
            h = silu * u
            # silu's slope is at most 1.1; its exponential within (2 + 1.2 |z|)
            # steps, its quotient and the products within 16 half steps
            dh = 1.1 * dz * (np.abs(u) + du) + np.abs(silu) * du + np.abs(h) * (ref.U16 + (20 + 3 * np.abs(z)) * ref.U32)
            hm = np.abs(h) + dh
            out[t] += v * (val[2][e] @ h)
            off[t] += abs(v) * (np.abs(val[2][e]) @ (dh + hm * rel) + mag[2][e] @ hm * (2 * f * ref.U32))
    return out, off + (np.abs(out) + off) * (ref.U16 + 20 * ref.U32)
