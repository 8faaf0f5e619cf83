"""FP64 CPU reference of the 4-bit (MXFP4) operators, in numpy.

Written from the format's definition alone: a block's scale is a power of two,
its values are the nearest of the 15 levels, ties to the one with the even
code.  Test infrastructure only.
"""
import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def shapes(rows, cols):
    """Shapes of the arrays (codes, scales) of a rows x cols matrix."""
    slabs = -(-cols // 128)
    return (rows, 64 * slabs), (slabs, -(-rows // 32) * 32, 4)


def quantize(x, noclip=False):
    """(codes, scales) of x, blocks along its rows."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    slabs = -(-cols // 128)
    v = np.zeros((rows, slabs * 128))
    v[:, :cols] = x
    v = v.reshape(rows, slabs * 4, 32)
    m = np.abs(v).max(axis=2) if slabs else np.zeros((rows, 0))
    finite = np.isfinite(v).all(axis=2)
    m = np.where(finite, m, 1.0)
    e = np.frexp(np.where(m > 0, m, 1.0))[1] - 1              # floor(log2 m)
    s = e - 2
    if noclip:
        s = s + (m > 6 * np.ldexp(1.0, s))
    s = np.where(m > 0, np.maximum(s, -127), -127)
    y = np.abs(np.where(finite[..., None], v, 0.0)) / np.ldexp(1.0, s)[..., None]
    y = np.minimum(y, 6.0)
    d = np.abs(y[..., None] - LEVELS)
    near = d.min(axis=-1, keepdims=True)
    tie = d == near
    # Of two levels equally near, the even code.
    code = np.where(tie, np.arange(8) % 2 * 8 + np.arange(8), 99).min(axis=-1) % 8
    code = np.where(tie.sum(axis=-1) == 1, tie.argmax(axis=-1), code)
    code = code + 8 * np.signbit(v)
    code = np.where(finite[..., None], code, 0).astype(np.uint8)
    flat = code.reshape(rows, slabs * 128)
    codes = flat[:, 0::2] | flat[:, 1::2] << 4
    byte = np.where(finite, s + 127, 255).astype(np.uint8)
    scales = np.zeros(shapes(rows, cols)[1], dtype=np.uint8)
    scales[:, :rows] = byte.reshape(rows, slabs, 4).transpose(1, 0, 2)
    return codes, scales


def values(codes, scales, cols):
    """The values that codes and scales stand for, in 64 bits."""
    rows, half = codes.shape
    c = np.empty((rows, 2 * half), dtype=np.uint8)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    v = LEVELS[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = scales[:, :rows].transpose(1, 0, 2).reshape(rows, half // 16).astype(np.int64)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return (v * np.repeat(f, 32, axis=1))[:, :cols]


def rounded(x, noclip=False):
    return values(*quantize(x, noclip), np.shape(x)[1])


def moe(x, router, up, down, top, norm, act_bits):
    """(y, bound) of the expert layer in 64 bits: up (E, 2F, H), down (E, H, F).

    bound: how far fp32 sums in any order, activations held to act_bits bits
    and exponentials good to a few units of fp32 may move y before its own
    rounding.
    """
    t_n, h_n = x.shape
    e_n, f2, _ = up.shape
    f_n = f2 // 2
    u = 2.0 ** -23            # a step of fp32: covers sums that cut instead of rounding
    y, bound = np.zeros_like(x), np.zeros_like(x)
    logits = x @ router.T
    for t in range(t_n):
        order = sorted(range(e_n), key=lambda e: (-logits[t, e], e))[:top]
        ex = np.exp(logits[t] - logits[t, order[0]])
        total = ex[order].sum() if norm else ex.sum()
        for e in order:
            p = ex[e] / total
            z = up[e] @ x[t]
            dz = u * h_n * (np.abs(up[e]) @ np.abs(x[t]))
            g, v, dg, dv = z[:f_n], z[f_n:], dz[:f_n], dz[f_n:]
            sig = 1 / (1 + np.exp(-g))
            act = g * sig * v
            dact = 1.1 * dg * (np.abs(v) + dv) + (np.abs(g * sig) + 1.1 * dg) * dv + np.abs(act) * (2.0 ** -act_bits + 16 * u)
            part = down[e] @ act
            size = np.abs(down[e]) @ np.abs(act)
            y[t] += p * part
            # The weight: an exponential, a sum of up to E of them, a quotient.
            bound[t] += p * (np.abs(down[e]) @ dact + size * u * (f_n + top + 32))
    return y, bound
