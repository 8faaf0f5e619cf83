"""FP64 CPU reference of the 8-bit integer operators, in numpy.

Written from the format's definition alone: a scale is the largest magnitude
over the number of levels, as the 32-bit float that the format keeps, values are
the nearest whole multiples, ties to the even one.  Test infrastructure only.
"""
import numpy as np

LEVELS, LEVELS16, GROUP = 127, 32639, 128
FLOOR = 2.0 ** -126


def padded(cols):
    return -(-cols // 128) * 128


def whole(x, levels=LEVELS):
    """(whole numbers, scales) of each row of x, in 64 bits; 0 and NaN where a row holds a NaN or an infinity."""
    x = np.asarray(x, dtype=np.float64)
    finite = np.isfinite(x).all(axis=-1, keepdims=True)
    v = np.where(finite, x, 0.0)
    m = np.abs(v).max(axis=-1, keepdims=True) if x.shape[-1] else np.zeros(x.shape[:-1] + (1,))
    s = np.maximum((m / levels).astype(np.float32).astype(np.float64), FLOOR)
    return np.rint(v / s), np.where(finite, s, np.nan)[..., 0]


def grouped(x):
    """The same for each 128 columns of a row: (rows, padded columns) and (rows, groups)."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    v = np.zeros((rows, padded(cols)))
    v[:, :cols] = x
    q, s = whole(v.reshape(rows, padded(cols) // GROUP, GROUP))
    return q.reshape(rows, -1), s


def values(q, s, cols):
    """What 8-bit numbers and scales (of rows or groups) stand for, rounded to 32 bits as the format has it."""
    s = np.asarray(s, dtype=np.float32)
    s = s[:, None] if s.ndim == 1 else np.repeat(s, GROUP, axis=1)[:, :cols]
    return np.asarray(q, dtype=np.float32)[:, :cols] * s


def scaled(total, sa, sb):
    """An exact sum as a float, times the smaller and then the larger of its two scales, in 32 bits."""
    x, y = np.broadcast_arrays(np.asarray(sa, np.float32), np.asarray(sb, np.float32))
    less = x < y
    return np.asarray(total, dtype=np.float32) * np.where(less, x, y) * np.where(less, y, x)


def product(a, sa, b, sb):
    """The product of whole numbers a (M, K) and b (N, K) with the scales of their rows."""
    return scaled(a @ b.T, sa[:, None], sb[None, :])


def fold(d, s):
    """A gradient times scales along its rows, in 32 bits."""
    return (np.asarray(d, np.float32) * np.asarray(s, np.float32)).astype(np.float64)


def backward(d, xq, sx, wq, sw):
    """(dX, dW) of the training step, both in 32 bits."""
    one = np.float32(1.0)
    dq, sd = whole(fold(d, sw[None, :]))
    dx = scaled(dq @ wq, sd[:, None], one)
    tq, st = whole(fold(d, sx[:, None]).T, LEVELS16)
    high = np.floor((tq + 128) / 256)
    low = tq - 256 * high
    # Each part's sum becomes a float; 256 times one plus the other is rounded once.
    parts = 256.0 * (high @ xq).astype(np.float32).astype(np.float64) + (low @ xq).astype(np.float32).astype(np.float64)
    return dx, scaled(parts, st[:, None], one)


def sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0, e) / (1.0 + e)


def gated(g, u):
    return g * sigmoid(g) * u


def gated_backward(d, g, u):
    """(dG, dU)."""
    p = sigmoid(g)
    return d * u * p * (1.0 + g * sigmoid(-g)), d * g * p
