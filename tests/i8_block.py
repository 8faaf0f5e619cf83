"""The gated block of examples/eight_bit_block.py: the example itself, the same steps by the 64-bit reference of the
8-bit operators, and how near gradients in 8 bits have to lie to those in floats."""
import importlib.util
import os

import numpy as np
import torch

from oracle import i8 as ref

# How far a gradient may be off, as a part of its norm.  Rounding a row to 8 bits is off by max / (127 sqrt(12)) at the
# root of the mean square; for rows of 48 to 128 normal values the largest is up to 3.5 times their root mean square,
# for H and the gate's gradients, products of such, up to 5: 0.8 and 1.1%.  These are independent, so squares add up.
#   y: x and W                                          1.1%
#   H: G and U from y, each with a slope of up to 1.2   1.9%;   rounded itself: 2.2%
#   dH: dZ and D                                        1.1%
#   dGU: dH, G and U from y and to 8 bits once more     2.5%
#   dX: dGU (1.1%) and W                                2.9%    dW: dGU (16 bits) and X 2.6%    dD: H 2.2%
# and half a step of bf16, 0.2%, wherever a tensor is held in it.
NEAR = 0.05


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "eight_bit_block.py")
    spec = importlib.util.spec_from_file_location("eight_bit_block", path)
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)
    return block


def distances(got, want):
    """||got - want|| / ||want|| of each pair."""
    return [float((g.double() - w).norm() / w.norm()) for g, w in zip(got, want)]


def near(got, want):
    return [d <= NEAR for d in distances(got, want)]


def host(t):
    return t.double().numpy()


def bf16(v):
    return torch.from_numpy(np.asarray(v, np.float32)).bfloat16()


def eight_bit(params, x, dz, slope=True):
    """Gradients of x, [G; U] and D by the reference's steps, tensors between them in bf16.  slope=False leaves the
    factor 1 + g (1 - p) out."""
    w, d = (host(p) for p in params)
    (xq, sx), (wq, sw), (dq, sd) = ref.whole(host(x)), ref.whole(w), ref.whole(d)
    y = host(bf16(ref.product(xq, sx, wq, sw)))
    f = y.shape[1] // 2
    h = host(bf16(ref.gated(y[:, :f], y[:, f:])))
    hq, sh = ref.whole(h)
    dh, dd = ref.backward(host(dz), hq, sh, dq, sd)
    dh = host(bf16(dh))
    g, u = (ref.values(*ref.grouped(v), f).astype(np.float64) for v in (y[:, :f], y[:, f:]))
    dg, du = ref.gated_backward(dh, g, u)
    if not slope:
        dg = dh * u * ref.sigmoid(g)
    dx, dw = ref.backward(host(bf16(np.concatenate((dg, du), 1))), xq, sx, wq, sw)
    return bf16(dx), torch.from_numpy(dw), torch.from_numpy(dd)
