"""The expert layer's inner activations keep 24 bits for every type of the
tokens: the operator rounds its result once, and nothing on the way there.

Inputs on which only that rounding can show: a token's gates are equal for all
inner rows of an expert, the other factors u are whole numbers near 8192, and a
row of `down` subtracts two activations from each other, so that a result is
silu(g) (u_1 - u_2), a thousandth of either activation.
"""
import numpy as np
import pytest
import torch

import fp32_sgemm_f32_amd as sg
from test_gpu_mx4 import close, dev, host, typed, values  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def case(rng, tokens, experts, inner, hidden, dtype, dev):
    """(x, router, up, down) as above: u = 8192 + k x_1 with k a level of the format."""
    x = np.zeros((tokens, hidden))
    x[:, 0], x[:, 1], x[:, 2] = 4096.0, 1 + np.arange(tokens) % 3, 1.0
    x[:, 3:] = rng.integers(-2, 3, (tokens, hidden - 3))
    up = np.zeros((experts, 2 * inner, hidden))
    up[:, :inner, 2] = rng.choice([0.5, 1.0, 1.5, 3.0], (experts, 1))
    up[:, inner:, 0] = 2.0
    up[:, inner:, 1] = rng.choice([0.0, 0.5, 1.0, 1.5, 2.0, 3.0], (experts, inner))
    down = np.zeros((experts, hidden, inner))
    for e in range(experts):
        for h in range(hidden):
            f = rng.choice(inner, 2, replace=False)
            down[e, h, f] = 1.0, -1.0
    router = rng.standard_normal((experts, hidden)) / 64
    router[:, :3] = 0.0
    t = lambda v: torch.from_numpy(v).float().to(dev)
    qu, qd = sg.mx4_quantize(t(up.reshape(-1, hidden))), sg.mx4_quantize(t(down.reshape(-1, inner)))
    assert np.array_equal(values(qu), up.reshape(-1, hidden)) and np.array_equal(values(qd), down.reshape(-1, inner))
    return t(x).to(dtype), t(router).to(dtype), qu, qd


def want(x, router, up, down, top):
    """(y, bound): g and u are exact whole and half numbers in any order of fp32 sums.  What is left: silu (16 steps of
    fp32, the same for all activations of an expert), the rounding of an activation (half a step each), a sum of six
    pieces, the weight (an exponential, a sum of `top`, a quotient: 40 + top steps), the sum over experts."""
    y, bound = np.zeros_like(x), np.zeros_like(x)
    logits = x @ router.T
    inner = down.shape[2]
    for t in range(x.shape[0]):
        order = sorted(range(len(router)), key=lambda e: (-logits[t, e], e))[:top]
        p = np.exp(logits[t, order] - logits[t, order[0]])
        p /= p.sum()
        for e, w in zip(order, p):
            z = up[e] @ x[t]
            g, u = z[:inner], z[inner:]
            act = g / (1 + np.exp(-g)) * u
            part, size = down[e] @ act, np.abs(down[e]) @ np.abs(act)
            y[t] += w * part
            bound[t] += w * (size * (6 + 0.5) * U + np.abs(part) * (16 + 40 + 2 * top) * U)
    return y, bound


# Few choices; more of them with few tokens (folded), and with many; short and long inner rows.
@typed
@pytest.mark.parametrize("tokens, top", [(1, 4), (2, 8), (3, 8), (5, 4), (8, 4), (20, 4), (64, 2)])
@pytest.mark.parametrize("inner", [40, 300, 1100])
def test_activations_keep_24_bits(dev, dtype, tokens, top, inner):  # noqa: F811
    rng = np.random.default_rng(tokens + inner)
    experts, hidden = 8, 48
    x, router, up, down = case(rng, tokens, experts, inner, hidden, dtype, dev)
    y, bound = want(host(x), host(router), values(up).reshape(experts, 2 * inner, hidden),
                    values(down).reshape(experts, hidden, inner), top)
    close(sg.mx4_moe(x, router, up, down, top), y, bound, dtype)
