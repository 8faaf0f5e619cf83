"""Weights beyond the largest float (codes from 2 on under scale byte 254, from 4
on under 253): the products take them as the numbers they are, so a result is
infinite only where it is itself too large, and zeros stay zeros.

Tolerances are those of the other 4-bit tests: n 2^-23 sum |a b| for a sum of n
exact products, half a step of the result's type.
"""
import numpy as np
import pytest
import torch

import fp32_sgemm_f32_amd as sg
from oracle import mx4 as ref
from test_gpu_mx4 import close, dev, host, normal, product_bound, random_mx4, typed, values  # noqa: F401

pytestmark = pytest.mark.gpu

# Tokens of every way through the thin product: folded, one, two and four tiles, two passes.
TOKENS = [1, 3, 5, 7, 13, 20, 50, 70]


def small(dtype):
    """Times a weight of 2^129, in every type's own range below."""
    return 2.0 ** -18 if dtype == torch.float16 else 2.0 ** -40


@typed
@pytest.mark.parametrize("s", [252, 253, 254])
def test_every_code(dev, dtype, s):  # noqa: F811
    codes = torch.zeros(16, 64, dtype=torch.uint8)
    codes[:, 0] = torch.arange(16) + 16 * 7         # column 0: every code; column 1: the largest, against zeros
    scales = torch.zeros(1, 32, 4, dtype=torch.uint8)
    scales[0, :16, 0] = s
    w = sg.Mx4(codes.to(dev), scales.to(dev), 16, 128)
    x = torch.zeros(4, 128, device=dev, dtype=dtype)
    x[0, 0], x[1, 0], x[2, 0] = small(dtype), -1.0, 1.5
    want = torch.from_numpy(host(x) @ values(w).T).float().to(dtype)     # one factor each: exact, or beyond the type's range
    assert torch.equal(sg.mx4_linear(x, w).cpu(), want)
    if dtype == torch.float32:
        q = sg.mx4_quantize(x)
        assert torch.equal(sg.mx4_gemm(q, w).cpu(), want)


@typed
@pytest.mark.parametrize("m", TOKENS)
@pytest.mark.parametrize("n, k", [(33, 130), (100, 1000), (40, 2100), (50, 5000)])
def test_linear(dev, dtype, m, n, k):  # noqa: F811
    rng = np.random.default_rng(m + k)
    w = random_mx4(rng, n, k, dev, 240, 255)
    x = normal(rng, m, k, dtype, dev, small(dtype))
    x[0] = 0.0
    X, W = host(x), values(w)
    got = sg.mx4_linear(x, w)
    close(got, X @ W.T, product_bound(X, W, 3), dtype)
    assert torch.equal(sg.mx4_linear(x, w), got)
    assert not got[0].any()


@typed
@pytest.mark.parametrize("m", [2, 13, 40])
def test_linear_keeps_the_other_rows(dev, dtype, m):  # noqa: F811
    """Rows without such a weight have the same bits beside rows with one."""
    rng = np.random.default_rng(m)
    n, k = 70, 2100
    x, w = normal(rng, m, k, dtype, dev, small(dtype)), random_mx4(rng, n, k, dev, 118, 130)
    alone = sg.mx4_linear(x, w)
    odd = [0, 17, 18, 69]
    w.scales[3, odd, 1], w.scales[16, odd, 1] = 254, 253
    w.codes[odd, 3 * 64 + 16] |= 7
    got = sg.mx4_linear(x, w)
    keep = [i for i in range(n) if i not in odd]
    assert torch.equal(got[:, keep], alone[:, keep])
    close(got, host(x) @ values(w).T, product_bound(host(x), values(w), 3), dtype)


@typed
@pytest.mark.parametrize("m", [3, 30])
def test_linear_infinite_and_nan_tokens(dev, dtype, m):  # noqa: F811
    rng = np.random.default_rng(15)
    x, w = normal(rng, m, 300, dtype, dev, small(dtype)), random_mx4(rng, 50, 300, dev, 240, 255)
    x[1, 7], x[2, 299] = float("nan"), float("inf")
    w.scales[0, 9, 2] = 255
    with np.errstate(invalid="ignore"):
        want = host(x) @ values(w).T
    got = host(sg.mx4_linear(x, w))
    assert np.array_equal(np.isnan(got), np.isnan(want))
    sure = np.isinf(want)
    assert np.array_equal(got[sure], want[sure])


def layer(rng, tokens, experts, hidden, inner, dtype, dev, std, up_scales, down_scales):  # noqa: F811
    x, router = normal(rng, tokens, hidden, dtype, dev, std), normal(rng, experts, hidden, dtype, dev)
    return (x, router, random_mx4(rng, experts * 2 * inner, hidden, dev, *up_scales),
            random_mx4(rng, experts * hidden, inner, dev, *down_scales))


# Few choices, folded and unfolded kernels; K in one piece and in several.
LAYERS = [(1, 8, 2), (3, 8, 6), (20, 4, 2)]


def check(x, router, up, down, top, dtype):
    e, h = router.shape
    f = down.shape[1]
    want, bound = ref.moe(host(x), host(router), values(up).reshape(e, 2 * f, h), values(down).reshape(e, h, f), top, True, 22)
    got = sg.mx4_moe(x, router, up, down, top)
    close(got, want, bound, dtype)
    assert torch.equal(sg.mx4_moe(x, router, up, down, top), got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("tokens, experts, top", LAYERS)
@pytest.mark.parametrize("hidden, inner", [(100, 40), (1100, 33), (4300, 20)])
def test_experts_up(dev, dtype, tokens, experts, top, hidden, inner):  # noqa: F811
    """Tokens so small that the inner activations are in range."""
    rng = np.random.default_rng(hidden)
    check(*layer(rng, tokens, experts, hidden, inner, dtype, dev, 2.0 ** -128 / hidden ** 0.5, (246, 255), (118, 122)), top, dtype)


@typed
@pytest.mark.parametrize("tokens, experts, top", LAYERS)
@pytest.mark.parametrize("hidden, inner", [(60, 40), (33, 900), (40, 2300)])
def test_experts_down(dev, dtype, tokens, experts, top, hidden, inner):  # noqa: F811
    """Inner activations near 2^-22."""
    rng = np.random.default_rng(inner)
    check(*layer(rng, tokens, experts, hidden, inner, dtype, dev, 2.0 ** -12 / hidden ** 0.5, (124, 128), (240, 255)), top, dtype)
