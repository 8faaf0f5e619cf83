"""The 4-bit operators on the GPU against their definitions in 64 bits.

Tolerances.  Quantisation and dequantisation are exact.  A product of n
exactly representable factors, summed in fp32 in any order and cutting or
rounding, is off by at most n 2^-23 sum |a b|; the store to a 16-bit type adds
half a step (eps / 2 relative, or half the least subnormal).
"""
import numpy as np
import pytest
import torch

import fp32_sgemm_f32_amd as sg
from oracle import mx4 as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
IDS = ["fp32", "bf16", "fp16"]
typed = pytest.mark.parametrize("dtype", TYPES, ids=IDS)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    sg.library()
    return torch.device("cuda:0")


def host(t):
    return t.detach().cpu().double().numpy()


def normal(rng, rows, cols, dtype, dev, std=1.0):
    x = rng.standard_normal((rows, cols)) * std
    big = rng.random(cols) < 0.02
    return torch.from_numpy(np.where(big, 12.0, 1.0) * x).to(dtype).to(dev)


def strided(t, pad, shift):
    """t in rows that are `pad` elements longer, starting `shift` elements into the allocation."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + shift,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[shift:].view(rows, cols + pad)[:, :cols]
    v.copy_(t)
    return v


def random_mx4(rng, rows, cols, dev, lo=118, hi=130):
    """An Mx4 of random codes and scales, zeros in the padding."""
    cs, ss = ref.shapes(rows, cols)
    c = rng.integers(0, 16, (rows, 2 * cs[1]), dtype=np.uint8)
    c[:, cols:] = 0
    s = np.zeros(ss, dtype=np.uint8)
    blocks = -(-cols // 32)
    word = np.zeros((rows, ss[0] * 4), dtype=np.uint8)
    word[:, :blocks] = rng.integers(lo, hi, (rows, blocks))
    s[:, :rows] = word.reshape(rows, ss[0], 4).transpose(1, 0, 2)
    codes = c[:, 0::2] | c[:, 1::2] << 4
    return sg.Mx4(torch.from_numpy(codes).to(dev), torch.from_numpy(s).to(dev), rows, cols)


def values(q):
    return ref.values(q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.shape[1])


def step(y, dtype):
    """Half a step of dtype at y."""
    f = torch.finfo(dtype)
    return np.maximum(np.abs(y) * (f.eps / 2), f.smallest_normal * f.eps / 2)


def close(got, want, bound, dtype=torch.float32):
    """got within bound of want, plus its type's own rounding (of either side of the bound)."""
    got = host(got)
    lim = bound + step(np.abs(want) + bound, dtype)
    # Beyond the type's largest value plus half its step a result rounds to infinity.
    f = torch.finfo(dtype)
    edge = f.max * (1 + f.eps / 4)
    with np.errstate(invalid="ignore"):
        right = np.abs(got - want) <= lim
    right |= (got == np.copysign(np.inf, want)) & (np.abs(want) + bound >= edge)
    bad = ~right
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
        f"{got[bad][0]} against {want[bad][0]}, allowed {lim[bad][0]}"


def product_bound(a, b, pieces=1):
    """Bound of an fp32 sum for a @ b.T (`pieces` addends per factor)."""
    return pieces * a.shape[1] * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T) + 2.0 ** -149


# ---- quantisation -----------------------------------------------------------------------------------------------

SHAPES = [(1, 1), (1, 32), (3, 31), (7, 33), (16, 128), (33, 129), (5, 260), (130, 255), (257, 96), (1, 5000), (200, 1)]


def check_quantized(q, x, noclip=False):
    codes, scales = ref.quantize(x, noclip)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)


@typed
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("rule", ["floor", "noclip"])
def test_quantize(dev, dtype, shape, rule):
    x = normal(np.random.default_rng(shape[0]), *shape, dtype, dev)
    noclip = rule == "noclip"
    check_quantized(sg.mx4_quantize(x, rule=rule), host(x), noclip)
    check_quantized(sg.mx4_quantize(x.t(), rule=rule), host(x).T, noclip)
    q, qt = sg.mx4_quantize_both(x, rule=rule)
    check_quantized(q, host(x), noclip)
    check_quantized(qt, host(x).T, noclip)


@typed
@pytest.mark.parametrize("pad, shift", [(0, 1), (1, 0), (8, 8), (3, 5), (4, 0)])
def test_quantize_strided(dev, dtype, pad, shift):
    x = strided(normal(np.random.default_rng(1), 37, 200, dtype, dev), pad, shift)
    q, qt = sg.mx4_quantize_both(x)
    check_quantized(q, host(x))
    check_quantized(qt, host(x).T)
    check_quantized(sg.mx4_quantize(x), host(x))
    qt, q = sg.mx4_quantize_both(x.t())      # a column-major view
    check_quantized(q, host(x))
    check_quantized(qt, host(x).T)


def borders():
    """For every scale byte a block holding its largest magnitudes, every code border, and the floats next to them."""
    rows = []
    edges = np.array([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0], dtype=np.float32)
    for s in range(-127, 126):
        for top in (4.0, 6.0, np.nextafter(np.float32(6), np.float32(9)), 7.0, np.nextafter(np.float32(8), np.float32(0))):
            with np.errstate(over="ignore", under="ignore"):
                v = np.ldexp(edges, s).astype(np.float32)
                t = np.ldexp(np.float32(top), s).astype(np.float32)
            if not np.isfinite(t):
                continue
            near = [v, np.nextafter(v, np.float32(np.inf)), -np.nextafter(v[1:], np.float32(-1))]
            w = np.concatenate(near)[:31]
            rows.append(np.concatenate([w, np.zeros(31 - len(w), np.float32), [t]]))
            w = -np.nextafter(v, np.float32(-1))
            rows.append(np.concatenate([w, np.zeros(31 - len(w), np.float32), [-t]]))
    return np.array(rows, dtype=np.float32)


@pytest.mark.parametrize("rule", ["floor", "noclip"])
def test_quantize_at_every_border_and_scale(dev, rule):
    x = torch.from_numpy(borders()).to(dev)
    check_quantized(sg.mx4_quantize(x, rule=rule), host(x), rule == "noclip")
    check_quantized(sg.mx4_quantize_both(x.t().contiguous(), rule=rule)[1], host(x), rule == "noclip")


@pytest.mark.parametrize("dtype", TYPES[1:], ids=IDS[1:])
def test_quantize_every_16_bit_value(dev, dtype):
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype).view(-1, 64).to(dev)
    check_quantized(sg.mx4_quantize(x), host(x))


def test_quantize_zeros_subnormals_nan_infinity(dev):
    x = torch.zeros(6, 64)
    x[1, :32] = 1e-45
    x[2, 5], x[2, 40] = float("nan"), 1.0
    x[3, 0], x[3, 33] = float("inf"), -2.0
    x[4] = -0.0
    x[5, :32] = torch.finfo(torch.float32).max
    for q in (sg.mx4_quantize(x.to(dev)), sg.mx4_quantize_both(x.to(dev))[0], sg.mx4_quantize(x.t().contiguous().to(dev).t())):
        check_quantized(q, x.double().numpy())


@typed
@pytest.mark.parametrize("shape", SHAPES + [(70, 513), (9, 1027)], ids=str)
def test_dequantize(dev, dtype, shape):
    q = random_mx4(np.random.default_rng(3), *shape, dev)
    want = torch.from_numpy(values(q)).to(dtype)
    assert torch.equal(sg.mx4_dequantize(q, dtype=dtype).cpu(), want)
    for pad, shift in ((0, 1), (1, 0), (5, 3), (8, 0)):
        out = strided(torch.zeros(shape, dtype=dtype, device=dev), pad, shift)
        whole = out._base
        whole.fill_(7.0)
        assert sg.mx4_dequantize(q, out=out) is out
        assert torch.equal(out.cpu(), want)
        assert int((whole != 7.0).sum()) <= int((want != 7.0).sum()), "written beside the matrix"


@typed
def test_dequantize_every_code_and_scale(dev, dtype):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)          # 256 rows x 512 columns: every byte, twice a block
    scales = torch.zeros(4, 256, 4, dtype=torch.uint8)
    scales[:] = torch.arange(256, dtype=torch.uint8).view(1, 256, 1)
    q = sg.Mx4(codes.to(dev), scales.to(dev), 256, 512)
    want = torch.from_numpy(values(q))
    if dtype == torch.float32:
        want = want.float().double()         # beyond the largest float: infinite
    want = want.to(dtype)
    got = sg.mx4_dequantize(q, dtype=dtype).cpu()
    assert torch.equal(torch.nan_to_num(got, nan=3.0, posinf=None), torch.nan_to_num(want, nan=3.0, posinf=None))
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())


# ---- the product ------------------------------------------------------------------------------------------------

GEMMS = [(1, 1, 1), (1, 17, 32), (33, 1, 31), (31, 65, 127), (64, 64, 128), (65, 63, 129), (100, 300, 257), (257, 255, 640),
         (130, 520, 1000), (1111, 500, 333), (1, 2000, 4096), (3000, 5, 100), (2100, 2050, 384), (4097, 4200, 65), (4200, 4097, 130), (4096, 4096, 128)]


@typed
@pytest.mark.parametrize("m, n, k", GEMMS)
def test_gemm(dev, dtype, m, n, k):
    rng = np.random.default_rng(m + n + k)
    a, b = random_mx4(rng, m, k, dev), random_mx4(rng, n, k, dev)
    A, B = values(a), values(b)
    close(sg.mx4_gemm(a, b, dtype=dtype), A @ B.T, product_bound(A, B), dtype)


@typed
@pytest.mark.parametrize("m, n, k", [(33, 70, 300), (300, 290, 256), (2100, 2050, 128)])
@pytest.mark.parametrize("alpha, beta", [(1.0, 1.0), (-0.5, 2.0), (0.0, 3.0), (2.0, 0.0)])
def test_gemm_adds_to_a_strided_result(dev, dtype, m, n, k, alpha, beta):
    rng = np.random.default_rng(k)
    a, b = random_mx4(rng, m, k, dev), random_mx4(rng, n, k, dev)
    A, B = values(a), values(b)
    for pad, shift in ((3, 1), (8, 8)):
        c = strided(normal(rng, m, n, dtype, dev), pad, shift)
        C = host(c)
        edge = c._base.clone()
        if beta == 0.0:
            c.fill_(float("nan"))
        assert sg.mx4_gemm(a, b, out=c, alpha=alpha, beta=beta) is c
        want = alpha * (A @ B.T) + beta * C
        bound = abs(alpha) * product_bound(A, B) + 2.0 ** -22 * (np.abs(alpha * (A @ B.T)) + np.abs(beta * C))
        close(c, want, bound, dtype)
        c.fill_(float("nan"))
        whole = c._base
        assert torch.equal(torch.isnan(whole), torch.isnan(whole) | torch.isnan(edge)), "written beside the matrix"


def test_gemm_of_nothing(dev):
    rng = np.random.default_rng(5)
    c = normal(rng, 5, 7, torch.float32, dev)
    C = c.clone()
    a, b = random_mx4(rng, 5, 0, dev), random_mx4(rng, 7, 0, dev)
    assert torch.equal(sg.mx4_gemm(a, b), torch.zeros(5, 7, device=dev))
    assert torch.equal(sg.mx4_gemm(a, b, out=c, alpha=float("inf"), beta=2.0), 2.0 * C)
    assert sg.mx4_gemm(random_mx4(rng, 0, 64, dev), random_mx4(rng, 7, 64, dev)).shape == (0, 7)
    # alpha == 0: A and B are not read, a NaN in them does not show
    a, b = random_mx4(rng, 5, 64, dev, 255, 256), random_mx4(rng, 7, 64, dev)
    assert torch.equal(sg.mx4_gemm(a, b, out=c, alpha=0.0, beta=0.5), C)


@pytest.mark.parametrize("m, n, k", [(70, 90, 256), (300, 300, 384), (2100, 2050, 256)])
def test_gemm_is_exact_on_whole_numbers_and_repeats(dev, m, n, k):
    rng = np.random.default_rng(6)
    a, b = random_mx4(rng, m, k, dev, 128, 130), random_mx4(rng, n, k, dev, 128, 130)   # 2 or 4 times 0 .. 6 by halves: whole
    A, B = values(a), values(b)
    first = sg.mx4_gemm(a, b)
    assert np.array_equal(host(first), A @ B.T)
    assert all(torch.equal(sg.mx4_gemm(a, b), first) for _ in range(3))


@pytest.mark.parametrize("m, n, k", [(40, 50, 300), (300, 300, 256)])
def test_gemm_keeps_nan_blocks_to_their_rows(dev, m, n, k):
    rng = np.random.default_rng(7)
    a, b = random_mx4(rng, m, k, dev), random_mx4(rng, n, k, dev)
    a.scales[1, 17, 3 if k >= 256 else 1] = 255
    b.scales[0, 33, 0] = 255
    nan = torch.isnan(sg.mx4_gemm(a, b)).cpu()
    want = torch.zeros(m, n, dtype=torch.bool)
    want[17], want[:, 33] = True, True
    assert torch.equal(nan, want)


def test_gemm_extreme_scales(dev):
    """Scales whose product is in range though each is far from 1."""
    rng = np.random.default_rng(8)
    a, b = random_mx4(rng, 64, 128, dev, 250, 251), random_mx4(rng, 64, 128, dev, 1, 2)
    A, B = values(a), values(b)
    close(sg.mx4_gemm(a, b), A @ B.T, product_bound(A, B))


@typed
def test_gemm_every_pair_of_scales(dev, dtype):
    """Row r of A holds 1 under scale byte r, row c of B the same under c: 2^(r + c - 254), or what it rounds to."""
    codes = torch.zeros(255, 64, dtype=torch.uint8)
    codes[:, 8] = 2
    scales = torch.zeros(1, 256, 4, dtype=torch.uint8)
    scales[0, :255, 0] = torch.arange(255)
    a = sg.Mx4(codes.to(dev), scales.to(dev), 255, 40)
    e = np.add.outer(np.arange(255), np.arange(255)) - 254
    want = torch.from_numpy(np.ldexp(1.0, e)).float().to(dtype)
    got = sg.mx4_gemm(a, a, dtype=dtype).cpu()
    assert torch.equal(got, want), (got != want).nonzero()[:5]


def test_quantised_product_against_floats(dev):
    x, w = (normal(np.random.default_rng(s), 200, 500, torch.float32, dev) for s in (9, 10))
    A, B = ref.rounded(host(x)), ref.rounded(host(w))
    close(sg.mx4_gemm(sg.mx4_quantize(x), sg.mx4_quantize(w)), A @ B.T, product_bound(A, B))


# ---- the training step ------------------------------------------------------------------------------------------

@typed
@pytest.mark.parametrize("m, n, k", [(1, 1, 1), (33, 70, 100), (130, 257, 64), (333, 40, 513), (1030, 1025, 300)])
def test_train(dev, dtype, m, n, k):
    rng = np.random.default_rng(11)
    x, w, dy = normal(rng, m, k, dtype, dev), normal(rng, n, k, dtype, dev, 0.1), normal(rng, m, n, dtype, dev, 0.01)
    y, saved = sg.mx4_train_forward(x, w)
    dx, dw = sg.mx4_train_backward(dy, saved)
    assert y.dtype == dtype and dx.dtype == dtype and dw.dtype == torch.float32
    X, W, D = host(x), host(w), host(dy)
    r = ref.rounded
    for got, a, b, t in ((y, r(X), r(W), dtype), (dx, r(D), r(W.T), dtype), (dw, r(D.T), r(X.T), torch.float32)):
        close(got, a @ b.T, product_bound(a, b), t)
    # A gradient given is added to.
    start = normal(rng, n, k, torch.float32, dev)
    both = start.clone()
    _, same = sg.mx4_train_backward(dy, saved, dW=both)
    assert same is both
    close(both, host(start) + r(D.T) @ r(X.T).T, product_bound(r(D.T), r(X.T)) + 2.0 ** -22 * (np.abs(host(start)) + np.abs(host(dw))))


@typed
@pytest.mark.parametrize("m, n, k", [(300, 520, 700), (2100, 2050, 2060), (2048, 4096, 1000), (4096, 4100, 4090), (4096, 4096, 4100),
                                     (250, 254, 65500)])
def test_train_equals_its_parts(dev, dtype, m, n, k):
    """The calls of a training step give bit for bit what quantising and multiplying one after the other gives, for all tiles
    and for products in one launch and in two."""
    rng = np.random.default_rng(31)
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(rng.integers(1 << 30)))
    x, w, dy = (torch.randn(s, generator=gen, device=dev).to(dtype) for s in ((m, k), (n, k), (m, n)))
    y, saved = sg.mx4_train_forward(x, w)
    start = torch.randn(n, k, generator=gen, device=dev)
    dw = start.clone()
    dx, _ = sg.mx4_train_backward(dy, saved, dW=dw)
    quant = sg.mx4_quantize
    assert torch.equal(y, sg.mx4_gemm(quant(x), quant(w), dtype=dtype))
    assert torch.equal(dx, sg.mx4_gemm(quant(dy), quant(w.t()), dtype=dtype))
    assert torch.equal(dw, sg.mx4_gemm(quant(dy.t()), quant(x.t()), out=start, beta=1.0))


def test_train_of_two_types_and_of_views(dev):
    """X and W of different types, column-major, strided: the same results as of the plain copies."""
    rng = np.random.default_rng(29)
    m, n, k = 70, 90, 200
    x, w, dy = normal(rng, m, k, torch.bfloat16, dev), normal(rng, n, k, torch.float32, dev), normal(rng, m, n, torch.bfloat16, dev)
    y, saved = sg.mx4_train_forward(x, w)
    want = (y, *sg.mx4_train_backward(dy, saved))
    close(y, ref.rounded(host(x)) @ ref.rounded(host(w)).T, product_bound(ref.rounded(host(x)), ref.rounded(host(w))), torch.bfloat16)
    columns = lambda t: t.t().contiguous().t()
    for a, b, d in ((columns(x), w, dy), (x, columns(w), columns(dy)), (strided(x, 3, 1), strided(w, 1, 0), strided(dy, 5, 2))):
        y, saved = sg.mx4_train_forward(a, b)
        for got, exp in zip((y, *sg.mx4_train_backward(d, saved)), want):
            assert torch.equal(got, exp)


@pytest.mark.parametrize("m, n, k", [(0, 5, 7), (5, 0, 7), (5, 7, 0), (0, 0, 0)])
def test_train_of_nothing(dev, m, n, k):
    x, w, dy = (torch.ones(s, device=dev) for s in ((m, k), (n, k), (m, n)))
    y, saved = sg.mx4_train_forward(x, w)
    dw = torch.ones(n, k, device=dev)
    dx, same = sg.mx4_train_backward(dy, saved, dW=dw)
    assert torch.equal(y, torch.zeros(m, n, device=dev)) and torch.equal(dx, torch.zeros(m, k, device=dev))
    assert same is dw and torch.equal(dw, torch.ones(n, k, device=dev))
    assert torch.equal(sg.mx4_train_backward(dy, saved)[1], torch.zeros(n, k, device=dev))


def test_train_refuses_what_does_not_fit(dev):
    x, w = torch.zeros(4, 64, device=dev), torch.zeros(6, 64, device=dev)
    y, saved = sg.mx4_train_forward(x, w)
    for call, kind in ((lambda: sg.mx4_train_forward(x, w[:, :32]), ValueError), (lambda: sg.mx4_train_forward(x, w.double()), TypeError),
                       (lambda: sg.mx4_train_forward(x, w, rule="up"), ValueError),
                       (lambda: sg.mx4_train_backward(y[:3], saved), ValueError), (lambda: sg.mx4_train_backward(x, saved), ValueError),
                       (lambda: sg.mx4_train_backward(y, saved, dW=w.bfloat16()), ValueError),
                       (lambda: sg.mx4_train_backward(y, saved, dW=w[:5]), ValueError)):
        with pytest.raises(kind):
            call()


def test_train_gradient_against_differences(dev):
    """On values that 4 bits hold exactly, before and after a step, the layer is bilinear: central differences of
    sum(dY * Y) are its gradient, exactly, up to the sums' fp32."""
    rng = np.random.default_rng(12)
    m, n, k = 40, 36, 70
    two_three = lambda *s: rng.choice([2.0, 3.0, -2.0, -3.0], s)
    X, W, D = two_three(m, k), two_three(n, k), two_three(m, n)
    t = lambda v: torch.from_numpy(v).float().to(dev)
    f = lambda X, W: float((host(sg.mx4_train_forward(t(X), t(W))[0]) * D).sum())
    _, saved = sg.mx4_train_forward(t(X), t(W))
    dx, dw = sg.mx4_train_backward(t(D), saved)
    for _ in range(5):
        v, u = rng.choice([-1.0, 0.0, 1.0], (m, k)), rng.choice([-1.0, 0.0, 1.0], (n, k))
        assert (f(X + v, W) - f(X - v, W)) / 2 == (host(dx) * v).sum()
        assert (f(X, W + u) - f(X, W - u)) / 2 == (host(dw) * u).sum()


# ---- the thin product -------------------------------------------------------------------------------------------

LINEARS = [(1, 1, 1), (1, 16, 128), (1, 100, 4096), (2, 33, 31), (7, 15, 130), (13, 501, 1640), (16, 64, 640), (17, 200, 100),
           (33, 48, 1000), (64, 130, 2050), (65, 70, 300), (130, 20, 129), (5, 3000, 96), (16, 40, 9000), (1, 5, 16400),
           (48, 30, 5001)]


@typed
@pytest.mark.parametrize("m, n, k", LINEARS)
def test_linear(dev, dtype, m, n, k):
    rng = np.random.default_rng(m * n + k)
    x, w = normal(rng, m, k, dtype, dev), random_mx4(rng, n, k, dev)
    X, W = host(x), values(w)
    first = sg.mx4_linear(x, w)
    close(first, X @ W.T, product_bound(X, W, 3), dtype)
    assert torch.equal(sg.mx4_linear(x, w), first)


@typed
@pytest.mark.parametrize("m", [1, 3, 20, 50])
@pytest.mark.parametrize("pad, shift", [(1, 0), (0, 1), (8, 0), (2, 6)])
def test_linear_strided(dev, dtype, m, pad, shift):
    rng = np.random.default_rng(13)
    n, k = 75, 333
    x, w = strided(normal(rng, m, k, dtype, dev), pad, shift), random_mx4(rng, n, k, dev)
    out = strided(torch.zeros(m, n, dtype=dtype, device=dev), pad, shift)
    edge = out._base.clone()
    assert sg.mx4_linear(x, w, out=out) is out
    X, W = host(x), values(w)
    close(out, X @ W.T, product_bound(X, W, 3), dtype)
    out.fill_(float("nan"))
    assert torch.equal(torch.isnan(out._base), torch.isnan(edge) | torch.isnan(out._base))


@typed
def test_linear_whole_type_range(dev, dtype):
    """Token values from the least subnormal to the largest: each piece of the split is exact."""
    rng = np.random.default_rng(14)
    f = torch.finfo(dtype)
    lo = int(np.log2(f.smallest_normal)) - (0 if dtype == torch.bfloat16 else 8)
    k = 256
    x = torch.from_numpy(rng.standard_normal((20, k)) * np.ldexp(1.0, rng.integers(lo, 10, (20, 1)))).to(dtype).to(dev)
    w = random_mx4(rng, 40, k, dev, 127, 129)
    X, W = host(x), values(w)
    close(sg.mx4_linear(x, w), X @ W.T, product_bound(X, W, 3), dtype)


@typed
@pytest.mark.parametrize("m", [3, 30])
def test_linear_nan_and_infinity_stay_in_their_rows(dev, dtype, m):
    rng = np.random.default_rng(15)
    x, w = normal(rng, m, 300, dtype, dev), random_mx4(rng, 50, 300, dev)
    x[1, 7], x[2, 299] = float("nan"), float("inf")
    w.scales[0, 9, 2] = 255
    with np.errstate(invalid="ignore"):
        want = host(x) @ values(w).T
    got = host(sg.mx4_linear(x, w))
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want))


def test_linear_of_nothing(dev):
    rng = np.random.default_rng(16)
    assert torch.equal(sg.mx4_linear(torch.empty(3, 0, device=dev), random_mx4(rng, 5, 0, dev)), torch.zeros(3, 5, device=dev))
    assert sg.mx4_linear(torch.empty(0, 64, device=dev), random_mx4(rng, 5, 64, dev)).shape == (0, 5)


# ---- the expert layer -------------------------------------------------------------------------------------------

def moe_case(rng, t, e, h, f, dtype, dev):
    x, router = normal(rng, t, h, dtype, dev, 0.5), normal(rng, e, h, dtype, dev, 1 / np.sqrt(h))
    up = sg.mx4_quantize(torch.from_numpy(rng.standard_normal((e * 2 * f, h)) / np.sqrt(h)).float().to(dev))
    down = sg.mx4_quantize(torch.from_numpy(rng.standard_normal((e * h, f)) / np.sqrt(f)).float().to(dev))
    return x, router, up, down


def moe_want(x, router, up, down, top, norm, dtype):
    e, h = router.shape
    f = down.shape[1]
    bits = 22 if dtype == torch.float32 else 15
    return ref.moe(host(x), host(router), values(up).reshape(e, 2 * f, h), values(down).reshape(e, h, f), top, norm, bits)


MOES = [(1, 1, 1, 1, 1), (1, 4, 128, 32, 2), (1, 8, 256, 96, 8), (2, 8, 100, 33, 3), (5, 16, 130, 64, 4), (16, 8, 257, 129, 2),
        (17, 6, 64, 200, 6), (33, 60, 96, 40, 4), (48, 16, 128, 160, 8), (64, 5, 72, 48, 1), (64, 128, 64, 32, 16), (3, 300, 40, 16, 5),
        (1, 1024, 33, 16, 16), (1, 16, 1200, 520, 3), (4, 8, 640, 1100, 2),
        (3, 4, 4200, 40, 4), (20, 4, 4200, 70, 2), (1, 4, 2200, 100, 2), (33, 3, 2200, 150, 2), (2, 3, 100, 3400, 2), (18, 2, 80, 3400, 2),
        (17, 3, 900, 900, 2), (40, 4, 1500, 300, 3), (30, 2, 2700, 450, 1)]


@typed
@pytest.mark.parametrize("t, e, h, f, top", MOES)
@pytest.mark.parametrize("norm", [True, False])
def test_moe(dev, dtype, t, e, h, f, top, norm):
    rng = np.random.default_rng(t + e + h)
    x, router, up, down = moe_case(rng, t, e, h, f, dtype, dev)
    want, bound = moe_want(x, router, up, down, top, norm, dtype)
    first = sg.mx4_moe(x, router, up, down, top, norm=norm)
    close(first, want, bound, dtype)
    assert torch.equal(sg.mx4_moe(x, router, up, down, top, norm=norm), first)


@typed
@pytest.mark.parametrize("t", [1, 9, 40])
def test_moe_equal_logits_take_the_lower_expert(dev, dtype, t):
    rng = np.random.default_rng(17)
    x, router, up, down = moe_case(rng, t, 12, 64, 32, dtype, dev)
    router[4:] = router[:4].repeat(2, 1)     # every logit three times
    want, bound = moe_want(x, router, up, down, 5, True, dtype)
    close(sg.mx4_moe(x, router, up, down, 5), want, bound, dtype)
    router.zero_()                           # all equal: the first `top`
    want, bound = moe_want(x, router, up, down, 3, False, dtype)
    close(sg.mx4_moe(x, router, up, down, 3, norm=False), want, bound, dtype)


@typed
@pytest.mark.parametrize("t", [1, 6, 20])
def test_moe_strided(dev, dtype, t):
    rng = np.random.default_rng(18)
    x, router, up, down = moe_case(rng, t, 9, 150, 70, dtype, dev)
    want, bound = moe_want(x, router, up, down, 3, True, dtype)
    for pad, shift in ((1, 0), (0, 1), (10, 3)):
        out = strided(torch.zeros(t, 150, dtype=dtype, device=dev), pad, shift)
        got = sg.mx4_moe(strided(x, pad, shift), strided(router, pad, shift), up, down, 3, out=out)
        assert got is out
        close(out, want, bound, dtype)


@pytest.mark.parametrize("t", [3, 24])
def test_moe_nan_token_stays_alone(dev, t):
    rng = np.random.default_rng(19)
    x, router, up, down = moe_case(rng, t, 8, 128, 64, torch.bfloat16, dev)
    clean = sg.mx4_moe(x, router, up, down, 2)
    assert sg.mx4_moe(x[:0], router, up, down, 2).shape == (0, 128)
    x[1, 5] = float("nan")
    got = sg.mx4_moe(x, router, up, down, 2)
    assert bool(got[1].isnan().all())
    keep = [i for i in range(t) if i != 1]
    assert torch.equal(got[keep], clean[keep])


def test_moe_refuses_what_does_not_fit(dev):
    rng = np.random.default_rng(20)
    x, router, up, down = moe_case(rng, 2, 4, 64, 32, torch.float32, dev)
    for args, kind in (((x, router.bfloat16(), up, down, 1), TypeError), ((x, router[:3], up, down, 1), ValueError),
                       ((x, router, down, up, 1), ValueError), ((x, router, up, down, 5), sg.SgemmError),
                       ((x, router, up, down, 0), sg.SgemmError), ((x.repeat(40, 1), router, up, down, 1), sg.SgemmError),
                       ((x.double(), router, up, down, 1), TypeError), ((x[0], router, up, down, 1), ValueError)):
        with pytest.raises(kind):
            sg.mx4_moe(*args)
    with pytest.raises(sg.SgemmError) as e:
        sg.mx4_moe(x, router, up, down, 1, out=x)
    assert e.value.status == sg.ERR_ALIAS
    with pytest.raises(ValueError):
        sg.mx4_moe(x, router, up, down, 1, out=torch.empty(2, 63, device=dev))


def test_python_refuses_what_does_not_fit(dev):
    rng = np.random.default_rng(21)
    a, b = random_mx4(rng, 4, 64, dev), random_mx4(rng, 4, 96, dev)
    x = torch.zeros(4, 64, device=dev)
    for call, kind in ((lambda: sg.mx4_gemm(a, b), ValueError), (lambda: sg.mx4_gemm(a, a, beta=1.0), ValueError),
                       (lambda: sg.mx4_gemm(a, a, out=x), ValueError), (lambda: sg.mx4_linear(x, b), ValueError),
                       (lambda: sg.mx4_linear(x.double(), a), TypeError), (lambda: sg.mx4_linear(x.t(), a), ValueError),
                       (lambda: sg.mx4_quantize(x[0]), ValueError), (lambda: sg.mx4_quantize(x[:, ::2]), ValueError),
                       (lambda: sg.mx4_quantize(x.int()), TypeError), (lambda: sg.mx4_dequantize(a, out=x[:3]), ValueError),
                       (lambda: sg.mx4_gemm(a, a, dtype=torch.float64), TypeError)):
        with pytest.raises(kind):
            call()


# ---- streams, graphs, large matrices ----------------------------------------------------------------------------

def whole_path(x, w, dy, router, up, down):
    """Every operator once."""
    y, saved = sg.mx4_train_forward(x, w)
    dx, dw = sg.mx4_train_backward(dy, saved)
    q = sg.mx4_quantize(w)
    z = sg.mx4_linear(x, q)
    return y, dx, dw, z, sg.mx4_dequantize(q, dtype=x.dtype), sg.mx4_moe(x, router, up, down, 2)


def path_inputs(dev, seed):
    rng = np.random.default_rng(seed)
    x, router, up, down = moe_case(rng, 20, 8, 200, 64, torch.bfloat16, dev)
    return x, normal(rng, 150, 200, torch.bfloat16, dev), normal(rng, 20, 150, torch.bfloat16, dev), router, up, down


def test_on_another_stream(dev):
    args = path_inputs(dev, 22)
    want = whole_path(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x, w, _, router, up, down = args
    got_y, saved = sg.mx4_train_forward(x, w, stream=s)
    got = (got_y, *sg.mx4_train_backward(args[2], saved, stream=s), sg.mx4_linear(x, sg.mx4_quantize(w, stream=s), stream=s),
           sg.mx4_dequantize(sg.mx4_quantize(w, stream=s), dtype=x.dtype, stream=s),
           sg.mx4_moe(x, router, up, down, 2, stream=s))
    with torch.cuda.stream(s):
        inside = whole_path(*args)
    s.synchronize()
    for a, b, c in zip(want, got, inside):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_graph_replays(dev):
    args = path_inputs(dev, 23)
    whole_path(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = whole_path(*args)
    for seed in (23, 24, 25, 26):
        fresh = path_inputs(dev, seed)
        for a, b in zip(args, fresh):
            if isinstance(a, sg.Mx4):
                a.codes.copy_(b.codes), a.scales.copy_(b.scales)
            else:
                a.copy_(b)
        want = whole_path(*fresh)
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_many_rows(dev):
    """More rows than one grid dimension counts, in every operator."""
    rows, cols = 700001, 32
    gen = torch.Generator(device=dev)
    gen.manual_seed(30)
    x = torch.randn(rows, cols, generator=gen, device=dev)
    q, qt = sg.mx4_quantize_both(x)
    y = sg.mx4_dequantize(q)
    yt = sg.mx4_dequantize(qt)
    for r in (0, 262144, 524288, 699968):       # whole blocks along the columns; the last has one row more
        assert np.array_equal(host(yt[:, r:r + 32]), ref.rounded(host(x[r:r + 32]).T))
    pick = torch.tensor([0, 1, 262143, 262144, 524287, 524288, 700000], device=dev)
    assert np.array_equal(host(y[pick]), ref.rounded(host(x[pick])))
    again = sg.mx4_quantize(x)
    assert torch.equal(again.codes, q.codes) and torch.equal(again.scales, q.scales)
    a = sg.mx4_quantize(x[:5])
    close(sg.mx4_gemm(q, a)[pick], host(y[pick]) @ ref.rounded(host(x[:5])).T, product_bound(host(y[pick]), ref.rounded(host(x[:5]))))
    close(sg.mx4_linear(x[:3], q)[:, pick], host(x[:3]) @ host(y[pick]).T, product_bound(host(x[:3]), host(y[pick]), 3))


def test_refuses_memory_that_is_not_the_devices(dev):
    """Addresses outside an allocation of the device, and arrays that reach past their allocation's end."""
    x, q = torch.zeros(4, 128, device=dev), sg.mx4_quantize(torch.zeros(4, 128, device=dev))
    c, s = q.codes.data_ptr(), q.scales.data_ptr()
    on_host = torch.zeros(4096, dtype=torch.uint8).data_ptr() & ~15
    call = sg.library().sgemm_f32_mx4_quantize
    stream = torch.cuda.current_stream().cuda_stream
    assert call(4, 128, 0, x.data_ptr(), 128, 0, c, on_host, None, None, stream) == sg.ERR_POINTER
    assert call(4, 128, 0, on_host, 128, 0, c, s, None, None, stream) == sg.ERR_POINTER
    big = torch.empty(64 << 20, dtype=torch.uint8, device=dev)     # an allocation of its own
    assert call(1 << 20, 128, 0, big.data_ptr(), 128, 0, c, s, None, None, stream) != sg.OK
    assert call(4, 128, 0, x.data_ptr(), 128, 0, c, s, None, None, stream) == sg.OK
    torch.cuda.synchronize()


def test_offsets_past_32_bits(dev):
    """Weights of 4.9 GB: rows at both ends and in the middle of all operators that read or write them."""
    rows, cols = 70000, 140000
    gen = torch.Generator(device=dev)
    gen.manual_seed(27)
    q = sg.Mx4(torch.randint(0, 256, (rows, 64 * 1094), generator=gen, device=dev, dtype=torch.uint8),
               torch.randint(118, 122, (1094, 70016, 4), generator=gen, device=dev, dtype=torch.uint8), rows, cols)
    q.codes[:, cols // 2:] = 0
    q.scales[1093, :, 3] = 0       # the last slab ends within its third block
    pick = torch.tensor([0, 1, 35000, 61356, 61357, 69983, 69999])

    def part(r):
        s = np.zeros((1094, 32, 4), dtype=np.uint8)
        s[:, 0] = q.scales[:, r].cpu().numpy()
        return ref.values(q.codes[r:r + 1].cpu().numpy(), s, cols)

    want = np.concatenate([part(int(r)) for r in pick])
    x = normal(np.random.default_rng(28), 3, cols, torch.bfloat16, dev)
    close(sg.mx4_linear(x, q)[:, pick.to(dev)], host(x) @ want.T, product_bound(host(x), want), torch.bfloat16)
    a = sg.mx4_quantize(x)
    close(sg.mx4_gemm(a, q)[:, pick.to(dev)], values(a) @ want.T, product_bound(values(a), want))
    y = sg.mx4_dequantize(q, dtype=torch.bfloat16)
    assert np.array_equal(host(y[pick.to(dev)]), want)
    # Values of 4 bits under their own scales survive the way back, blocks of largest code below 4 under other scales.
    again = sg.mx4_quantize(y)
    assert torch.equal(sg.mx4_dequantize(again, dtype=torch.bfloat16)[pick.to(dev)], y[pick.to(dev)])


def test_example(dev):
    """The example's parts: training lowers the loss, serving is as far off as 4 bits make it, graph and eager agree."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "four_bit_block.py")
    spec = importlib.util.spec_from_file_location("four_bit_block", path)
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)
    W, first, last = block.train(60, dev)
    assert last < 0.2 * first
    # Rounding to levels a sixth to a half apart: an error of at most a quarter of each weight, far less on average.
    assert 0.0 < block.serve(W, 4, dev) < 0.25
    eager, replayed = block.decode(3, dev)
    assert torch.equal(eager, replayed) and bool(torch.isfinite(eager).all())
