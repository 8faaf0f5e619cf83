"""The 8-bit integer operators on the GPU against the 64-bit reference.

Whole numbers and scales have to be the reference's, and so have the products:
their sums are exact, and what follows (a sum as a float, times one scale, times
the other, rounded to the result's type) is done the same way there.  Only where
exponentials enter are there bounds, counted in roundings.
"""
import numpy as np
import pytest
import torch

import fp32_sgemm_f32_amd as sg
from oracle import i8 as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
typed = pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "bf16", "fp16"])
U = 2.0 ** -24      # half a step of fp32, relatively


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


def random_i8(rng, rows, cols, dev, scales=None):
    q = np.zeros((rows, ref.padded(cols)), dtype=np.int8)
    q[:, :cols] = rng.integers(-127, 128, (rows, cols))
    s = np.ldexp(1.0 + rng.random(rows), rng.integers(-9, 3, rows)) if scales is None else scales
    return sg.I8(torch.from_numpy(q).to(dev), torch.from_numpy(np.asarray(s, np.float32)).to(dev), rows, cols)


def parts(q):
    """(whole numbers, scales) of an I8 in 64 bits."""
    return host(q.values)[:, :q.shape[1]], host(q.scales)


def same(got, want, dtype=torch.float32):
    """got is want (32 bits) rounded to dtype."""
    w = torch.from_numpy(np.asarray(want, np.float32)).to(dtype)
    g = got.detach().cpu()
    assert g.dtype == dtype and g.shape == w.shape
    bad = ~((g == w) | (g.isnan() & w.isnan()))
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: {g[bad][0]} against {w[bad][0]}"


def close(got, want, bound, dtype):
    """got within bound of want, plus half a step of its type."""
    f = torch.finfo(dtype)
    got = host(got)
    lim = bound + np.maximum((np.abs(want) + bound) * (f.eps / 2), f.smallest_normal * f.eps / 2)
    # Beyond the type's largest value plus half its step a result rounds to infinity.
    edge = f.max * (1 + f.eps / 4)
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(got - want) <= lim) | ((got == np.copysign(np.inf, want)) & (np.abs(want) + bound >= edge)))
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} against {want[bad][0]}"


def check_rows(q, x):
    want, s = ref.whole(x)
    rows, cols = want.shape
    assert q.shape == (rows, cols) and q.group is None
    assert np.array_equal(host(q.values)[:, :cols], want) and not host(q.values)[:, cols:].any()
    assert np.array_equal(host(q.scales), s, equal_nan=True)


def check_groups(q, x):
    want, s = ref.grouped(x)
    assert q.shape == x.shape and q.group == 128
    assert np.array_equal(host(q.values), want) and np.array_equal(host(q.scales), s, equal_nan=True)


# ---- quantisation -----------------------------------------------------------------------------------------------

SHAPES = [(1, 1), (1, 32), (3, 31), (7, 33), (16, 128), (33, 129), (5, 260), (130, 255), (257, 96), (1, 5000), (200, 1), (3, 2048),
          (3, 2049), (2, 8193), (4, 8192), (2, 33000), (1, 32769), (300, 7)]


@typed
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_quantize(dev, dtype, shape):
    x = normal(np.random.default_rng(1), *shape, dtype, dev)
    check_rows(sg.i8_quantize(x), host(x))
    check_rows(sg.i8_quantize(x.t()), host(x).T)
    check_groups(sg.i8_quantize(x, group=128), host(x))


@typed
@pytest.mark.parametrize("pad, shift", [(0, 1), (1, 0), (8, 8), (3, 5), (4, 0)])
def test_quantize_strided(dev, dtype, pad, shift):
    x = normal(np.random.default_rng(2), 37, 300, dtype, dev)
    v = strided(x, pad, shift)
    check_rows(sg.i8_quantize(v), host(x))
    check_rows(sg.i8_quantize(v.t()), host(x).T)
    check_groups(sg.i8_quantize(v, group=128), host(x))
    # a column-major view of a piece
    check_rows(sg.i8_quantize(v[3:, 5:].t()), host(x)[3:, 5:].T)


def near_borders(rng, scale, levels):
    """A row whose scale is `scale`: its largest number, and values on and a float beside each half."""
    half = (np.arange(-levels, levels) + 0.5) * scale
    f = half.astype(np.float32)
    assert np.array_equal(f, half)       # scales with few bits keep halves exact
    row = np.concatenate([f, np.nextafter(f, np.float32(np.inf)), np.nextafter(f, np.float32(-np.inf)), [np.float32(levels * scale)]])
    return rng.permutation(row)


@pytest.mark.parametrize("scale", [1.0, 0.75, 2.0 ** -100, 2.0 ** 100, 1.375 * 2.0 ** -126, 2.0 ** -126])
def test_quantize_at_every_border(dev, scale):
    x = near_borders(np.random.default_rng(3), scale, 127)[None, :].repeat(3, 0)
    t = torch.from_numpy(x).to(dev)
    assert float(ref.whole(x)[1][0]) == scale
    check_rows(sg.i8_quantize(t), x)
    check_rows(sg.i8_quantize(t.t().contiguous().t()), x)


@pytest.mark.parametrize("seed", range(4))
def test_quantize_floats_next_to_borders_of_any_scale(dev, seed):
    """Rows of random largest values, filled with the floats that lie nearest to (n + 1/2) s, on both sides."""
    rng = np.random.default_rng(seed)
    m = np.ldexp(1.0 + rng.random(64), rng.integers(-60, 60, 64)).astype(np.float32)
    s = (m.astype(np.float64) / 127).astype(np.float32).astype(np.float64)
    f = ((np.arange(-127, 127) + 0.5)[None, :] * s[:, None]).astype(np.float32)
    x = np.concatenate([f, np.nextafter(f, np.float32(np.inf)), np.nextafter(f, np.float32(-np.inf)), m[:, None]], 1)
    x = np.clip(x, -m[:, None], m[:, None])
    check_rows(sg.i8_quantize(torch.from_numpy(x).to(dev)), x)
    check_rows(sg.i8_quantize(torch.from_numpy(np.ascontiguousarray(x.T)).to(dev).t()), x)
    check_groups(sg.i8_quantize(torch.from_numpy(x[:, -128:]).to(dev).contiguous(), group=128), x[:, -128:])


@pytest.mark.parametrize("dtype", TYPES[1:], ids=["bf16", "fp16"])
def test_quantize_every_16_bit_value(dev, dtype):
    """Every finite value, in rows of like size and in rows of all sizes."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(dtype)
    v = v[torch.isfinite(v)]
    v = v[: len(v) // 256 * 256]
    for x in (v.view(-1, 256), v.view(256, -1)):
        check_rows(sg.i8_quantize(x.to(dev)), host(x))
        check_rows(sg.i8_quantize(x.t().contiguous().to(dev).t()), host(x))
        check_groups(sg.i8_quantize(x.contiguous().to(dev), group=128), host(x))


def test_quantize_zeros_subnormals_nan_infinity(dev):
    x = np.zeros((8, 300), dtype=np.float32)
    x[1] = np.float32(2.0 ** -149)
    x[2, ::3] = np.float32(2.0 ** -130)
    x[3, 7] = np.nan
    x[4, 299] = -np.inf
    x[5] = np.finfo(np.float32).max
    x[6, 128:] = np.inf
    x[7] = -np.float32(1e-37)
    t = torch.from_numpy(x).to(dev)
    check_rows(sg.i8_quantize(t), x)
    check_rows(sg.i8_quantize(torch.from_numpy(np.ascontiguousarray(x.T)).to(dev).t()), x)
    check_groups(sg.i8_quantize(t, group=128), x)


@typed
@pytest.mark.parametrize("shape", SHAPES + [(70, 513), (9, 1027)], ids=str)
def test_dequantize(dev, dtype, shape):
    x = normal(np.random.default_rng(4), *shape, torch.float32, dev)
    for group in (None, 128):
        q = sg.i8_quantize(x, group=group)
        want = ref.values(host(q.values), host(q.scales), shape[1])
        same(sg.i8_dequantize(q, dtype=dtype), want, dtype)
        out = strided(torch.zeros(shape, dtype=dtype, device=dev), 3, 1)
        wide = out._base if out._base is not None else out
        before = wide.clone()
        assert sg.i8_dequantize(q, out=out) is out
        same(out, want, dtype)
        # what lies between the rows is left as it was
        out.copy_(torch.zeros(shape, dtype=dtype, device=dev))
        assert torch.equal(wide.isnan(), before.isnan())


def test_quantize_of_nothing(dev):
    for shape in ((0, 5), (5, 0), (0, 0)):
        x = torch.zeros(shape, device=dev)
        for q in (sg.i8_quantize(x), sg.i8_quantize(x, group=128)):
            assert q.shape == shape and sg.i8_dequantize(q).shape == shape


# ---- products ---------------------------------------------------------------------------------------------------

GEMMS = [(1, 1, 1), (1, 16, 128), (5, 70, 33), (33, 70, 300), (64, 64, 64), (65, 63, 127), (130, 129, 200), (300, 290, 256),
         (257, 300, 640), (1111, 999, 2050), (17, 2000, 1000), (2000, 17, 1000), (2, 5000, 4096), (48, 513, 8200), (640, 640, 129)]


def gemm_want(a, b):
    (x, sx), (y, sy) = parts(a), parts(b)
    return ref.product(x, sx, y, sy)


@typed
@pytest.mark.parametrize("m, n, k", GEMMS)
def test_gemm(dev, dtype, m, n, k):
    rng = np.random.default_rng(5)
    a, b = random_i8(rng, m, k, dev), random_i8(rng, n, k, dev)
    same(sg.i8_gemm(a, b, dtype=dtype), gemm_want(a, b), dtype)


@typed
@pytest.mark.parametrize("m, n, k", [(3, 70, 300), (33, 70, 300), (300, 290, 256), (2100, 2050, 128)])
@pytest.mark.parametrize("alpha, beta", [(1.0, 1.0), (-0.5, 2.0), (0.0, 3.0), (2.0, 0.0)])
def test_gemm_adds_to_a_strided_result(dev, dtype, m, n, k, alpha, beta):
    rng = np.random.default_rng(6)
    a, b = random_i8(rng, m, k, dev), random_i8(rng, n, k, dev)
    old = normal(rng, m, n, dtype, dev)
    out = strided(old, 3, 1)
    if beta == 0.0:
        out.fill_(float("nan"))      # not read
    base = out._base
    around = base.isnan()
    sg.i8_gemm(a, b, out=out, alpha=alpha, beta=beta)
    p = gemm_want(a, b).astype(np.float64) * alpha        # a power of two: exact
    want = p + (beta * host(old) if beta else 0.0)
    # one more rounding of the sum (and of beta times the old value, where they are not fused)
    close(out, want, 2 * U * (np.abs(want) + np.abs(beta * host(old))), dtype)
    out.fill_(float("nan")) if beta == 0.0 else None
    assert torch.equal(base.isnan(), around)


def test_gemm_of_nothing(dev):
    a, b = sg.i8_quantize(torch.ones(5, 0, device=dev)), sg.i8_quantize(torch.ones(7, 0, device=dev))
    assert torch.equal(sg.i8_gemm(a, b), torch.zeros(5, 7, device=dev))
    c = torch.ones(5, 7, device=dev)
    sg.i8_gemm(a, b, out=c, beta=2.0)
    assert torch.equal(c, torch.full((5, 7), 2.0, device=dev))
    n = sg.i8_quantize(torch.full((5, 9), float("nan"), device=dev))
    sg.i8_gemm(n, n, out=c[:, :5], alpha=0.0, beta=1.0)      # neither is read
    assert torch.equal(c, torch.full((5, 7), 2.0, device=dev))
    for m, n in ((0, 3), (3, 0)):
        assert sg.i8_gemm(sg.i8_quantize(torch.ones(m, 4, device=dev)), sg.i8_quantize(torch.ones(n, 4, device=dev))).shape == (m, n)


@pytest.mark.parametrize("m, n", [(1, 40), (20, 5), (70, 90), (300, 130)])
def test_gemm_of_the_longest_sum(dev, m, n):
    """131072 products of the largest numbers: the sums reach 2^31 less a little, in both signs."""
    k = 1 << 17
    x, y = torch.full((m, k), 127, dtype=torch.int8, device=dev), torch.full((n, k), 127, dtype=torch.int8, device=dev)
    x[::2] = -127
    y[1, ::2] = 126
    a, b = sg.I8(x, torch.ones(m, device=dev), m, k), sg.I8(y, torch.ones(n, device=dev), n, k)
    same(sg.i8_gemm(a, b), gemm_want(a, b))
    long = sg.I8(torch.zeros(2, k + 128, dtype=torch.int8, device=dev), torch.ones(2, device=dev), 2, k + 1)
    with pytest.raises(ValueError):
        sg.i8_gemm(long, long)


@pytest.mark.parametrize("m, n, k", [(3, 50, 300), (40, 50, 300), (300, 300, 256)])
def test_gemm_keeps_nan_to_its_rows(dev, m, n, k):
    rng = np.random.default_rng(7)
    x, y = normal(rng, m, k, torch.float32, dev), normal(rng, n, k, torch.float32, dev)
    x[1, 5], y[7, 0] = float("inf"), float("nan")
    a, b = sg.i8_quantize(x), sg.i8_quantize(y)
    got = sg.i8_gemm(a, b)
    same(got, gemm_want(a, b))
    nan = torch.zeros(m, n, dtype=torch.bool, device=dev)
    nan[1], nan[:, 7] = True, True
    assert torch.equal(got.isnan(), nan)


@pytest.mark.parametrize("m", [2, 100])
def test_gemm_scales_far_apart(dev, m):
    """Neither order of the two scales may overflow or vanish where the result does not."""
    rng = np.random.default_rng(8)
    s = np.ldexp(1.0, rng.integers(-126, 120, m)).astype(np.float32)
    t = np.ldexp(1.0, rng.integers(-126, 120, 130)).astype(np.float32)
    a, b = random_i8(rng, m, 200, dev, s), random_i8(rng, 130, 200, dev, t)
    got = sg.i8_gemm(a, b)
    with np.errstate(over="ignore"):
        same(got, gemm_want(a, b))
    (x, sx), (y, sy) = parts(a), parts(b)
    want = (x @ y.T) * sx[:, None] * sy[None, :]
    inside = (np.abs(want) < 2.0 ** 127) & (np.abs(want) > 2.0 ** -125)
    assert inside.sum() > 50 and np.array_equal(host(got)[inside], want[inside])


@pytest.mark.parametrize("m, n, k", [(5, 90, 256), (70, 90, 256), (300, 300, 384), (2100, 2050, 256)])
def test_gemm_repeats(dev, m, n, k):
    rng = np.random.default_rng(9)
    a, b = random_i8(rng, m, k, dev), random_i8(rng, n, k, dev)
    first = sg.i8_gemm(a, b)
    for _ in range(3):
        assert torch.equal(first, sg.i8_gemm(a, b))


LINEARS = [(1, 1, 1), (1, 16, 128), (1, 100, 4096), (2, 33, 31), (7, 15, 130), (8, 200, 257), (9, 200, 257), (13, 501, 1640), (16, 64, 640),
           (17, 200, 100), (33, 48, 1000), (64, 130, 2050), (65, 70, 300), (130, 20, 129), (5, 3001, 96), (16, 40, 9000), (1, 5, 16400),
           (48, 30, 5001), (1, 4096, 4096), (3, 1000, 33000)]


@typed
@pytest.mark.parametrize("m, n, k", LINEARS)
def test_linear(dev, dtype, m, n, k):
    rng = np.random.default_rng(10)
    x, w = normal(rng, m, k, dtype, dev), random_i8(rng, n, k, dev)
    q, s = ref.whole(host(x))
    want = ref.product(q, s, *parts(w))
    same(sg.i8_linear(x, w), want, dtype)
    assert torch.equal(sg.i8_gemm(sg.i8_quantize(x), w, dtype=dtype), sg.i8_linear(x, w))


@typed
@pytest.mark.parametrize("m", [1, 3, 20, 70])
@pytest.mark.parametrize("pad, shift", [(1, 0), (0, 1), (8, 0), (2, 6)])
def test_linear_strided(dev, dtype, m, pad, shift):
    rng = np.random.default_rng(11)
    x, w = normal(rng, m, 300, dtype, dev), random_i8(rng, 77, 300, dev)
    out = strided(torch.zeros(m, 77, dtype=dtype, device=dev), pad, shift)
    base = out._base
    sg.i8_linear(strided(x, pad, shift), w, out=out)
    same(out, ref.product(*ref.whole(host(x)), *parts(w)), dtype)
    assert int(base.isnan().sum()) == base.numel() - m * 77


@typed
@pytest.mark.parametrize("m", [1, 3, 30])
def test_linear_nan_and_infinity_stay_in_their_rows(dev, dtype, m):
    rng = np.random.default_rng(12)
    x, w = normal(rng, m, 200, dtype, dev), random_i8(rng, 50, 200, dev)
    clean = sg.i8_linear(x, w)
    x[m - 1, 3] = float("nan") if m % 2 else float("-inf")
    w.scales[7] = float("nan")
    got = sg.i8_linear(x, w)
    assert got[m - 1].isnan().all() and got[:, 7].isnan().all()
    keep = torch.ones(50, dtype=torch.bool, device=dev)
    keep[7] = False
    assert torch.equal(got[:m - 1][:, keep], clean[:m - 1][:, keep])


def test_linear_of_nothing(dev):
    w = sg.i8_quantize(torch.ones(7, 0, device=dev))
    assert torch.equal(sg.i8_linear(torch.ones(5, 0, device=dev), w), torch.zeros(5, 7, device=dev))
    w = sg.i8_quantize(torch.ones(7, 4, device=dev))
    assert sg.i8_linear(torch.ones(0, 4, device=dev), w).shape == (0, 7)
    assert sg.i8_linear(torch.ones(3, 4, device=dev), sg.i8_quantize(torch.ones(0, 4, device=dev))).shape == (3, 0)


# ---- training ---------------------------------------------------------------------------------------------------

TRAINS = [(1, 1, 1), (33, 70, 100), (130, 257, 64), (333, 40, 513), (1030, 1025, 300), (40, 1000, 129), (5, 3, 2100), (128, 128, 128),
          (700, 513, 900)]


@typed
@pytest.mark.parametrize("m, n, k", TRAINS)
def test_train(dev, dtype, m, n, k):
    rng = np.random.default_rng(13)
    x, w, d = normal(rng, m, k, dtype, dev), normal(rng, n, k, dtype, dev, k ** -0.5), normal(rng, m, n, dtype, dev, 0.1)
    y, saved = sg.i8_train_forward(x, w)
    (xq, sx), (wq, sw) = ref.whole(host(x)), ref.whole(host(w))
    check_rows(saved[0], host(x)), check_rows(saved[1], host(w))
    same(y, ref.product(xq, sx, wq, sw), dtype)
    dx, dw = sg.i8_train_backward(d, saved)
    want_x, want_w = ref.backward(host(d), xq, sx, wq, sw)
    same(dx, want_x, dtype)
    same(dw, want_w)
    # once more, into a gradient that is there, from a strided dY
    old = normal(rng, n, k, torch.float32, dev)
    acc = strided(old, 5, 3)
    around = acc._base.isnan()
    again, got = sg.i8_train_backward(strided(d, 3, 1), saved, dW=acc)
    assert got is acc and torch.equal(again, dx)
    total = want_w.astype(np.float64) + host(old)
    close(acc, total, 0.0, torch.float32)
    assert torch.equal(acc._base.isnan(), around)


@typed
def test_train_of_two_types_views_and_given_weights(dev, dtype):
    rng = np.random.default_rng(14)
    m, n, k = 70, 90, 200
    x, w, d = normal(rng, m, k, dtype, dev), normal(rng, n, k, torch.float32, dev), normal(rng, m, n, torch.float16, dev, 0.01)
    y, saved = sg.i8_train_forward(x, w)
    dx, dw = sg.i8_train_backward(d, saved)
    assert y.dtype == dtype and dx.dtype == torch.float16 and dw.dtype == torch.float32
    for a, b in ((x.t().contiguous().t(), w), (x, w.t().contiguous().t()), (strided(x, 3, 1), strided(w, 1, 2)), (x, sg.i8_quantize(w))):
        other, kept = sg.i8_train_forward(a, b)
        assert torch.equal(other, y)
        assert torch.equal(kept[0].values, saved[0].values) and torch.equal(kept[1].scales, saved[1].scales)
        for dd in (d, d.t().contiguous().t()):
            got = sg.i8_train_backward(dd, kept)
            assert torch.equal(got[0], dx) and torch.equal(got[1], dw)


@pytest.mark.parametrize("m, n, k", [(0, 5, 7), (5, 0, 7), (5, 7, 0), (0, 0, 0)])
def test_train_of_nothing(dev, m, n, k):
    x, w, d = torch.ones(m, k, device=dev), torch.ones(n, k, device=dev), torch.ones(m, n, device=dev)
    y, saved = sg.i8_train_forward(x, w)
    assert torch.equal(y, torch.zeros(m, n, device=dev))
    dx, dw = sg.i8_train_backward(d, saved)
    assert torch.equal(dx, torch.zeros(m, k, device=dev)) and torch.equal(dw, torch.zeros(n, k, device=dev))
    kept = torch.full((n, k), 3.0, device=dev)
    sg.i8_train_backward(d, saved, dW=kept)
    assert torch.equal(kept, torch.full((n, k), 3.0, device=dev))


def test_train_nan_reaches_what_depends_on_it(dev):
    rng = np.random.default_rng(15)
    m, n, k = 40, 50, 60
    x, w, d = normal(rng, m, k, torch.float32, dev), normal(rng, n, k, torch.float32, dev), normal(rng, m, n, torch.float32, dev)
    d[3, 4] = float("inf")
    x[7, 0] = float("nan")
    y, saved = sg.i8_train_forward(x, w)
    dx, dw = sg.i8_train_backward(d, saved)
    want = torch.zeros(m, n, dtype=torch.bool, device=dev)
    want[7] = True
    assert torch.equal(y.isnan(), want)
    assert dx[3].isnan().all() and not dx[torch.arange(m, device=dev) != 3].isnan().any()
    assert dw.isnan().all()       # every channel's sum takes token 7
    x[7, 0] = 0.0
    _, saved = sg.i8_train_forward(x, w)
    dw = sg.i8_train_backward(d, saved)[1]
    assert dw[4].isnan().all() and not dw[torch.arange(n, device=dev) != 4].isnan().any()


def test_train_refuses_what_does_not_fit(dev):
    x, w = torch.ones(4, 8, device=dev), torch.ones(5, 8, device=dev)
    _, saved = sg.i8_train_forward(x, w)
    for call in (lambda: sg.i8_train_forward(x, torch.ones(5, 9, device=dev)), lambda: sg.i8_train_backward(torch.ones(4, 4, device=dev), saved),
                 lambda: sg.i8_train_backward(torch.ones(4, 5, device=dev), saved, dW=torch.ones(5, 9, device=dev)),
                 lambda: sg.i8_train_backward(torch.ones(4, 5, device=dev), (saved[0], sg.i8_quantize(w, group=128))),
                 lambda: sg.i8_train_forward(torch.ones(1, (1 << 17) + 1, device=dev), torch.ones(1, (1 << 17) + 1, device=dev))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        sg.i8_train_backward(torch.ones(4, 5, device=dev), (x, w))


def test_train_gradient_against_differences(dev):
    """On whole numbers with a 127 in each row, before and after a step, the layer is bilinear: central differences of
    sum(dY * Y) are its gradient, exactly.  (dY: whole numbers too, with a 127 in each row, or a 32639 in each column.)"""
    rng = np.random.default_rng(16)
    m, n, k = 40, 36, 70

    def small(rows, cols, top, axis):
        v = rng.integers(-9, 10, (rows, cols)).astype(np.float64)
        (v[:, 0] if axis else v[0, :])[:] = top
        return v

    X, W = small(m, k, 127, 1), small(n, k, 127, 1)
    t = lambda v: torch.from_numpy(v).float().to(dev)
    for D, which in ((small(m, n, 127, 1), 0), (small(m, n, 32639, 0), 1)):
        f = lambda X, W: float((host(sg.i8_train_forward(t(X), t(W))[0]) * D).sum())
        _, saved = sg.i8_train_forward(t(X), t(W))
        grad = host(sg.i8_train_backward(t(D), saved)[which])
        for _ in range(5):
            u = rng.choice([-1.0, 0.0, 1.0], (X, W)[which].shape)
            u[:, 0] = 0.0
            there, back = (f(X + u, W), f(X - u, W)) if which == 0 else (f(X, W + u), f(X, W - u))
            assert (there - back) / 2 == (grad * u).sum()


# ---- the gated activation ---------------------------------------------------------------------------------------

GATED = [(1, 1), (3, 100), (77, 1001), (300, 256), (5, 127), (2, 5000), (129, 8), (1, 14336)]


@typed
@pytest.mark.parametrize("rows, inner", GATED)
@pytest.mark.parametrize("pad, shift", [(0, 0), (3, 1)])
def test_swiglu(dev, dtype, rows, inner, pad, shift):
    rng = np.random.default_rng(17)
    x = normal(rng, rows, 2 * inner, dtype, dev, 2.0)
    d = normal(rng, rows, inner, dtype, dev, 0.1)
    gu = strided(x, pad, shift)
    h, (g, u) = sg.i8_swiglu_forward(gu)
    G, V = host(x)[:, :inner], host(x)[:, inner:]
    check_groups(g, G), check_groups(u, V)
    # exp (2 halves of a step), the sum, the quotient, the product: 6 roundings, with room for their products
    want = ref.gated(G, V)
    close(h, want, 7 * U * np.abs(want) + 2.0 ** -149, dtype)
    out = strided(torch.zeros(rows, 2 * inner, dtype=dtype, device=dev), pad, shift)
    assert sg.i8_swiglu_backward(strided(d, pad, shift), (g, u), out=out) is out
    G, V = (ref.values(host(q.values), host(q.scales), inner).astype(np.float64) for q in (g, u))
    D = host(d)
    dg, du = ref.gated_backward(D, G, V)
    p = ref.sigmoid(G)
    # the same, and five more for the slope; its two addends can cancel
    bound_g = 14 * U * np.abs(D * V * p) * (1.0 + np.abs(G) * ref.sigmoid(-G)) + 2.0 ** -148
    bound_u = 8 * U * np.abs(du) + 2.0 ** -148
    close(out, np.concatenate((dg, du), 1), np.concatenate((bound_g, bound_u), 1), dtype)
    assert int(out._base.isnan().sum()) == out._base.numel() - out.numel()


def test_swiglu_far_values_nan_and_infinity(dev):
    x = torch.zeros(5, 512, device=dev)
    x[0, :256] = torch.linspace(-300, 300, 256, device=dev)
    x[0, 256:] = 2.0
    x[1, 3], x[2, 256 + 200] = float("nan"), float("inf")
    x[3, :256], x[3, 256:] = -3e38, 3e38
    x[4, 0], x[4, 256] = float("-inf"), 1.0
    h, saved = sg.i8_swiglu_forward(x)
    want = ref.gated(host(x)[0, :256], host(x)[0, 256:])
    # exp of -300 and less is infinite in 32 bits: the activation is 0 there
    close(h[:1], want[None, :], 7 * U * np.abs(want)[None, :] + 1e-36, torch.float32)
    assert h[1, 3].isnan() and not h[1, 4:].isnan().any()
    assert h[3].eq(0).all()
    grad = sg.i8_swiglu_backward(torch.ones(5, 256, device=dev), saved)
    assert torch.isfinite(grad[0]).all() and torch.isfinite(grad[3]).all()
    # a group with a NaN or an infinity is NaN, and with it the gradients that take it: no others
    assert grad[1, :128].isnan().all() and torch.isfinite(grad[1, 128:256]).all() and grad[1, 256:384].isnan().all()
    assert grad[2, 128:256].isnan().all() and torch.isfinite(grad[2, :128]).all() and torch.isfinite(grad[2, 256:]).all()
    assert grad[4, :128].isnan().all() and torch.isfinite(grad[4, 128:256]).all()


def test_swiglu_gradient_against_differences(dev):
    """Central differences of sum(dH * H) in 64 bits at the checkpoint's values: an error of the difference (h^2 times a
    third derivative below 2 |u|) and of the gradient's roundings."""
    rng = np.random.default_rng(18)
    x = normal(rng, 9, 400, torch.float32, dev)
    d = normal(rng, 9, 200, torch.float32, dev)
    _, (g, u) = sg.i8_swiglu_forward(x)
    got = host(sg.i8_swiglu_backward(d, (g, u)))
    G, V = (ref.values(host(q.values), host(q.scales), 200).astype(np.float64) for q in (g, u))
    D, e = host(d), 1e-4
    dg = D * (ref.gated(G + e, V) - ref.gated(G - e, V)) / (2 * e)
    du = D * (ref.gated(G, V + e) - ref.gated(G, V - e)) / (2 * e)
    size = np.abs(D) * (1.0 + np.abs(G)) * (1.0 + np.abs(V))
    assert (np.abs(got - np.concatenate((dg, du), 1)) <= np.concatenate((size, size), 1) * (14 * U + e * e + 1e-11)).all()


def test_swiglu_of_nothing_and_refusals(dev):
    for m, f in ((0, 4), (4, 0)):
        h, saved = sg.i8_swiglu_forward(torch.ones(m, 2 * f, device=dev))
        assert h.shape == (m, f) and sg.i8_swiglu_backward(torch.ones(m, f, device=dev), saved).shape == (m, 2 * f)
    x = torch.ones(4, 8, device=dev)
    _, saved = sg.i8_swiglu_forward(x)
    for call in (lambda: sg.i8_swiglu_forward(torch.ones(4, 7, device=dev)), lambda: sg.i8_swiglu_backward(x, saved),
                 lambda: sg.i8_swiglu_forward(x, out=torch.ones(4, 8, device=dev)), lambda: sg.i8_swiglu_forward(x.t()),
                 lambda: sg.i8_swiglu_backward(torch.ones(4, 4, device=dev), (saved[0], sg.i8_quantize(torch.ones(4, 4, device=dev))))):
        with pytest.raises(ValueError):
            call()


# ---- refusals, streams, graphs, large matrices ------------------------------------------------------------------

def test_python_refuses_what_does_not_fit(dev):
    x, q = torch.ones(4, 8, device=dev), sg.i8_quantize(torch.ones(5, 8, device=dev))
    short = sg.i8_quantize(torch.ones(5, 7, device=dev))
    for call in (lambda: sg.i8_gemm(q, short), lambda: sg.i8_linear(x, short), lambda: sg.i8_gemm(q, q, beta=1.0),
                 lambda: sg.i8_gemm(q, q, out=torch.ones(5, 4, device=dev)), lambda: sg.i8_linear(x, q, out=torch.ones(4, 5, device=dev).half()),
                 lambda: sg.i8_quantize(torch.ones(8, device=dev)), lambda: sg.i8_quantize(x.t(), group=128),
                 lambda: sg.i8_quantize(x[:, ::2]), lambda: sg.i8_gemm(q, sg.i8_quantize(x, group=128)),
                 lambda: sg.i8_linear(x, sg.i8_quantize(x, group=128))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sg.i8_quantize(x.double()), lambda: sg.i8_dequantize(q, dtype=torch.float64), lambda: sg.i8_gemm(q, x),
                 lambda: sg.i8_linear(q, q)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(sg.SgemmError):
        sg.i8_dequantize(q, out=q.values.view(torch.float32)[:, :8])     # over its own input


def test_refuses_memory_that_is_not_the_devices(dev):
    x = torch.zeros(4, 128, device=dev)
    q = sg.i8_quantize(x)
    v, s = q.values.data_ptr(), q.scales.data_ptr()
    on_host = torch.zeros(4096, dtype=torch.uint8).data_ptr() & ~15
    call = sg.library().sgemm_f32_i8_quantize
    stream = torch.cuda.current_stream().cuda_stream
    assert call(0, 4, 128, 0, 0, x.data_ptr(), 128, v, on_host, None, 0, stream) == sg.ERR_POINTER
    assert call(0, 4, 128, 0, 0, on_host, 128, v, s, None, 0, stream) == sg.ERR_POINTER
    big = torch.empty(64 << 20, dtype=torch.uint8, device=dev)     # an allocation of its own
    assert call(0, 1 << 20, 128, 0, 0, big.data_ptr(), 128, v, s, None, 0, stream) != sg.OK
    assert call(0, 4, 128, 0, 0, x.data_ptr(), 128, v, s, None, 0, stream) == sg.OK
    torch.cuda.synchronize()


def whole_path(x, w, wg, d):
    """A layer, a gated activation and a second layer, forward and backward, and the first once more for serving."""
    y, saved = sg.i8_train_forward(x, w)
    h, kept = sg.i8_swiglu_forward(y)
    z, last = sg.i8_train_forward(h, wg)
    dh, dwg = sg.i8_train_backward(d, last)
    dy = sg.i8_swiglu_backward(dh, kept)
    dx, dw = sg.i8_train_backward(dy, saved)
    q = sg.i8_quantize(w)
    return (z, dx, dw, dwg, sg.i8_linear(x, q), sg.i8_linear(x[:1], q), sg.i8_gemm(saved[0], sg.i8_quantize(w.t().contiguous().t())),
            sg.i8_dequantize(sg.i8_quantize(x, group=128), dtype=x.dtype))


def path_inputs(dev, seed):
    rng = np.random.default_rng(seed)
    t = torch.bfloat16
    return (normal(rng, 100, 200, t, dev), normal(rng, 300, 200, t, dev, 0.07), normal(rng, 90, 150, t, dev, 0.08),
            normal(rng, 100, 90, t, dev, 0.01))


def test_a_run_of_them_against_the_reference(dev):
    x, w, wg, d = path_inputs(dev, 19)
    z, dx, dw, dwg, *_ = whole_path(x, w, wg, d)
    (xq, sx), (wq, sw), (vq, sv) = ref.whole(host(x)), ref.whole(host(w)), ref.whole(host(wg))
    y = torch.from_numpy(ref.product(xq, sx, wq, sw)).bfloat16()
    h, kept = sg.i8_swiglu_forward(y.to(dev))
    want = ref.gated(host(y)[:, :150], host(y)[:, 150:])
    close(h, want, 7 * U * np.abs(want) + 2.0 ** -149, torch.bfloat16)
    hq, sh = ref.whole(host(h))
    same(z, ref.product(hq, sh, vq, sv), torch.bfloat16)
    dh, want_wg = ref.backward(host(d), hq, sh, vq, sv)
    same(dwg, want_wg)
    dy = sg.i8_swiglu_backward(torch.from_numpy(dh).bfloat16().to(dev), kept)
    want_x, want_w = ref.backward(host(dy), xq, sx, wq, sw)
    same(dx, want_x, torch.bfloat16)
    same(dw, want_w)


def test_on_another_stream(dev):
    args = path_inputs(dev, 20)
    want = whole_path(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x, w, wg, d = args
    y, saved = sg.i8_train_forward(x, w, stream=s)
    h, kept = sg.i8_swiglu_forward(y, stream=s)
    z, last = sg.i8_train_forward(h, wg, stream=s)
    dh, dwg = sg.i8_train_backward(d, last, stream=s)
    dx, dw = sg.i8_train_backward(sg.i8_swiglu_backward(dh, kept, stream=s), saved, stream=s)
    q = sg.i8_quantize(w, stream=s)
    got = (z, dx, dw, dwg, sg.i8_linear(x, q, stream=s), sg.i8_linear(x[:1], q, stream=s), sg.i8_gemm(saved[0], q, stream=s),
           sg.i8_dequantize(sg.i8_quantize(x, group=128, stream=s), dtype=x.dtype, stream=s))
    with torch.cuda.stream(s):
        inside = whole_path(*args)
    s.synchronize()
    for a, b, c in zip(want, got, inside):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_two_streams_at_once(dev):
    args = [path_inputs(dev, seed) for seed in (21, 22)]
    want = [whole_path(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(whole_path(*args[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


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
    """More rows than one grid dimension counts, in the operators that take them."""
    rows, cols = 700001, 32
    gen = torch.Generator(device=dev)
    gen.manual_seed(30)
    x = torch.randn(rows, cols, generator=gen, device=dev)
    q, g, t = sg.i8_quantize(x), sg.i8_quantize(x, group=128), sg.i8_quantize(x.t())
    assert torch.equal(q.values, g.values) and torch.equal(q.scales, g.scales[:, 0])
    pick = torch.tensor([0, 1, 262143, 262144, 524287, 524288, 700000], device=dev)
    part = sg.i8_quantize(x[pick])
    check_rows(part, host(x[pick]))
    assert torch.equal(q.values[pick], part.values) and torch.equal(q.scales[pick], part.scales)
    s = x.abs().amax(0).double().div(127).float()
    assert torch.equal(t.scales, s) and torch.equal(t.values[:, :rows].double(), (x.t().double() / s.double()[:, None]).round())
    same(sg.i8_dequantize(q)[pick], ref.values(host(part.values), host(part.scales), cols))
    a = sg.i8_quantize(x[:5])
    same(sg.i8_gemm(q, a)[pick], gemm_want(part, a))
    same(sg.i8_linear(x[:3], q)[:, pick], gemm_want(sg.i8_quantize(x[:3]), part))
    h, saved = sg.i8_swiglu_forward(x)
    small, kept = sg.i8_swiglu_forward(x[pick])
    assert torch.equal(h[pick], small) and torch.equal(saved[1].values[pick], kept[1].values)
    d = torch.randn(rows, 16, generator=gen, device=dev)
    assert torch.equal(sg.i8_swiglu_backward(d, saved)[pick], sg.i8_swiglu_backward(d[pick], kept))


def test_offsets_past_32_bits(dev):
    """A matrix of 5.2 GB (its floats 10.5): rows at both ends and in the middle, of all operators that read or write it."""
    rows, cols = 40000, 131000
    gen = torch.Generator(device=dev)
    gen.manual_seed(27)
    x = torch.randn(rows, cols, generator=gen, device=dev, dtype=torch.bfloat16)
    pick = torch.tensor([0, 1, 16383, 16384, 32767, 32768, 39999], device=dev)
    q, g = sg.i8_quantize(x), sg.i8_quantize(x, group=128)
    part = sg.i8_quantize(x[pick])
    check_rows(part, host(x[pick]))
    assert torch.equal(q.values[pick], part.values) and torch.equal(q.scales[pick], part.scales)
    check_groups(sg.i8_quantize(x[pick], group=128), host(x[pick]))
    assert torch.equal(g.values[pick], sg.i8_quantize(x[pick], group=128).values)
    same(sg.i8_dequantize(q, dtype=torch.bfloat16)[pick], ref.values(host(part.values), host(part.scales), cols), torch.bfloat16)
    few = sg.i8_quantize(x[5:8])
    want = gemm_want(few, part)
    same(sg.i8_gemm(few, q)[:, pick], want)
    same(sg.i8_linear(x[5:8], q)[:, pick], want, torch.bfloat16)
    wide = sg.i8_quantize(x[:300])
    same(sg.i8_gemm(wide, q)[:4][:, pick], gemm_want(sg.i8_quantize(x[:4]), part))
    del g
    # down K: the gradient of inputs with those weights, one token's and a batch's
    w, d = q, torch.randn(200, rows, generator=gen, device=dev, dtype=torch.bfloat16)
    tokens = sg.i8_quantize(x[:200])
    dx, dw = sg.i8_train_backward(d, (tokens, w))
    v = (d.float() * q.scales[None, :])
    s = (v.abs().amax(1).double() / 127).float()
    n = (v.double() / s.double()[:, None]).round()
    at = torch.tensor([0, 1, 70000, 130999], device=dev)
    total = n @ w.values[:, at].double()
    same(dx[:, at], ref.scaled(total.cpu().numpy(), host(s)[:, None], np.float32(1.0)), torch.bfloat16)
    v = (d.float() * tokens.scales[:, None])[:, pick]
    s = (v.abs().amax(0).double() / 32639).float()
    n = (v.double() / s.double()[None, :]).round()
    near = (n.t() @ tokens.values[:, :cols].double()) * s.double()[:, None]
    # two sums as floats, their sum, the scale: four roundings
    size = 256 * ((n.abs() / 256).ceil().t() @ tokens.values[:, :cols].double().abs()) * s.double()[:, None]
    assert ((dw[pick].double() - near).abs() <= 4 * U * size).all()


def test_example(dev):
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "eight_bit_block.py")
    spec = importlib.util.spec_from_file_location("eight_bit_block", path)
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)
    params = block.parameters(48, 64, dev)
    x = torch.randn(20, 48, device=dev, dtype=torch.bfloat16)
    out, kept = block.forward(params, x)
    grads = block.backward(params, torch.ones_like(out), kept)
    assert [tuple(g.shape) for g in grads] == [(20, 48), (128, 48), (48, 64)]
    # The gradients of the same block in floats, in 64 bits: each factor of each sum was held to half of 1/127 of its
    # row's (group's) largest, so a sum is off by at most a few hundredths of what its parts could add up to.
    want, sizes = block.float_gradients(params, x, torch.ones_like(out))
    for g, w, s in zip(grads, want, sizes):
        assert ((g.double() - w).abs() <= 0.05 * s).all()
    eager, replayed = block.decode(params, 3, dev)
    assert torch.equal(eager, replayed) and bool(torch.isfinite(eager).all())
