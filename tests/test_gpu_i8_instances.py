"""Every choice of kernel that the 8-bit products make, by sizes that reach it on 256 compute units, against exact sums:
whole and ragged tiles, every type, with and without an old result."""
import numpy as np
import pytest
import torch

import fp32_sgemm_f32_amd as sg
from oracle import i8 as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
typed = pytest.mark.parametrize("dtype", TYPES, ids=["fp32", "bf16", "fp16"])


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    sg.library()
    return torch.device("cuda:0")


def random_i8(gen, rows, cols, dev):
    q = torch.zeros(rows, ref.padded(cols), dtype=torch.int8, device=dev)
    q[:, :cols] = torch.randint(-127, 128, (rows, cols), generator=gen, device=dev, dtype=torch.int8)
    return sg.I8(q, torch.rand(rows, generator=gen, device=dev) + 0.5, rows, cols)


def scaled(total, sa, sb):
    """An exact sum as a float, times the smaller and then the larger scale."""
    less = sa < sb
    return total.float() * torch.where(less, sa, sb) * torch.where(less, sb, sa)


def want(a, b):
    total = a.values[:, :a.shape[1]].double() @ b.values[:, :a.shape[1]].double().t()
    sa, sb = torch.broadcast_tensors(a.scales[:, None], b.scales[None, :])
    return scaled(total, sa, sb)


# tiles of 256 x 256; 256 x 128; 128 x 128 (two workgroups on a CU, or a deep ring); 64 x 64; 64 x 32 and 32 x 32 (two sets of waves)
# ... and grids of tiles that are cut into a part for each XCD
PRODUCTS = [(4096, 4096, 256), (8192, 8190, 300), (8700, 8900, 130), (4100, 4090, 130), (4352, 7600, 129), (2100, 2500, 130), (2176, 2560, 384), (2048, 4096, 256), (3000, 3010, 333), (1920, 6272, 130), (2048, 1100, 200), (2100, 1024, 640),
            (700, 1300, 333), (704, 1344, 256), (200, 300, 700), (64, 32, 128), (65, 33, 1290), (20, 300, 129), (9, 5000, 1000), (300, 20, 520),
            (32, 64, 256), (5000, 31, 140)]


@typed
@pytest.mark.parametrize("m, n, k", PRODUCTS)
def test_product(dev, dtype, m, n, k):
    gen = torch.Generator(device=dev)
    gen.manual_seed(m + n + k)
    a, b = random_i8(gen, m, k, dev), random_i8(gen, n, k, dev)
    exact = want(a, b)
    got = sg.i8_gemm(a, b, dtype=dtype)
    assert torch.equal(got, exact.to(dtype))
    wide = torch.full((m, n + 3), float("nan"), dtype=dtype, device=dev)
    out = wide[:, 1:n + 1]
    sg.i8_gemm(a, b, out=out)
    assert torch.equal(out, exact.to(dtype)) and int(wide.isnan().sum()) == 3 * m + int(out.isnan().sum())
    # into an old result: twice, and away again
    sg.i8_gemm(a, b, out=got, alpha=-2.0 ** -20, beta=0.0)
    first = got.clone()
    sg.i8_gemm(a, b, out=got, alpha=2.0 ** -20, beta=1.0)
    assert torch.equal(first, (exact * -2.0 ** -20).to(dtype))
    assert (got.double() - (first.double() + exact.double() * 2.0 ** -20)).abs().max() <= torch.finfo(dtype).eps * first.double().abs().max()


# one to eight waves that share rows, two or four eights of rows a wave, rows or columns few
THIN = [(m, n, k) for m in (1, 3, 8) for n, k in ((40, 100), (17, 300), (333, 600), (1000, 1500), (9001, 260), (8200, 1100))]


@typed
@pytest.mark.parametrize("m, n, k", THIN)
def test_few_rows(dev, dtype, m, n, k):
    gen = torch.Generator(device=dev)
    gen.manual_seed(m + n + k)
    a, b = random_i8(gen, m, k, dev), random_i8(gen, n, k, dev)
    exact = want(a, b)
    assert torch.equal(sg.i8_gemm(a, b, dtype=dtype), exact.to(dtype))
    assert torch.equal(sg.i8_gemm(b, a, dtype=dtype), exact.t().to(dtype))
    x = torch.randn(m, k, generator=gen, device=dev).to(dtype)
    assert torch.equal(sg.i8_linear(x, b), want(sg.i8_quantize(x), b).to(dtype))


@pytest.mark.parametrize("m, n, k", [(1, 16500, 8192), (3, 40000, 4096), (1, 700, 16384), (1, 600, 16400), (4, 500, 4096), (5, 500, 4096)])
def test_linear_where_its_choice_changes(dev, m, n, k):
    """Weights beyond 128 MiB, and tokens up to and beyond what every workgroup quantises for itself."""
    gen = torch.Generator(device=dev)
    gen.manual_seed(m)
    w = random_i8(gen, n, k, dev)
    x = torch.randn(m, k, generator=gen, device=dev).bfloat16()
    assert torch.equal(sg.i8_linear(x, w), want(sg.i8_quantize(x), w).bfloat16())


# The backward products: both in tiles of 256 x 256, of 128 x 128, in small ones (two or three workgroups on a CU), and
# apart in each size
TRAINS = [(4096, 2048, 4096), (4200, 2100, 4100), (2100, 1100, 2500), (4096, 300, 4096), (100, 2048, 4096), (100, 1100, 2500), (300, 2048, 4096),
          (20, 2048, 4096), (600, 2048, 4096), (1500, 2048, 4096), (700, 513, 900), (333, 1000, 1536), (4096, 100, 4096), (1000, 1000, 3000),
          (20, 30, 40), (2100, 700, 5000), (9, 4097, 130), (4097, 9, 130), (2500, 4100, 33), (2000, 500, 2000), (200, 600, 3000), (1024, 1024, 1024), (1000, 800, 4000)]


@pytest.mark.parametrize("m, n, k", TRAINS)
@pytest.mark.parametrize("dtype", TYPES[:2], ids=["fp32", "bf16"])
def test_backward(dev, dtype, m, n, k):
    gen = torch.Generator(device=dev)
    gen.manual_seed(m + n + k)
    x, w = random_i8(gen, m, k, dev), random_i8(gen, n, k, dev)
    d = torch.randn(m, n, generator=gen, device=dev).to(dtype)
    old = torch.randn(n, k, generator=gen, device=dev)
    dx, dw = sg.i8_train_backward(d, (x, w))
    _, again = sg.i8_train_backward(d, (x, w), dW=old.clone())

    def whole(v, levels):
        s = (v.abs().amax(1, keepdim=True).double() / levels).float()
        return (v.double() / s.double()).round(), s

    one = torch.ones(1, 1, device=dev)
    q, s = whole(d.float() * w.scales[None, :], 127)
    assert torch.equal(dx, scaled(q @ w.values[:, :k].double(), *torch.broadcast_tensors(s, one)).to(dtype))
    q, s = whole((d.float() * x.scales[:, None]).t(), 32639)
    high = ((q + 128) / 256).floor()
    xq = x.values[:, :k].double()
    parts = 256.0 * (high @ xq).float().double() + ((q - 256 * high) @ xq).float().double()
    exact = scaled(parts, *torch.broadcast_tensors(s, one))
    assert torch.equal(dw, exact)
    # added to what was there: one rounding
    assert ((again.double() - (exact.double() + old.double())).abs() <= np.ldexp(1.0, -24) * (exact.double() + old.double()).abs() + 1e-45).all()
