"""The choices of kernel that test_gpu_i8_instances.py leaves out, against exact sums: its training steps in fp16, more of
them in every type, prompts of up to 8192 rows, many tiles by column, and the longest sum of a weights' gradient."""
import i8_instances as inst
import numpy as np
import pytest
import test_gpu_i8_instances as cases
import torch

import fp32_sgemm_f32_amd as sg

pytestmark = pytest.mark.gpu

typed = pytest.mark.parametrize("dtype", cases.TYPES, ids=["fp32", "bf16", "fp16"])


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    sg.library()
    return torch.device("cuda:0")


@pytest.mark.parametrize("m, n, k", cases.TRAINS)
def test_backward_of_fp16(dev, m, n, k):
    cases.test_backward(dev, torch.float16, m, n, k)


@typed
@pytest.mark.parametrize("m, n, k", inst.STEPS)
def test_backward(dev, dtype, m, n, k):
    cases.test_backward(dev, dtype, m, n, k)


@typed
@pytest.mark.parametrize("m, n, k", inst.PROMPTS)
def test_linear_of_prompts(dev, dtype, m, n, k):
    gen = torch.Generator(device=dev)
    gen.manual_seed(m)
    x, w = torch.randn(m, k, generator=gen, device=dev).to(dtype), cases.random_i8(gen, n, k, dev)
    q = sg.i8_quantize(x)
    s = (x.double().abs().amax(1) / 127).float()
    assert torch.equal(q.scales, s) and torch.equal(q.values[:, :k].double(), (x.double() / s.double()[:, None]).round())
    assert torch.equal(sg.i8_linear(x, w), cases.want(q, w).to(dtype))


@typed
@pytest.mark.parametrize("rows, cols", inst.COLUMNS)
def test_quantize_by_column(dev, dtype, rows, cols):
    gen = torch.Generator(device=dev)
    gen.manual_seed(rows)
    x = torch.randn(rows, cols, generator=gen, device=dev).to(dtype)
    q = sg.i8_quantize(x.t())
    s = (x.double().abs().amax(0) / 127).float()
    assert q.shape == (cols, rows) and torch.equal(q.scales, s) and not q.values[:, rows:].any()
    assert torch.equal(q.values[:, :rows].double(), (x.double() / s.double()).round().t())


def test_weights_gradient_of_the_longest_sum(dev):
    """131072 tokens: 16-bit numbers whose high byte is 127 and whose low byte is 127 or -128, against 127 and -127, so
    that both parts' sums come to within two parts in a hundred of 2^31, in both signs."""
    m, n, k = 1 << 17, 5, 130
    near, most = 256 * 127 - 128, 32639
    d = torch.full((m, n), float(near), device=dev)         # low byte -128
    d[:, 1] = -float(near - 256)                            # and -126: -128 with it, of negative numbers
    d[1::2, 2] = -float(near)
    d[:, 3] = float(most)                                   # low byte 127
    d[0], d[0, 1] = float(most), -float(most)               # the scale of every channel is 1
    d[:, 4] = torch.randint(-most, most + 1, (m,), device=dev).float()
    d[0, 4] = float(most)
    x = torch.full((m, 256), 127, dtype=torch.int8, device=dev)
    x[:, 1::3] = -127
    x[1::2, 2::3] = -127
    x[:, k:] = 0
    w = sg.I8(torch.ones(n, 256, dtype=torch.int8, device=dev).index_fill_(1, torch.arange(k, 256, device=dev), 0), torch.ones(n, device=dev), n, k)
    _, dw = sg.i8_train_backward(d, (sg.I8(x, torch.ones(m, device=dev), m, k), w))
    q, xq = d.t().double(), x[:, :k].double()
    high = ((q + 128) / 256).floor()
    low = q - 256 * high
    sums = [high @ xq, low @ xq]
    assert all(0.98 * 2.0 ** 31 < float(v) < 2.0 ** 31 for s in sums for v in (s.max(), -s.min()))
    parts = 256.0 * sums[0].float().double() + sums[1].float().double()
    assert np.array_equal(dw.cpu().numpy(), parts.float().cpu().numpy())
