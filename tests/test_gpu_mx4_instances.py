"""Every kernel instance of the 4-bit products and of the expert layer against
the 64-bit reference, past one chunk of K and at ragged edges.  The cases, and
which instance each takes, stand in mx4_instances.py and are checked against
the built library in test_mx4_instances.py.

Tolerances as in test_gpu_mx4.py: n 2^-23 sum |a b| for sums of n exact
products, half a step of the result's type.
"""
import mx4_instances as inst
import numpy as np
import pytest
import torch

import fp32_sgemm_f32_amd as sg
from oracle import mx4 as ref
from test_gpu_mx4 import close, dev, host, normal, product_bound, random_mx4, strided, typed, values  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cus(dev):  # noqa: F811
    assert torch.cuda.get_device_properties(dev).multi_processor_count == inst.CUS, "the cases are made for 256 CUs"


@pytest.fixture(scope="module")
def operands(dev):  # noqa: F811
    """The factors of a product and their product in 64 bits, made once for all types."""
    made = {}

    def of(m, n, k):
        if (m, n, k) not in made:
            made.clear()
            rng = np.random.default_rng(m + n + k)
            a, b = random_mx4(rng, m, k, dev), random_mx4(rng, n, k, dev)
            A, B = values(a), values(b)
            made[m, n, k] = a, b, A @ B.T, product_bound(A, B)
        return made[m, n, k]

    return of


@typed
@pytest.mark.parametrize("m, n, k", inst.GEMMS)
def test_gemm(dev, operands, dtype, m, n, k):  # noqa: F811
    a, b, want, bound = operands(m, n, k)
    got = sg.mx4_gemm(a, b, dtype=dtype)
    close(got, want, bound, dtype)
    assert torch.equal(sg.mx4_gemm(a, b, dtype=dtype), got)


@typed
@pytest.mark.parametrize("m, n, k", inst.ADDING)
def test_gemm_adds_to_a_strided_result(dev, operands, dtype, m, n, k):  # noqa: F811
    a, b, product, bound = operands(m, n, k)
    gen = torch.Generator(device=dev)
    gen.manual_seed(k)
    c = strided(torch.randn(m, n, generator=gen, device=dev).to(dtype), 3, 1)
    C = host(c)
    beside = torch.isnan(c._base)
    assert sg.mx4_gemm(a, b, out=c, alpha=-0.5, beta=2.0) is c
    close(c, 2.0 * C - 0.5 * product, 0.5 * bound + 2.0 ** -22 * (np.abs(0.5 * product) + np.abs(2.0 * C)), dtype)
    assert torch.equal(torch.isnan(c._base), beside), "written beside the matrix"


@pytest.mark.parametrize("m, n, k", inst.STEPS)
@typed
def test_train(dev, dtype, m, n, k):  # noqa: F811
    """Whole rows of the three results, from every tile of 64 rows and at the end."""
    gen = torch.Generator(device=dev)
    gen.manual_seed(m)
    x, w, dy = (torch.randn(s, generator=gen, device=dev).to(dtype) for s in ((m, k), (n, k), (m, n)))
    y, saved = sg.mx4_train_forward(x, w)
    dx, dw = sg.mx4_train_backward(dy, saved)
    rng = np.random.default_rng(n)
    r = ref.rounded
    for got, a, b, t in ((y, x, w, dtype), (dx, dy, w.t(), dtype), (dw, dy.t(), x.t(), torch.float32)):
        rows = a.shape[0]
        pick = np.unique(np.minimum(np.arange(0, rows, 64) + rng.integers(0, 64, -(-rows // 64)), rows - 1))
        pick = np.union1d(pick, [0, rows - 1])
        at = torch.from_numpy(pick).to(dev)
        A, B = r(host(a[at])), r(host(b))
        close(got[at], A @ B.T, product_bound(A, B), t)


@typed
@pytest.mark.parametrize("m", inst.LINEAR_TOKENS)
@pytest.mark.parametrize("k", inst.LINEAR_COLS)
def test_linear(dev, dtype, m, k):  # noqa: F811
    rng = np.random.default_rng(m + k)
    n = 333
    x, w = normal(rng, m, k, dtype, dev), random_mx4(rng, n, k, dev)
    X, W = host(x), values(w)
    got = sg.mx4_linear(x, w)
    close(got, X @ W.T, product_bound(X, W, 3), dtype)
    assert torch.equal(sg.mx4_linear(x, w), got)


@pytest.mark.parametrize("dtype, lo", [(torch.float32, 126), (torch.bfloat16, 126), (torch.float16, 14)], ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("m", inst.LINEAR_TOKENS)
def test_linear_largest_tokens(dev, dtype, lo, m):  # noqa: F811
    """Tokens up to the largest value of their type, where a first piece that were rounded would be infinite."""
    rng = np.random.default_rng(m)
    k = 300
    f = torch.finfo(dtype)
    x = torch.from_numpy((1 + rng.random((m, k))) * 2.0 ** lo * rng.choice([-2.0, -1.0, 1.0, 2.0], (m, k))).clamp(f.min, f.max).to(dtype).to(dev)
    x[0, ::7], x[0, 3::7] = f.max, f.min
    w = random_mx4(rng, 40, k, dev, 100, 110)
    X, W = host(x), values(w)
    assert np.isfinite(X).all()
    close(sg.mx4_linear(x, w), X @ W.T, product_bound(X, W, 3), dtype)


def check_experts(dev, dtype, tokens, top, hidden, inner):  # noqa: F811
    rng = np.random.default_rng(hidden + inner)
    experts = 7
    x, router = normal(rng, tokens, hidden, dtype, dev, 0.5), normal(rng, experts, hidden, dtype, dev, 1 / np.sqrt(hidden))
    up = random_mx4(rng, experts * 2 * inner, hidden, dev, 120, 124)
    down = random_mx4(rng, experts * hidden, inner, dev, 120, 124)
    norm = bool(rng.integers(2))
    want, bound = ref.moe(host(x), host(router), values(up).reshape(experts, 2 * inner, hidden),
                          values(down).reshape(experts, hidden, inner), top, norm, 22)
    got = sg.mx4_moe(x, router, up, down, top, norm=norm)
    close(got, want, bound, dtype)
    assert torch.equal(sg.mx4_moe(x, router, up, down, top, norm=norm), got)


@typed
@pytest.mark.parametrize("tokens, top", inst.EXPERT_TOKENS)
@pytest.mark.parametrize("hidden", inst.EXPERT_HIDDEN)
def test_experts_by_hidden(dev, dtype, tokens, top, hidden):  # noqa: F811
    check_experts(dev, dtype, tokens, top, hidden, 40)


@typed
@pytest.mark.parametrize("tokens, top", inst.EXPERT_TOKENS)
@pytest.mark.parametrize("inner", inst.EXPERT_INNER)
def test_experts_by_inner(dev, dtype, tokens, top, inner):  # noqa: F811
    check_experts(dev, dtype, tokens, top, 48, inner)
