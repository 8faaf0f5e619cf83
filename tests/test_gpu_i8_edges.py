"""Edges of the 8-bit integer operators on the GPU against the 64-bit reference: gates whose exponential leaves fp32's
range while the result does not, and matrices without columns."""
import numpy as np
import pytest
import torch

import fp32_sgemm_f32_amd as sg
from oracle import i8 as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24      # half a step of fp32, relatively


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    sg.library()
    return torch.device("cuda:0")


def host(t):
    return t.detach().cpu().double().numpy()


def within(got, want, bound):
    """got within bound of want, plus half a step of fp32."""
    got, lim = host(got), bound + np.maximum(U * (np.abs(want) + bound), 2.0 ** -150)
    bad = ~(np.abs(got - want) <= lim)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: {got[bad][0]} against {want[bad][0]}"


def far_gates():
    """Gates of -80 to -200, whose exp is between 2e-35 and nothing, a group of 128 columns for each size of u and dh:
    (G, u, dh), where u and dh are a power of two for each group."""
    rows, sizes = 24, [(0, 0), (20, 0), (60, -20), (100, 3), (126, 0), (0, 100), (126, 126), (-60, 126), (126, -100), (70, 70)]
    rng = np.random.default_rng(40)
    top = -np.linspace(81, 200, rows)[:, None]
    g = (top * (1 - 0.03 * rng.random((rows, 128 * len(sizes))))).astype(np.float32)
    sign = lambda: rng.choice([-1.0, 1.0], g.shape)
    u, d = (sign() * np.repeat(np.ldexp(1.0, [p[i] for p in sizes]), 128)[None, :] for i in (0, 1))
    return g, u.astype(np.float32), d.astype(np.float32)


def test_swiglu_keeps_what_far_gates_leave(dev):
    """exp(g) is below fp32's least normal number from g = -87.3 on, exp(-g) infinite from -88.7 on; times g, u (and dh)
    the results need not be small.  exp(g / 2) enters twice, each off by two halves of a step, and the result is rounded
    once (`within`); up to -87 the quotient's form: two, and four of its sums and products.  Below -174.6 exp(g / 2) lies
    under the least normal number too: off by 2^-150, which its square takes twice, times at most 2^-126."""
    g, u, d = far_gates()
    h, saved = sg.i8_swiglu_forward(torch.from_numpy(np.concatenate((g, u), 1)).to(dev))
    G, V, D = (x.astype(np.float64) for x in (g, u, d))
    lost = 2.0 ** -275
    want = G * np.exp(G) / (1 + np.exp(G)) * V
    within(h, want, 7 * U * np.abs(want) + np.abs(G * V) * lost + 2.0 ** -149)
    # The gradient, at the values that the checkpoint holds.  (The formula's five more roundings, for gates up to -87.)
    G, V = (ref.values(host(q.values), host(q.scales), g.shape[1]).astype(np.float64) for q in saved)
    assert G.min() < -190 and (G > -87).sum() > 100
    p = np.exp(G) / (1 + np.exp(G))
    dg, du = D * V * p * (1 + G / (1 + np.exp(G))), D * G * p
    # Up to -87 a product of dh and u in fp32 comes first: not beyond its largest number.
    inside = (G < -87) | (np.abs(D * V) < 2.0 ** 127)
    grad = sg.i8_swiglu_backward(torch.from_numpy(d).to(dev), saved)
    n = g.shape[1]
    # (what reaches fp32's largest number is infinite)
    clip = np.where(inside & (np.abs(dg) < 2.0 ** 127), dg, 0.0)
    part = torch.where(torch.from_numpy(inside & (np.abs(dg) < 2.0 ** 127)).to(dev), grad[:, :n], torch.zeros((), device=dev))
    within(part, clip, 14 * U * np.abs(clip) + np.abs(D * V * (1 + G)) * lost + 2.0 ** -148)
    within(grad[:, n:], du, 8 * U * np.abs(du) + np.abs(D * G) * lost + 2.0 ** -148)
    assert ((np.abs(want) > 2.0 ** -126) & (G < -100)).sum() > 500 and ((np.abs(dg) > 2.0 ** -126) & (G < -100)).sum() > 500


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_swiglu_far_gates_of_16_bits(dev, dtype):
    g = torch.linspace(-200, -80, 512).to(dtype).view(4, 128).to(dev)
    u = torch.full((4, 128), torch.finfo(dtype).max / 2, dtype=dtype, device=dev)
    h, _ = sg.i8_swiglu_forward(torch.cat((g, u), 1))
    G, V = host(g), host(u)
    want = G * np.exp(G) / (1 + np.exp(G)) * V
    f = torch.finfo(dtype)
    lim = 7 * U * np.abs(want) + np.abs(G * V) * 2.0 ** -275 + 2.0 ** -149
    lim = lim + np.maximum((np.abs(want) + lim) * (f.eps / 2), f.smallest_normal * f.eps / 2)
    assert (np.abs(host(h) - want) <= lim).all()


def test_scales_of_matrices_without_columns(dev):
    """The largest magnitude of nothing is 0, so the scale is the least one: not what the memory held before."""
    floor = 2.0 ** -126

    def check(q, rows):
        assert q.values.shape == (rows, 0) and q.scales.shape == (rows,) and q.group is None
        assert torch.equal(q.scales, torch.full((rows,), floor, device=dev))

    side = torch.cuda.Stream()
    for stream in (None, side):
        for rows in (1, 5, 100):
            x, w = torch.ones(rows, 0, device=dev), torch.ones(7, 0, device=dev, dtype=torch.bfloat16)
            with torch.cuda.stream(stream or torch.cuda.current_stream()):      # memory that held something else
                dirty = [torch.full((128,), float("nan"), device=dev) for _ in range(8)]
                del dirty
            torch.cuda.synchronize()
            q = sg.i8_quantize(x, stream=stream)
            _, saved = sg.i8_train_forward(x, w, stream=stream)
            _, given = sg.i8_train_forward(x, sg.i8_quantize(w, stream=stream), stream=stream)
            torch.cuda.synchronize()
            check(q, rows), check(saved[0], rows), check(saved[1], 7), check(given[0], rows), check(given[1], 7)
            assert sg.i8_quantize(x, group=128).scales.shape == (rows, 0)
            back = sg.I8(q.values, q.scales, rows, 0)
            assert torch.equal(sg.i8_gemm(back, given[1]), torch.zeros(rows, 7, device=dev))


def test_scales_without_columns_in_a_graph(dev):
    x = torch.ones(5, 0, device=dev)
    sg.i8_quantize(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = sg.i8_quantize(x)
    scales = q.scales
    for _ in range(3):
        scales.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert scales.eq(2.0 ** -126).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("inner", [1, 13, 130])
def test_swiglu_far_gates_of_ragged_strided_rows(dev, dtype, inner):
    """Far gates beside near ones, at the end of rows that lie apart: nothing between the rows is written."""
    rows, rng = 5, np.random.default_rng(41)
    g = np.where(rng.random((rows, inner)) < 0.5, -95.0 - 8 * rng.random((rows, inner)), rng.standard_normal((rows, inner)))
    g[:, -1] = -100.0
    x = torch.from_numpy(np.concatenate((g, np.full_like(g, 2.0 ** 100)), 1)).to(dtype).to(dev)
    d = torch.from_numpy(rng.standard_normal((rows, inner)) * 2.0 ** -20).to(dtype).to(dev)

    def apart(cols):
        return torch.full((rows, cols + 3), float("nan"), dtype=dtype, device=dev)[:, 1:1 + cols]

    h, out = apart(inner), apart(2 * inner)
    _, saved = sg.i8_swiglu_forward(x, out=h)
    sg.i8_swiglu_backward(d, saved, out=out)
    for t in (h, out):
        assert int(t._base.isnan().sum()) == 3 * rows
    f = torch.finfo(dtype)

    def near(got, want, bound):
        lim = bound + np.maximum((np.abs(want) + bound) * (f.eps / 2), f.smallest_normal * f.eps / 2)
        assert (np.abs(host(got) - want) <= lim).all()

    G, V, D = host(x)[:, :inner], host(x)[:, inner:], host(d)
    want = ref.gated(G, V)
    near(h, want, 7 * U * np.abs(want) + 2.0 ** -149)
    G, V = (ref.values(host(q.values), host(q.scales), inner).astype(np.float64) for q in saved)
    dg, du = ref.gated_backward(D, G, V)
    p = ref.sigmoid(G)
    near(out[:, :inner], dg, 14 * U * np.abs(D * V * p) * (1.0 + np.abs(G) * ref.sigmoid(-G)) + 2.0 ** -148)
    near(out[:, inner:], du, 8 * U * np.abs(du) + 2.0 ** -148)
    assert (np.abs(dg[:, -1]) > 2.0 ** -126).all() and (np.abs(want[:, -1]) > 2.0 ** -126).all()
