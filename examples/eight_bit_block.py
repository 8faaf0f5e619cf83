"""A gated block in 8 bits: y = silu(x G^T) * (x U^T), z = y D^T.

  train   forward and backward with i8_train_forward / i8_train_backward and
          i8_swiglu_forward / i8_swiglu_backward: what is kept between the
          passes is a byte a value, and the master weights stay in fp32
  serve   weights quantised once, tokens one at a time with i8_linear, the step
          recorded into a graph and replayed

    python examples/eight_bit_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp32_sgemm_f32_amd as sg  # noqa: E402


def parameters(hidden, inner, dev, seed=0):
    """[G; U] (2 inner x hidden) and D (hidden x inner), in fp32."""
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    return [torch.randn(2 * inner, hidden, generator=gen, device=dev) * hidden ** -0.5,
            torch.randn(hidden, inner, generator=gen, device=dev) * inner ** -0.5]


def forward(params, x):
    """z and the 8-bit checkpoint."""
    gu, first = sg.i8_train_forward(x, params[0])
    h, gate = sg.i8_swiglu_forward(gu)
    z, second = sg.i8_train_forward(h, params[1])
    return z, (first, gate, second)


def backward(params, dz, kept):
    """Gradients of x, [G; U] and D."""
    first, gate, second = kept
    dh, dd = sg.i8_train_backward(dz, second)
    dgu = sg.i8_swiglu_backward(dh, gate)
    dx, dw = sg.i8_train_backward(dgu, first)
    return dx, dw, dd


def float_gradients(params, x, dz):
    """The same gradients of the block in 64-bit floats, and for each the sum of the magnitudes of its parts, every
    factor as large as the largest that shares its scale."""
    w, d = (p.double().requires_grad_() for p in params)
    x64 = x.double().requires_grad_()
    g, u = (x64 @ w.t()).chunk(2, 1)
    h = g * torch.sigmoid(g) * u
    z = h @ d.t()
    grads = torch.autograd.grad(z, (x64, w, d), dz.double())
    row = lambda t: t.detach().abs().amax(1, keepdim=True).expand_as(t)
    dh = row(dz.double()) @ row(d)
    dgu = torch.cat([dh * (1 + row(u)) * 1.1, dh * (1 + row(g))], 1)
    dgu = row(dgu)
    return grads, (dgu @ row(w), dgu.t() @ row(x64), row(dz.double()).t() @ row(h))


def train(steps, dev, rate=0.05):
    """Mean squared distance to a fixed block's outputs, first and last."""
    params, target = parameters(256, 512, dev, 0), parameters(256, 512, dev, 1)
    first = last = None
    for step in range(steps):
        gen = torch.Generator(device=dev)
        gen.manual_seed(100 + step)
        x = torch.randn(512, 256, generator=gen, device=dev).bfloat16()
        g, u = (x.float() @ target[0].t()).chunk(2, 1)
        want = (g * torch.sigmoid(g) * u) @ target[1].t()
        z, kept = forward(params, x)
        error = z.float() - want
        last = float((error * error).mean())
        first = last if first is None else first
        _, dw, dd = backward(params, (error * (2.0 / x.shape[0])).bfloat16(), kept)
        params[0] -= rate * dw
        params[1] -= rate * dd
    return first, last


def serve(weights, x):
    """One step of a served block, weights in 8 bits."""
    gu, d = weights
    h, _ = sg.i8_swiglu_forward(sg.i8_linear(x, gu))
    return sg.i8_linear(h, d)


def decode(params, tokens, dev):
    """Tokens one after another, eagerly and by replaying a graph of one step."""
    weights = [sg.i8_quantize(p) for p in params]
    gen = torch.Generator(device=dev)
    gen.manual_seed(7)
    xs = torch.randn(tokens, 1, params[0].shape[1], generator=gen, device=dev).bfloat16()
    eager = torch.cat([serve(weights, x) for x in xs])
    slot = xs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = serve(weights, slot)
    replayed = []
    for x in xs:
        slot.copy_(x)
        graph.replay()
        replayed.append(out.clone())
    return eager, torch.cat(replayed)


def main():
    dev = torch.device("cuda:0")
    first, last = train(100, dev)
    print(f"trained in 8 bits: mean squared error {first:.4f} -> {last:.4f}")
    eager, replayed = decode(parameters(1024, 2048, dev), 8, dev)
    print(f"served 8 tokens, graph and eager agree: {bool(torch.equal(eager, replayed))}")


if __name__ == "__main__":
    main()
