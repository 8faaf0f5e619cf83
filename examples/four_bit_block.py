"""The 4-bit calls as a program uses them: train a layer, then serve it.

    python examples/four_bit_block.py [--steps 60] [--tokens 16]

1. A layer W (N x K) learns a teacher's map by gradient descent; the three
   products of every step run on 4-bit operands (mx4_train_forward and
   mx4_train_backward), the weights themselves stay in float32.
2. The trained weights are quantised once (mx4_quantize) and serve single
   tokens (mx4_linear).
3. A small stack of expert layers with 4-bit experts (mx4_moe) carries a token
   through a few steps, captured once as a graph and replayed.

Synthetic data, random weights.  Prints what each part reached.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp32_sgemm_f32_amd as sg  # noqa: E402


def train(steps, device, batch=512, n=384, k=640, rate=0.2):
    """(trained weights, first loss, last loss) of a layer that learns a teacher's map."""
    gen = torch.Generator(device=device)
    gen.manual_seed(0)
    teacher = torch.randn(n, k, generator=gen, device=device) / k ** 0.5
    W = torch.zeros(n, k, device=device)
    losses = []
    for _ in range(steps):
        X = torch.randn(batch, k, generator=gen, device=device).bfloat16()
        Y, saved = sg.mx4_train_forward(X, W, rule="noclip")
        miss = Y.float() - sg.matmul(X.float(), teacher.t())
        losses.append(float(miss.square().mean()))
        _, dW = sg.mx4_train_backward((miss / batch).bfloat16(), saved)
        W -= rate * dW
    return W, losses[0], losses[-1]


def serve(W, tokens, device):
    """How far one token at a time on 4-bit weights is from the float product, relative to its size."""
    gen = torch.Generator(device=device)
    gen.manual_seed(1)
    q = sg.mx4_quantize(W, rule="noclip")
    far = size = 0.0
    for _ in range(tokens):
        x = torch.randn(1, W.shape[1], generator=gen, device=device).bfloat16()
        y, exact = sg.mx4_linear(x, q).double(), x.double() @ W.double().t()
        far, size = far + float((y - exact).square().sum()), size + float(exact.square().sum())
    return (far / size) ** 0.5


class ExpertStack:
    """Layers x + experts(x / rms(x)) with 4-bit experts."""

    def __init__(self, layers, experts, top, hidden, inner, device):
        gen = torch.Generator(device=device)
        gen.manual_seed(2)

        def weights(rows, cols, *shape):
            return torch.randn(*shape, rows, cols, generator=gen, device=device) / cols ** 0.5

        self.top = top
        self.layers = [(weights(experts, hidden).bfloat16(),
                        sg.mx4_quantize(weights(2 * inner, hidden, experts).flatten(0, 1)),
                        sg.mx4_quantize(weights(hidden, inner, experts).flatten(0, 1))) for _ in range(layers)]

    def __call__(self, x):
        for router, up, down in self.layers:
            rms = x.float().square().mean(1, keepdim=True).add(1e-6).rsqrt()
            x = x + sg.mx4_moe((x * rms).bfloat16(), router, up, down, self.top)
        return x


def decode(tokens, device, steps=4):
    """The stack's output for `tokens` tokens, eagerly and from a replayed graph."""
    stack = ExpertStack(3, 16, 4, 512, 256, device)
    gen = torch.Generator(device=device)
    gen.manual_seed(3)
    x = torch.randn(tokens, 512, generator=gen, device=device).bfloat16()
    stack(x)                                     # the first call loads the kernels
    torch.cuda.synchronize()
    graph, static = torch.cuda.CUDAGraph(), x.clone()
    with torch.cuda.graph(graph):
        out = stack(static)
    eager, replayed = x, x
    for _ in range(steps):
        eager = stack(eager)
        static.copy_(replayed)
        graph.replay()
        replayed = out.clone()
    return eager, replayed


def main():
    args = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    args.add_argument("--steps", type=int, default=60)
    args.add_argument("--tokens", type=int, default=16)
    args = args.parse_args()
    device = torch.device("cuda:0")
    W, first, last = train(args.steps, device)
    print(f"training in 4 bits: loss {first:.4f} -> {last:.4f} in {args.steps} steps")
    print(f"served in 4 bits: {serve(W, args.tokens, device):.3f} of the float product's size away")
    eager, replayed = decode(args.tokens, device)
    print(f"expert stack, {args.tokens} tokens: graph and eager calls {'agree' if torch.equal(eager, replayed) else 'DIFFER'}, "
          f"rms {float(eager.float().square().mean().sqrt()):.3f}")


if __name__ == "__main__":
    main()
