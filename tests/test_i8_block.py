"""What the gradient check of the gated block takes and what it refuses (no GPU), and the example's own gradients."""
import i8_block
import pytest
import torch

SIZES = [(20, 48, 64), (33, 128, 96)]      # tokens, hidden, inner


def inputs(block, tokens, hidden, inner, dev):
    gen = torch.Generator()
    gen.manual_seed(tokens)
    x, dz = torch.randn(tokens, hidden, generator=gen), torch.randn(tokens, hidden, generator=gen) * 0.1
    params = block.parameters(hidden, inner, torch.device("cpu"))
    return [p.to(dev) for p in params], x.bfloat16().to(dev), dz.bfloat16().to(dev)


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_check_takes_rounding_and_refuses_mistakes(size):
    block = i8_block.example()
    params, x, dz = inputs(block, *size, "cpu")
    want = block.float_gradients(params, x, dz)[0]
    got = i8_block.eight_bit(params, x, dz)
    assert all(i8_block.near(got, want)), i8_block.distances(got, want)
    dx, dw, dd = got
    half = dw.shape[0] // 2
    for wrong in ([torch.zeros_like(g) for g in got], [-g for g in got], [g * 127 for g in got], [g * 0.9 for g in got],
                  [dx.roll(1, 0), torch.cat((dw[half:], dw[:half])), dd.roll(1, 1)]):
        assert not any(i8_block.near(wrong, want))
    # without the slope's second term G's gradient is wrong, and x's
    assert i8_block.near(i8_block.eight_bit(params, x, dz, slope=False), want) == [False, False, True]


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_example_gradients(size):
    block = i8_block.example()
    params, x, dz = inputs(block, *size, torch.device("cuda:0"))
    out, kept = block.forward(params, x)
    got = block.backward(params, dz, kept)
    want = block.float_gradients(params, x, dz)[0]
    assert out.dtype == x.dtype and [g.shape for g in got] == [w.shape for w in want]
    assert all(i8_block.near(got, want)), i8_block.distances(got, want)
