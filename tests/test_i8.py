"""The 8-bit integer operators on the host: sizes of the format, refusals of the C
entry points before anything touches the GPU, refusals of the Python calls, and
the reference itself at the format's edges."""
import ctypes

import numpy as np
import pytest
import torch

import fp32_sgemm_f32_amd as sg
from oracle import i8 as ref

P = 1 << 20      # addresses that no check may follow
FAR = 1 << 40


def lib():
    return sg.library()


@pytest.mark.parametrize("rows, cols", [(0, 0), (1, 1), (31, 128), (32, 129), (33, 4096), (1 << 22, 4096), (0, 5), (5, 0)])
@pytest.mark.parametrize("group", [0, 128])
def test_sizes_of_the_arrays(rows, cols, group):
    v, s = ctypes.c_longlong(), ctypes.c_longlong()
    assert lib().sgemm_f32_i8_bytes(rows, cols, group, ctypes.byref(v), ctypes.byref(s)) == sg.OK
    assert v.value == rows * ref.padded(cols)
    assert s.value == 4 * rows * (ref.padded(cols) // 128 if group else min(cols, 1))
    assert lib().sgemm_f32_i8_bytes(rows, cols, group, None, None) == sg.OK


def test_sizes_out_of_range():
    for rows, cols in ((-1, 1), (1, -1), ((1 << 22) + 1, 1), (1, (1 << 22) + 1), (1 << 22, 4097), (1 << 22, 1 << 22)):
        assert lib().sgemm_f32_i8_bytes(rows, cols, 0, None, None) == sg.ERR_SHAPE
    assert lib().sgemm_f32_i8_bytes(4, 4, 64, None, None) == sg.ERR_CONFIG


def quantize(trans=0, rows=4, cols=128, group=0, type=0, X=P, ldx=128, q=P * 2, s=P * 3, scratch=None, nbytes=0):
    return lib().sgemm_f32_i8_quantize(trans, rows, cols, group, type, X, ldx, q, s, scratch, nbytes, None)


@pytest.mark.parametrize("status, args", [
    (sg.ERR_SHAPE, dict(rows=-1)), (sg.ERR_SHAPE, dict(cols=(1 << 22) + 1, ldx=1 << 23)),
    (sg.ERR_SHAPE, dict(trans=1, rows=1 << 21, cols=8193, ldx=1 << 21, scratch=FAR, nbytes=1 << 30)),
    (sg.ERR_CONFIG, dict(type=3)), (sg.ERR_CONFIG, dict(type=-1)), (sg.ERR_CONFIG, dict(group=32)), (sg.ERR_CONFIG, dict(trans=2)),
    (sg.ERR_CONFIG, dict(trans=1, group=128)),
    (sg.ERR_LD, dict(ldx=127)), (sg.ERR_LD, dict(trans=1, ldx=3)),
    (sg.ERR_NULL, dict(X=None)), (sg.ERR_NULL, dict(q=None)), (sg.ERR_NULL, dict(s=None)), (sg.ERR_NULL, dict(trans=1)),
    (sg.ERR_SCRATCH, dict(trans=1, scratch=FAR, nbytes=16)), (sg.ERR_ALIGN, dict(trans=1, scratch=FAR + 64, nbytes=1 << 20)),
    (sg.ERR_ALIAS, dict(trans=1, scratch=P * 2, nbytes=1 << 20)),
    (sg.ERR_ALIGN, dict(X=P + 2)), (sg.ERR_ALIGN, dict(q=P * 2 + 8)), (sg.ERR_ALIGN, dict(s=P * 3 + 2)),
    (sg.ERR_ALIGN, dict(type=1, X=P + 1)),
    (sg.ERR_ALIAS, dict(q=P)), (sg.ERR_ALIAS, dict(s=P * 2 + 16)),
])
def test_quantize_refuses(status, args):
    assert quantize(**args) == status


def test_quantize_scratch():
    n = ctypes.c_longlong()
    call = lib().sgemm_f32_i8_quantize_scratch
    assert call(0, 4, 4, ctypes.byref(n)) == sg.OK and n.value == 0
    assert call(1, 4, 4, ctypes.byref(n)) == sg.OK and n.value > 0
    assert call(1, 4, 4, None) == sg.ERR_NULL
    assert call(2, 4, 4, ctypes.byref(n)) == sg.ERR_CONFIG
    assert call(1, -1, 4, ctypes.byref(n)) == sg.ERR_SHAPE


def dequantize(rows=4, cols=128, group=0, q=P, s=P * 2, type=0, Y=P * 3, ldy=128):
    return lib().sgemm_f32_i8_dequantize(rows, cols, group, q, s, type, Y, ldy, None)


@pytest.mark.parametrize("status, args", [
    (sg.ERR_SHAPE, dict(rows=-1)), (sg.ERR_CONFIG, dict(type=7)), (sg.ERR_CONFIG, dict(group=1)), (sg.ERR_LD, dict(ldy=100)),
    (sg.ERR_NULL, dict(q=None)), (sg.ERR_NULL, dict(s=None)), (sg.ERR_NULL, dict(Y=None)),
    (sg.ERR_ALIGN, dict(q=P + 4)), (sg.ERR_ALIGN, dict(Y=P * 3 + 2)), (sg.ERR_ALIAS, dict(Y=P)),
])
def test_dequantize_refuses(status, args):
    assert dequantize(**args) == status


def gemm(M=4, N=4, K=128, alpha=1.0, a=P, sa=P * 2, b=P * 3, sb=P * 4, beta=0.0, type=0, C=P * 5, ldc=4):
    return lib().sgemm_f32_i8_gemm(M, N, K, alpha, a, sa, b, sb, beta, type, C, ldc, None)


@pytest.mark.parametrize("status, args", [
    (sg.ERR_SHAPE, dict(M=-1)), (sg.ERR_SHAPE, dict(N=-1)), (sg.ERR_SHAPE, dict(K=-1)), (sg.ERR_SHAPE, dict(K=(1 << 17) + 1)),
    (sg.ERR_CONFIG, dict(type=5)),
    (sg.ERR_LD, dict(ldc=3)), (sg.ERR_NULL, dict(a=None)), (sg.ERR_NULL, dict(sb=None)), (sg.ERR_NULL, dict(C=None)),
    (sg.ERR_NULL, dict(K=0, C=None)), (sg.ERR_ALIGN, dict(b=P * 3 + 8)), (sg.ERR_ALIGN, dict(sa=P * 2 + 1)),
    (sg.ERR_ALIAS, dict(C=P * 3)), (sg.ERR_ALIAS, dict(C=P * 2)),
])
def test_gemm_refuses(status, args):
    assert gemm(**args) == status


def linear(M=100, N=4, K=128, type=0, X=P, ldx=128, w=FAR, s=FAR * 2, Y=FAR * 3, ldy=4, scratch=FAR * 4, nbytes=1 << 20):
    return lib().sgemm_f32_i8_linear(M, N, K, type, X, ldx, w, s, Y, ldy, scratch, nbytes, None)


@pytest.mark.parametrize("status, args", [
    (sg.ERR_SHAPE, dict(M=-1)), (sg.ERR_SHAPE, dict(K=(1 << 17) + 1, ldx=1 << 23)), (sg.ERR_CONFIG, dict(type=3)),
    (sg.ERR_LD, dict(ldx=127)), (sg.ERR_LD, dict(ldy=3)), (sg.ERR_NULL, dict(X=None)), (sg.ERR_NULL, dict(w=None)),
    (sg.ERR_NULL, dict(Y=None)), (sg.ERR_NULL, dict(s=None)), (sg.ERR_ALIGN, dict(X=P + 1)), (sg.ERR_ALIGN, dict(w=FAR + 4)),
    (sg.ERR_ALIAS, dict(Y=P)), (sg.ERR_ALIAS, dict(Y=FAR)),
    # enough rows that their 8-bit form is written out
    (sg.ERR_NULL, dict(scratch=None)), (sg.ERR_SCRATCH, dict(nbytes=16)), (sg.ERR_ALIGN, dict(scratch=FAR * 4 + 64)),
    (sg.ERR_ALIAS, dict(scratch=FAR)),
])
def test_linear_refuses(status, args):
    assert linear(**args) == status


def test_linear_scratch():
    n = ctypes.c_longlong()
    call = lib().sgemm_f32_i8_linear_scratch
    assert call(100, 4, 128, 0, ctypes.byref(n)) == sg.OK and n.value > 0
    assert call(100, 4, 0, 0, ctypes.byref(n)) == sg.OK and n.value == 0
    assert call(4, 4, 128, 3, ctypes.byref(n)) == sg.ERR_CONFIG
    assert call(-1, 4, 128, 0, ctypes.byref(n)) == sg.ERR_SHAPE
    assert call(4, 4, 128, 0, None) == sg.ERR_NULL


def forward(M=4, N=8, K=128, type=0, X=FAR, ldx=128, type_w=0, W=FAR * 2, ldw=128, Y=FAR * 3, ldy=8, xq=FAR * 4, sx=FAR * 5, wq=FAR * 6,
            sw=FAR * 7):
    return lib().sgemm_f32_i8_train_forward(M, N, K, type, X, ldx, type_w, W, ldw, Y, ldy, xq, sx, wq, sw, None)


@pytest.mark.parametrize("status, args", [
    (sg.ERR_SHAPE, dict(M=-1)), (sg.ERR_SHAPE, dict(N=-1)), (sg.ERR_SHAPE, dict(K=-1)), (sg.ERR_SHAPE, dict(M=(1 << 17) + 1)),
    (sg.ERR_SHAPE, dict(N=(1 << 17) + 1)), (sg.ERR_SHAPE, dict(K=(1 << 17) + 1)), (sg.ERR_CONFIG, dict(type=3)),
    (sg.ERR_CONFIG, dict(type_w=3)), (sg.ERR_LD, dict(ldx=127)), (sg.ERR_LD, dict(ldw=127)),
    (sg.ERR_LD, dict(ldy=7)), (sg.ERR_NULL, dict(X=None)), (sg.ERR_NULL, dict(Y=None)), (sg.ERR_NULL, dict(sw=None)),
    (sg.ERR_ALIGN, dict(xq=FAR * 4 + 8)), (sg.ERR_ALIAS, dict(Y=FAR)), (sg.ERR_ALIAS, dict(xq=FAR * 6)),
])
def test_train_forward_refuses(status, args):
    assert forward(**args) == status


def backward(M=4, N=8, K=128, type=0, D=FAR, ldd=8, xq=FAR * 2, sx=FAR * 3, wq=FAR * 4, sw=FAR * 5, dX=FAR * 6, lddx=128,
             dW=FAR * 7, lddw=128, scratch=FAR * 8, nbytes=1 << 20):
    return lib().sgemm_f32_i8_train_backward(M, N, K, type, D, ldd, xq, sx, wq, sw, dX, lddx, 0.0, dW, lddw, scratch, nbytes, None)


@pytest.mark.parametrize("status, args", [
    (sg.ERR_SHAPE, dict(M=-1)), (sg.ERR_SHAPE, dict(M=(1 << 17) + 1)), (sg.ERR_CONFIG, dict(type=3)), (sg.ERR_LD, dict(ldd=7)),
    (sg.ERR_LD, dict(lddx=127)), (sg.ERR_LD, dict(lddw=127)), (sg.ERR_NULL, dict(D=None)), (sg.ERR_NULL, dict(dW=None)),
    (sg.ERR_NULL, dict(xq=None)), (sg.ERR_NULL, dict(sw=None)), (sg.ERR_NULL, dict(scratch=None)), (sg.ERR_ALIGN, dict(dW=FAR * 7 + 2)),
    (sg.ERR_ALIGN, dict(scratch=FAR * 8 + 16)), (sg.ERR_SCRATCH, dict(nbytes=100)), (sg.ERR_ALIAS, dict(dX=FAR * 7)),
    (sg.ERR_ALIAS, dict(dW=FAR)), (sg.ERR_ALIAS, dict(scratch=FAR * 4)),
])
def test_train_backward_refuses(status, args):
    assert backward(**args) == status


def test_train_scratch():
    n = ctypes.c_longlong()
    call = lib().sgemm_f32_i8_train_scratch
    assert call(4, 8, 128, ctypes.byref(n)) == sg.OK and n.value > 0
    assert call(0, 8, 128, ctypes.byref(n)) == sg.OK and n.value == 0
    assert call(4, 8, 128, None) == sg.ERR_NULL
    assert call(-1, 8, 128, ctypes.byref(n)) == sg.ERR_SHAPE


def gated(rows=4, inner=128, type=0, GU=FAR, ld=256, H=FAR * 2, ldh=128, g=FAR * 3, sg_=FAR * 4, u=FAR * 5, su=FAR * 6):
    return lib().sgemm_f32_i8_swiglu_forward(rows, inner, type, GU, ld, H, ldh, g, sg_, u, su, None)


@pytest.mark.parametrize("status, args", [
    (sg.ERR_SHAPE, dict(rows=-1)), (sg.ERR_SHAPE, dict(inner=(1 << 21) + 1)), (sg.ERR_CONFIG, dict(type=3)), (sg.ERR_LD, dict(ld=255)),
    (sg.ERR_LD, dict(ldh=127)), (sg.ERR_NULL, dict(GU=None)), (sg.ERR_NULL, dict(H=None)), (sg.ERR_NULL, dict(su=None)),
    (sg.ERR_ALIGN, dict(g=FAR * 3 + 8)), (sg.ERR_ALIGN, dict(H=FAR * 2 + 1)), (sg.ERR_ALIAS, dict(H=FAR)), (sg.ERR_ALIAS, dict(u=FAR * 3)),
])
def test_swiglu_forward_refuses(status, args):
    assert gated(**args) == status


def gated_backward(rows=4, inner=128, type=0, D=FAR, ld=128, g=FAR * 3, sg_=FAR * 4, u=FAR * 5, su=FAR * 6, out=FAR * 7, ldo=256):
    return lib().sgemm_f32_i8_swiglu_backward(rows, inner, type, D, ld, g, sg_, u, su, out, ldo, None)


@pytest.mark.parametrize("status, args", [
    (sg.ERR_SHAPE, dict(rows=-1)), (sg.ERR_SHAPE, dict(inner=(1 << 21) + 1)), (sg.ERR_CONFIG, dict(type=-1)), (sg.ERR_LD, dict(ld=127)),
    (sg.ERR_LD, dict(ldo=255)), (sg.ERR_NULL, dict(D=None)), (sg.ERR_NULL, dict(out=None)), (sg.ERR_NULL, dict(g=None)),
    (sg.ERR_ALIGN, dict(u=FAR * 5 + 8)), (sg.ERR_ALIAS, dict(out=FAR)), (sg.ERR_ALIAS, dict(out=FAR * 3)),
])
def test_swiglu_backward_refuses(status, args):
    assert gated_backward(**args) == status


def test_empty_calls_touch_nothing():
    assert quantize(rows=0, X=None, q=None, s=None) == sg.OK
    assert dequantize(cols=0, q=None, s=None, Y=None) == sg.OK
    assert gemm(M=0, a=None, sa=None, C=None) == sg.OK
    assert gemm(N=0, b=None, sb=None, C=None) == sg.OK
    assert linear(N=0, w=None, s=None, Y=None) == sg.OK
    assert gated(rows=0, GU=None, H=None) == sg.OK
    assert gated_backward(inner=0, D=None, out=None) == sg.OK


# ---- the Python calls ----

def cpu_matrix(rows, cols, group=None):
    kp = ref.padded(cols)
    return sg.I8(torch.zeros(rows, kp, dtype=torch.int8), torch.ones((rows, kp // 128) if group else rows), rows, cols, group)


def test_i8_checks_its_arrays():
    q = cpu_matrix(33, 130)
    assert q.shape == (33, 130) and q.values.shape == (33, 256) and q.scales.shape == (33,) and q.group is None
    assert cpu_matrix(33, 130, 128).scales.shape == (33, 2)
    assert "33 x 130" in repr(q)
    for args in ((q.values, q.scales, 33, 120), (q.values[:, ::2], q.scales, 33, 100), (q.values, q.scales, -1, 130),
                 (q.values, q.scales, 33, 130, 64), (q.values, q.scales, 33, 130, 128), (q.values, q.scales[:5], 33, 130),
                 (q.values, q.scales, 1 << 22, 1 << 22)):
        with pytest.raises(ValueError):
            sg.I8(*args)
    for args in ((q.values.float(), q.scales, 33, 130), (q.values, q.scales.double(), 33, 130), (None, q.scales, 33, 130)):
        with pytest.raises(TypeError):
            sg.I8(*args)


def test_python_refuses_what_is_not_on_a_device():
    x, q, g = torch.zeros(4, 128), cpu_matrix(4, 128), cpu_matrix(4, 64, 128)
    for call in (lambda: sg.i8_quantize(x), lambda: sg.i8_quantize(None), lambda: sg.i8_dequantize(q), lambda: sg.i8_dequantize(x),
                 lambda: sg.i8_gemm(q, q), lambda: sg.i8_gemm(x, q), lambda: sg.i8_linear(x, q), lambda: sg.i8_train_forward(x, x),
                 lambda: sg.i8_train_forward(x, q), lambda: sg.i8_train_backward(x, (q, q)), lambda: sg.i8_swiglu_forward(x),
                 lambda: sg.i8_swiglu_backward(x, (g, g))):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        sg.i8_quantize(x, group=64)


# ---- the reference ----

def test_reference_rounds_ties_to_even_numbers():
    x = np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 0.4999, 0.5001]]) * 0.25
    q, s = ref.whole(x)
    assert np.array_equal(q, [[127, 0, 2, 2, 0, -2, 0, 1]]) and s[0] == 0.25
    assert np.array_equal(ref.whole(np.zeros((1, 3)))[0], np.zeros((1, 3))) and ref.whole(np.zeros((1, 3)))[1][0] == 2.0 ** -126
    q, s = ref.whole(np.array([[np.inf, 1.0], [1.0, 2.0]]))
    assert np.isnan(s[0]) and not q[0].any() and q[1, 1] == 127


def test_reference_keeps_representable_values():
    rng = np.random.default_rng(0)
    q = rng.integers(-127, 128, (5, 256)).astype(np.float64)
    q[:, ::128] = 127
    x = ref.values(q, np.array([0.5, 1.0, 2.0, 2.0 ** -100, 2.0 ** 100]), 256)
    assert np.array_equal(ref.whole(x)[0], q) and np.array_equal(ref.grouped(x)[0], q)
