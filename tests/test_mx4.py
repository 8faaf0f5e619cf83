"""The 4-bit operators on the host: sizes of the format, refusals of the C
entry points before anything touches the GPU, refusals of the Python calls,
and the reference itself at the format's edges."""
import ctypes

import numpy as np
import pytest
import torch

import fp32_sgemm_f32_amd as sg
from oracle import mx4 as ref

P = 1 << 20      # an address that no check may follow
FAR = 1 << 40


def lib():
    return sg.library()


@pytest.mark.parametrize("rows, cols", [(0, 0), (1, 1), (31, 128), (32, 129), (33, 4096), (1 << 22, 1 << 22)])
def test_sizes_of_the_arrays(rows, cols):
    c, s = ctypes.c_longlong(), ctypes.c_longlong()
    assert lib().sgemm_f32_mx4_bytes(rows, cols, ctypes.byref(c), ctypes.byref(s)) == sg.OK
    shape_c, shape_s = ref.shapes(rows, cols)
    assert c.value == np.prod(shape_c, dtype=np.int64) and s.value == np.prod(shape_s, dtype=np.int64)
    assert lib().sgemm_f32_mx4_bytes(rows, cols, None, None) == sg.OK


def test_sizes_out_of_range():
    for rows, cols in ((-1, 1), (1, -1), ((1 << 22) + 1, 1), (1, (1 << 22) + 1)):
        assert lib().sgemm_f32_mx4_bytes(rows, cols, None, None) == sg.ERR_SHAPE


def quantize(rows=4, cols=128, type=0, X=P, ldx=128, rule=0, c=P * 2, s=P * 3, ct=None, st=None):
    return lib().sgemm_f32_mx4_quantize(rows, cols, type, X, ldx, rule, c, s, ct, st, None)


@pytest.mark.parametrize("status, args", [
    (sg.ERR_SHAPE, dict(rows=-1)), (sg.ERR_SHAPE, dict(cols=(1 << 22) + 1)),
    (sg.ERR_CONFIG, dict(type=3)), (sg.ERR_CONFIG, dict(type=-1)), (sg.ERR_CONFIG, dict(rule=2)),
    (sg.ERR_LD, dict(ldx=127)), (sg.ERR_NULL, dict(X=None)), (sg.ERR_NULL, dict(c=None, s=None)),
    (sg.ERR_NULL, dict(s=None)), (sg.ERR_NULL, dict(ct=P * 4)),
    (sg.ERR_ALIGN, dict(X=P + 2)), (sg.ERR_ALIGN, dict(c=P * 2 + 8)), (sg.ERR_ALIGN, dict(s=P * 3 + 2)),
    (sg.ERR_ALIGN, dict(type=1, X=P + 1)),
    (sg.ERR_ALIAS, dict(c=P)), (sg.ERR_ALIAS, dict(s=P * 2 + 16)), (sg.ERR_ALIAS, dict(ct=P * 2, st=P * 5)),
])
def test_quantize_refuses(status, args):
    assert quantize(**args) == status


def dequantize(rows=4, cols=128, c=P, s=P * 2, type=0, Y=P * 3, ldy=128):
    return lib().sgemm_f32_mx4_dequantize(rows, cols, c, s, type, Y, ldy, None)


@pytest.mark.parametrize("status, args", [
    (sg.ERR_SHAPE, dict(rows=-1)), (sg.ERR_CONFIG, dict(type=7)), (sg.ERR_LD, dict(ldy=100)),
    (sg.ERR_NULL, dict(c=None)), (sg.ERR_NULL, dict(s=None)), (sg.ERR_NULL, dict(Y=None)),
    (sg.ERR_ALIGN, dict(c=P + 4)), (sg.ERR_ALIGN, dict(Y=P * 3 + 2)), (sg.ERR_ALIAS, dict(Y=P)),
])
def test_dequantize_refuses(status, args):
    assert dequantize(**args) == status


def gemm(M=4, N=4, K=128, alpha=1.0, a=P, sa=P * 2, b=P * 3, sb=P * 4, beta=0.0, type=0, C=P * 5, ldc=4):
    return lib().sgemm_f32_mx4_gemm(M, N, K, alpha, a, sa, b, sb, beta, type, C, ldc, None)


@pytest.mark.parametrize("status, args", [
    (sg.ERR_SHAPE, dict(M=-1)), (sg.ERR_SHAPE, dict(N=-1)), (sg.ERR_SHAPE, dict(K=-1)), (sg.ERR_CONFIG, dict(type=5)),
    (sg.ERR_LD, dict(ldc=3)), (sg.ERR_NULL, dict(a=None)), (sg.ERR_NULL, dict(sb=None)), (sg.ERR_NULL, dict(C=None)),
    (sg.ERR_NULL, dict(K=0, C=None)), (sg.ERR_ALIGN, dict(b=P * 3 + 8)), (sg.ERR_ALIAS, dict(C=P * 3)),
    (sg.ERR_ALIAS, dict(C=P * 2)),
])
def test_gemm_refuses(status, args):
    assert gemm(**args) == status


def linear(M=4, N=4, K=128, type=0, X=P, ldx=128, c=P * 2, s=P * 3, Y=P * 4, ldy=4, scratch=None, nbytes=0):
    return lib().sgemm_f32_mx4_linear(M, N, K, type, X, ldx, c, s, Y, ldy, scratch, nbytes, None)


@pytest.mark.parametrize("status, args", [
    (sg.ERR_SHAPE, dict(M=-1)), (sg.ERR_SHAPE, dict(K=(1 << 22) + 1, ldx=1 << 23)), (sg.ERR_CONFIG, dict(type=3)),
    (sg.ERR_LD, dict(ldx=127)), (sg.ERR_LD, dict(ldy=3)), (sg.ERR_NULL, dict(X=None)), (sg.ERR_NULL, dict(c=None)),
    (sg.ERR_NULL, dict(Y=None)), (sg.ERR_ALIGN, dict(X=P + 1)), (sg.ERR_ALIGN, dict(c=P * 2 + 4)),
    (sg.ERR_ALIAS, dict(Y=P)), (sg.ERR_ALIAS, dict(Y=P * 3)),
    # K long enough to be shared: scratch memory is needed
    (sg.ERR_NULL, dict(K=16384, ldx=16384)), (sg.ERR_SCRATCH, dict(K=16384, ldx=16384, scratch=FAR, nbytes=16)),
    (sg.ERR_ALIGN, dict(K=16384, ldx=16384, scratch=FAR + 64, nbytes=1 << 20)),
    (sg.ERR_ALIAS, dict(K=16384, ldx=16384, scratch=P * 2, nbytes=1 << 20)),
])
def test_linear_refuses(status, args):
    assert linear(**args) == status


def test_linear_scratch():
    n = ctypes.c_longlong()
    call = lib().sgemm_f32_mx4_linear_scratch
    assert call(4, 4, 128, 0, ctypes.byref(n)) == sg.OK and n.value == 0
    assert call(4, 100, 16384, 0, ctypes.byref(n)) == sg.OK and n.value > 0
    once = n.value
    assert call(64, 100, 16384, 0, ctypes.byref(n)) == sg.OK and n.value >= once
    most = n.value
    assert call(64 * 100 + 4, 100, 16384, 0, ctypes.byref(n)) == sg.OK and n.value == most   # 64 rows at a time
    assert call(4, 4, 128, 3, ctypes.byref(n)) == sg.ERR_CONFIG
    assert call(-1, 4, 128, 0, ctypes.byref(n)) == sg.ERR_SHAPE
    assert call(4, 4, 128, 0, None) == sg.ERR_NULL


def forward(M=4, N=8, K=128, type=0, X=FAR, ldx=128, type_w=0, W=FAR * 2, ldw=128, rule=0, Y=FAR * 3, ldy=8, xt=FAR * 4, sxt=FAR * 5,
            wt=FAR * 6, swt=FAR * 7, scratch=FAR * 8, nbytes=1 << 20):
    return lib().sgemm_f32_mx4_train_forward(M, N, K, type, X, ldx, type_w, W, ldw, rule, Y, ldy, xt, sxt, wt, swt, scratch,
                                             nbytes, None)


def backward(M=4, N=8, K=128, type=0, D=FAR, ldd=8, rule=0, xt=FAR * 2, sxt=FAR * 3, wt=FAR * 4, swt=FAR * 5, dX=FAR * 6, lddx=128,
             dW=FAR * 7, lddw=128, scratch=FAR * 8, nbytes=1 << 20):
    return lib().sgemm_f32_mx4_train_backward(M, N, K, type, D, ldd, rule, xt, sxt, wt, swt, dX, lddx, 0.0, dW, lddw, scratch,
                                              nbytes, None)


@pytest.mark.parametrize("status, args", [
    (sg.ERR_SHAPE, dict(M=-1)), (sg.ERR_SHAPE, dict(N=-1)), (sg.ERR_SHAPE, dict(K=-1)), (sg.ERR_CONFIG, dict(type=3)),
    (sg.ERR_CONFIG, dict(type_w=3)), (sg.ERR_CONFIG, dict(rule=2)), (sg.ERR_LD, dict(ldx=127)), (sg.ERR_LD, dict(ldw=127)),
    (sg.ERR_LD, dict(ldy=7)), (sg.ERR_NULL, dict(X=None)), (sg.ERR_NULL, dict(Y=None)), (sg.ERR_NULL, dict(swt=None)),
    (sg.ERR_NULL, dict(scratch=None)), (sg.ERR_ALIGN, dict(scratch=FAR * 8 + 16)), (sg.ERR_ALIGN, dict(xt=FAR * 4 + 8)),
    (sg.ERR_SCRATCH, dict(nbytes=100)), (sg.ERR_ALIAS, dict(Y=FAR)), (sg.ERR_ALIAS, dict(scratch=FAR * 2)),
    (sg.ERR_ALIAS, dict(xt=FAR * 6)),
])
def test_train_forward_refuses(status, args):
    assert forward(**args) == status


@pytest.mark.parametrize("status, args", [
    (sg.ERR_SHAPE, dict(M=-1)), (sg.ERR_CONFIG, dict(type=3)), (sg.ERR_CONFIG, dict(rule=-1)), (sg.ERR_LD, dict(ldd=7)),
    (sg.ERR_LD, dict(lddx=127)), (sg.ERR_LD, dict(lddw=127)), (sg.ERR_NULL, dict(D=None)), (sg.ERR_NULL, dict(dW=None)),
    (sg.ERR_NULL, dict(xt=None)), (sg.ERR_NULL, dict(scratch=None)), (sg.ERR_ALIGN, dict(dW=FAR * 7 + 2)),
    (sg.ERR_SCRATCH, dict(nbytes=100)), (sg.ERR_ALIAS, dict(dX=FAR * 7)), (sg.ERR_ALIAS, dict(dW=FAR)),
])
def test_train_backward_refuses(status, args):
    assert backward(**args) == status


def test_train_scratch():
    f, b = ctypes.c_longlong(), ctypes.c_longlong()
    call = lib().sgemm_f32_mx4_train_scratch
    assert call(4, 8, 128, ctypes.byref(f), ctypes.byref(b)) == sg.OK and f.value > 0 and b.value > 0
    assert call(4, 8, 128, None, None) == sg.OK
    assert call(-1, 8, 128, None, None) == sg.ERR_SHAPE


def moe(tokens=2, hidden=128, inner=32, experts=4, top=2, norm=1, type=0, X=FAR, ldx=128, router=FAR * 2, ldr=128,
        up=FAR * 3, sup=FAR * 4, down=FAR * 5, sdown=FAR * 6, Y=FAR * 7, ldy=128, scratch=FAR * 8, nbytes=1 << 30):
    return lib().sgemm_f32_mx4_moe(tokens, hidden, inner, experts, top, norm, type, X, ldx, router, ldr, up, sup, down,
                                   sdown, Y, ldy, scratch, nbytes, None)


@pytest.mark.parametrize("status, args", [
    (sg.ERR_SHAPE, dict(tokens=-1)), (sg.ERR_SHAPE, dict(tokens=65)), (sg.ERR_SHAPE, dict(top=0)),
    (sg.ERR_SHAPE, dict(top=5)), (sg.ERR_SHAPE, dict(experts=64, top=17)), (sg.ERR_SHAPE, dict(experts=0, top=0)),
    (sg.ERR_SHAPE, dict(experts=1025)), (sg.ERR_SHAPE, dict(hidden=0)), (sg.ERR_SHAPE, dict(inner=0)),
    (sg.ERR_SHAPE, dict(inner=1 << 20)), (sg.ERR_SHAPE, dict(hidden=1 << 21, ldx=1 << 21, ldr=1 << 21, ldy=1 << 21)),
    (sg.ERR_CONFIG, dict(type=3)), (sg.ERR_CONFIG, dict(norm=2)),
    (sg.ERR_LD, dict(ldx=127)), (sg.ERR_LD, dict(ldr=127)), (sg.ERR_LD, dict(ldy=127)),
    (sg.ERR_NULL, dict(X=None)), (sg.ERR_NULL, dict(router=None)), (sg.ERR_NULL, dict(sdown=None)),
    (sg.ERR_NULL, dict(scratch=None)), (sg.ERR_ALIGN, dict(scratch=FAR * 8 + 128)), (sg.ERR_ALIGN, dict(up=FAR * 3 + 8)),
    (sg.ERR_SCRATCH, dict(nbytes=16)), (sg.ERR_ALIAS, dict(Y=FAR)), (sg.ERR_ALIAS, dict(scratch=FAR * 3)),
])
def test_moe_refuses(status, args):
    assert moe(**args) == status


def test_moe_scratch_refuses_what_the_call_refuses():
    n = ctypes.c_longlong()
    call = lib().sgemm_f32_mx4_moe_scratch
    assert call(2, 128, 32, 4, 2, 0, ctypes.byref(n)) == sg.OK and n.value > 0
    assert call(2, 128, 32, 4, 2, 0, None) == sg.ERR_NULL
    assert call(65, 128, 32, 4, 2, 0, ctypes.byref(n)) == sg.ERR_SHAPE
    assert call(2, 128, 32, 4, 2, 3, ctypes.byref(n)) == sg.ERR_CONFIG


def test_empty_calls_touch_nothing():
    assert quantize(rows=0, X=None, c=None, s=None) == sg.OK
    assert dequantize(cols=0, c=None, s=None, Y=None) == sg.OK
    assert gemm(M=0, a=None, sa=None, C=None) == sg.OK
    assert linear(N=0, c=None, s=None, Y=None) == sg.OK
    assert gemm(N=0, b=None, sb=None, C=None) == sg.OK
    assert moe(tokens=0, X=None, Y=None, scratch=None) == sg.OK


# ---- the Python calls ----

def cpu_matrix(rows, cols):
    c, s = ref.shapes(rows, cols)
    return sg.Mx4(torch.zeros(c, dtype=torch.uint8), torch.zeros(s, dtype=torch.uint8), rows, cols)


def test_mx4_checks_its_arrays():
    q = cpu_matrix(33, 130)
    assert q.shape == (33, 130) and q.codes.shape == (33, 128) and q.scales.shape == (2, 64, 4)
    with pytest.raises(ValueError):
        sg.Mx4(q.codes, q.scales, 33, 120)
    with pytest.raises(ValueError):
        sg.Mx4(q.codes[:, ::2], q.scales, 33, 100)
    with pytest.raises(ValueError):
        sg.Mx4(q.codes, q.scales, -1, 130)
    with pytest.raises(TypeError):
        sg.Mx4(q.codes.float(), q.scales, 33, 130)


def test_python_refuses_what_is_not_on_a_device():
    x, q = torch.zeros(4, 128), cpu_matrix(4, 128)
    for call in (lambda: sg.mx4_quantize(x), lambda: sg.mx4_quantize_both(x), lambda: sg.mx4_dequantize(q),
                 lambda: sg.mx4_gemm(q, q), lambda: sg.mx4_linear(x, q), lambda: sg.mx4_moe(x, x, q, q, 1),
                 lambda: sg.mx4_train_forward(x, x), lambda: sg.mx4_quantize(None), lambda: sg.mx4_gemm(x, q)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        sg.mx4_quantize(x, rule="nearest")


# ---- the reference ----

def test_reference_rounds_ties_to_even_codes_and_clips():
    x = np.array([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, 7.5, -0.25, -5.0, 0.2499, 0.2501]])
    want = [[0, 1, 1, 2, 2, 4, 4, 6, 6, 0, -4, 0, 0.5]]
    assert np.array_equal(ref.rounded(x), want)
    assert np.array_equal(ref.rounded(np.array([[7.0, 1.0]])), [[6.0, 1.0]])
    assert np.array_equal(ref.rounded(np.array([[7.0, 1.0]]), noclip=True), [[8.0, 1.0]])
    assert np.isnan(ref.rounded(np.array([[np.inf, 1.0]]))).all()


def test_reference_keeps_representable_values():
    rng = np.random.default_rng(0)
    codes, scales = rng.integers(0, 256, (5, 128), dtype=np.uint8), np.zeros((2, 32, 4), dtype=np.uint8)
    scales[:, :5] = rng.integers(1, 252, (2, 5, 4))
    x = ref.values(codes, scales, 256)
    assert np.array_equal(ref.rounded(x), x)
