"""Binding of the microscaled 4-bit (MXFP4) calls of libsgemm_f32.

A 4-bit matrix is an Mx4: the two device arrays that include/sgemm_f32.h
describes, and the size they stand for.  As in the package itself, every step
runs in the HIP library; PyTorch holds the memory and names the stream.
Results are allocated on the stream that the call runs on; tensors used on a
stream other than the current one are recorded on it, so that freeing them
early does no harm.
"""
import ctypes

SCALE_FLOOR = 0
SCALE_NOCLIP = 1
MAX_DIM = 1 << 22
_RULES = {"floor": SCALE_FLOOR, "noclip": SCALE_NOCLIP}


def _bind(lib):
    """Argument types of the 4-bit entry points."""
    i, p, f, ll = ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_longlong
    lib.sgemm_f32_mx4_bytes.argtypes = [i, i, ctypes.POINTER(ll), ctypes.POINTER(ll)]
    lib.sgemm_f32_mx4_quantize.argtypes = [i, i, i, p, i, i, p, p, p, p, p]
    lib.sgemm_f32_mx4_dequantize.argtypes = [i, i, p, p, i, p, i, p]
    lib.sgemm_f32_mx4_gemm.argtypes = [i, i, i, f, p, p, p, p, f, i, p, i, p]
    lib.sgemm_f32_mx4_linear.argtypes = [i, i, i, i, p, i, p, p, p, i, p, ll, p]
    lib.sgemm_f32_mx4_linear_scratch.argtypes = [i, i, i, i, ctypes.POINTER(ll)]
    lib.sgemm_f32_mx4_moe.argtypes = [i, i, i, i, i, i, i, p, i, p, i, p, p, p, p, p, i, p, ll, p]
    lib.sgemm_f32_mx4_moe_scratch.argtypes = [i, i, i, i, i, i, ctypes.POINTER(ll)]
    for name in ("bytes", "quantize", "dequantize", "gemm", "linear", "linear_scratch", "moe", "moe_scratch"):
        getattr(lib, "sgemm_f32_mx4_" + name).restype = i


def _shapes(rows, cols):
    slabs = (cols + 127) // 128
    return (rows, slabs * 64), (slabs, (rows + 31) // 32 * 32, 4)


class Mx4:
    """A rows x cols matrix in 4-bit codes with a scale byte per 32 values of a row.

    codes: uint8 (rows, kp / 2), kp = cols rounded up to 128; column k of a row
    in its byte k // 2, even k in the low four bits.  scales: uint8
    (kp / 128, rows rounded up to 32, 4); the scale of block b of row r is at
    [b // 4, r, b % 4] and stands for 2 ** (s - 127).  Both contiguous, zeros
    beyond cols (and, for scales, beyond rows).
    """

    __slots__ = ("codes", "scales", "shape")

    def __init__(self, codes, scales, rows, cols):
        import torch

        if not (0 <= rows <= MAX_DIM and 0 <= cols <= MAX_DIM):
            raise ValueError(f"rows and cols must be in [0, {MAX_DIM}]")
        want = _shapes(rows, cols)
        for t, n, shape in ((codes, "codes", want[0]), (scales, "scales", want[1])):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8:
                raise TypeError(f"{n} must be a uint8 tensor")
            if tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{n} of a {rows} x {cols} matrix must be contiguous {shape}, not {tuple(t.shape)}")
        if codes.device != scales.device:
            raise ValueError("codes and scales must be on one device")
        self.codes, self.scales, self.shape = codes, scales, (rows, cols)

    @property
    def device(self):
        return self.codes.device

    def __repr__(self):
        return f"Mx4({self.shape[0]} x {self.shape[1]}, {self.device})"


def _type(dtype):
    import torch

    code = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}.get(dtype)
    if code is None:
        raise TypeError(f"type must be float32, bfloat16 or float16, not {dtype}")
    return code


def _floats(t, name, device=None):
    """(type, leading dimension) of a row-major float matrix on a HIP device."""
    import torch

    from . import _row_major_ld

    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a tensor on a HIP device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    return _type(t.dtype), _row_major_ld(t, name)


def _packed(q, name, device=None):
    if not isinstance(q, Mx4):
        raise TypeError(f"{name} must be an Mx4")
    if not q.codes.is_cuda:
        raise TypeError(f"{name} must be on a HIP device")
    if device is not None and q.device != device:
        raise ValueError(f"{name} must be on {device}")
    return q


class _Run:
    """One call: the stream it runs on, its allocations, its launch."""

    __slots__ = ("device", "stream", "other")

    def __init__(self, device, stream):
        import torch

        current = torch.cuda.current_stream(device)
        self.device = device
        self.stream = current if stream is None else stream
        self.other = self.stream != current

    def empty(self, shape, dtype):
        import torch

        if self.other:
            with torch.cuda.stream(self.stream):
                return torch.empty(shape, dtype=dtype, device=self.device)
        return torch.empty(shape, dtype=dtype, device=self.device)

    def mx4(self, rows, cols):
        import torch

        codes, scales = _shapes(rows, cols)
        return Mx4(self.empty(codes, torch.uint8), self.empty(scales, torch.uint8), rows, cols)

    def call(self, name, tensors, *args):
        """Calls sgemm_f32_<name>(*args, stream); `tensors` are the caller's that it uses."""
        import torch

        from . import OK, SgemmError, library

        fn = getattr(library(), "sgemm_f32_" + name)
        if self.other:
            for t in tensors:
                for x in (t.codes, t.scales) if isinstance(t, Mx4) else (t,):
                    x.record_stream(self.stream)
        if torch.cuda.current_device() == self.device.index:
            st = fn(*args, self.stream.cuda_stream)
        else:
            with torch.cuda.device(self.device):
                st = fn(*args, self.stream.cuda_stream)
        if st != OK:
            raise SgemmError(st, "sgemm_f32_" + name)


def _result(run, out, shape, dtype):
    if out is None:
        return run.empty(shape, dtype)
    if tuple(out.shape) != tuple(shape) or out.dtype != dtype:
        raise ValueError(f"out must be {tuple(shape)} of {dtype}")
    return out


def _quantize(X, along, down, rule, stream):
    if rule not in _RULES:
        raise ValueError(f"rule must be one of {sorted(_RULES)}")
    import torch

    if isinstance(X, torch.Tensor) and X.dim() == 2 and X.stride(1) != 1 and X.shape[1] > 1 and X.stride(0) == 1:
        # A column-major view: its memory read the other way, without a copy.
        qt, q = _quantize(X.t(), down, along, rule, stream)
        return q, qt
    ty, ld = _floats(X, "X")
    rows, cols = X.shape
    run = _Run(X.device, stream)
    q = run.mx4(rows, cols) if along else None
    qt = run.mx4(cols, rows) if down else None
    run.call("mx4_quantize", (X,), rows, cols, ty, X.data_ptr(), ld, _RULES[rule],
             *((q.codes.data_ptr(), q.scales.data_ptr()) if along else (None, None)),
             *((qt.codes.data_ptr(), qt.scales.data_ptr()) if down else (None, None)))
    return q, qt


def mx4_quantize(X, rule="floor", stream=None):
    """X (float32, bfloat16 or float16, row- or column-major) as an Mx4, blocks along its rows.

    rule: "floor" takes the scale 2^(floor(log2 m) - 2) for the block's largest
    magnitude m (values above 6 scales become 6), "noclip" the least power of
    two with m <= 6 scales.  Values are rounded to the nearest code, ties to
    the even one.  A block with a NaN or an infinity becomes NaN.
    mx4_quantize(X.t()) gives the blocks along X's columns.
    """
    return _quantize(X, True, False, rule, stream)[0]


def mx4_quantize_both(X, rule="floor", stream=None):
    """(mx4_quantize(X), mx4_quantize(X.t())) in one pass over X."""
    return _quantize(X, True, True, rule, stream)


def mx4_dequantize(q, dtype=None, out=None, stream=None):
    """The values of an Mx4 as float32 (or `dtype`, or `out`'s type)."""
    import torch

    _packed(q, "q")
    run = _Run(q.device, stream)
    if out is None:
        out = run.empty(q.shape, torch.float32 if dtype is None else dtype)
    elif tuple(out.shape) != q.shape or dtype not in (None, out.dtype):
        raise ValueError(f"out must be {q.shape} of the given dtype")
    ty, ld = _floats(out, "out", q.device)
    run.call("mx4_dequantize", (q, out), *q.shape, q.codes.data_ptr(), q.scales.data_ptr(), ty, out.data_ptr(), ld)
    return out


def mx4_gemm(A, B, out=None, dtype=None, alpha=1.0, beta=0.0, stream=None):
    """alpha * A @ B^T + beta * out for Mx4 matrices A (M, K) and B (N, K), sums in fp32.

    out (M, N) is allocated as float32 (or `dtype`) if None (then beta must be 0).
    """
    import torch

    _packed(A, "A")
    _packed(B, "B", A.device)
    if A.shape[1] != B.shape[1]:
        raise ValueError(f"inner dimensions differ: {A.shape[1]} vs {B.shape[1]}")
    M, N, K = A.shape[0], B.shape[0], A.shape[1]
    run = _Run(A.device, stream)
    if out is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs out")
        out = run.empty((M, N), torch.float32 if dtype is None else dtype)
    elif tuple(out.shape) != (M, N) or dtype not in (None, out.dtype):
        raise ValueError(f"out must be {(M, N)} of the given dtype")
    ty, ld = _floats(out, "out", A.device)
    run.call("mx4_gemm", (A, B, out), M, N, K, float(alpha), A.codes.data_ptr(), A.scales.data_ptr(),
             B.codes.data_ptr(), B.scales.data_ptr(), float(beta), ty, out.data_ptr(), ld)
    return out


def mx4_train_forward(X, W, rule="floor", stream=None):
    """Y = q(X) q(W)^T for X (M, K) and a layer's weights W (N, K), in X's type.

    Returns (Y, saved); `saved` holds X^T and W^T in 4 bits, quantised along M
    and N, for mx4_train_backward.
    """
    q, qt = mx4_quantize_both(X, rule, stream)
    w, wt = mx4_quantize_both(W, rule, stream)
    return mx4_gemm(q, w, dtype=X.dtype, stream=stream), (qt, wt, rule)


def mx4_train_backward(dY, saved, dW=None, stream=None):
    """(dX, dW) = (q(dY) q(W^T)^T, q(dY^T) q(X^T)^T): the gradients of
    mx4_train_forward with the rounding taken as the identity.  dX comes in
    dY's type, dW in float32; a dW given is added to."""
    import torch

    xt, wt, rule = saved
    d, dt = mx4_quantize_both(dY, rule, stream)
    dX = mx4_gemm(d, wt, dtype=dY.dtype, stream=stream)
    if dW is None:
        return dX, mx4_gemm(dt, xt, dtype=torch.float32, stream=stream)
    return dX, mx4_gemm(dt, xt, out=dW, beta=1.0, stream=stream)


def mx4_linear(X, W, out=None, stream=None):
    """X @ W^T for float rows X (M, K) and 4-bit weights W (N, K), in X's type.

    X is used as it is (no rounding to 4 bits), sums are in fp32.  Made for one
    token or a few: W is read once for up to 64 rows.
    """
    ty, ldx = _floats(X, "X")
    _packed(W, "W", X.device)
    M, K = X.shape
    if K != W.shape[1]:
        raise ValueError(f"inner dimensions differ: {K} vs {W.shape[1]}")
    N = W.shape[0]
    run = _Run(X.device, stream)
    out = _result(run, out, (M, N), X.dtype)
    _, ldy = _floats(out, "out", X.device)
    import torch

    from . import library
    need = ctypes.c_longlong()
    library().sgemm_f32_mx4_linear_scratch(M, N, K, ty, ctypes.byref(need))
    scratch = run.empty((need.value,), torch.uint8) if need.value else None
    run.call("mx4_linear", (X, W, out), M, N, K, ty, X.data_ptr(), ldx, W.codes.data_ptr(), W.scales.data_ptr(),
             out.data_ptr(), ldy, None if scratch is None else scratch.data_ptr(), need.value)
    return out


def mx4_moe(X, router, gate_up, down, top, norm=True, out=None, stream=None):
    """A mixture-of-experts layer for up to 64 tokens X (T, H), in X's type.

    router (E, H) in X's type; gate_up an Mx4 of (E * 2 * F, H), expert after
    expert, F gate rows and then F up rows; down an Mx4 of (E * H, F).  A token
    goes to the `top` experts of largest logit X router^T (lower index first on
    equal ones) and gets the sum of p_e D_e (silu(G_e x) * (U_e x)), with p the
    softmax over those (norm) or over all experts.
    """
    import torch

    from . import OK, SgemmError, library

    ty, ldx = _floats(X, "X")
    tr, ldr = _floats(router, "router", X.device)
    _packed(gate_up, "gate_up", X.device)
    _packed(down, "down", X.device)
    T, H = X.shape
    E, F = router.shape[0], down.shape[1]
    if tr != ty:
        raise TypeError("router must have X's type")
    if router.shape[1] != H or gate_up.shape != (E * 2 * F, H) or down.shape[0] != E * H:
        raise ValueError(f"router {tuple(router.shape)}, gate_up {gate_up.shape} and down {down.shape} do not fit "
                         f"together with {H} columns of X")
    need = ctypes.c_longlong()
    st = library().sgemm_f32_mx4_moe_scratch(T, H, F, E, top, ty, ctypes.byref(need))
    if st != OK:
        raise SgemmError(st, "sgemm_f32_mx4_moe")
    run = _Run(X.device, stream)
    out = _result(run, out, (T, H), X.dtype)
    _, ldy = _floats(out, "out", X.device)
    scratch = run.empty((need.value,), torch.uint8)
    run.call("mx4_moe", (X, router, gate_up, down, out), T, H, F, E, top, int(bool(norm)), ty, X.data_ptr(), ldx,
             router.data_ptr(), ldr, gate_up.codes.data_ptr(), gate_up.scales.data_ptr(), down.codes.data_ptr(),
             down.scales.data_ptr(), out.data_ptr(), ldy, scratch.data_ptr(), need.value)
    return out
