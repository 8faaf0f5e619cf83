"""Binding of the microscaled 4-bit (MXFP4) calls of libsgemm_f32.

A 4-bit matrix is an Mx4: the two device arrays that include/sgemm_f32.h
describes, and the size they stand for.  As in the package itself, every step
runs in the HIP library; PyTorch holds the memory and names the stream.
Results are allocated on the stream that the call runs on; tensors used on a
stream other than the current one are recorded on it, so that freeing them
early does no harm.  Nothing here is recorded for automatic differentiation:
mx4_train_backward is the gradient of mx4_train_forward.

The small calls are bound by this file's time on the host, so a call asks
PyTorch for as little as it can: one allocation for the two arrays of a result
(its tensors are made when they are asked for), the current stream as a bare
handle, no module looked up twice.
"""
import ctypes
import functools
import operator

SCALE_FLOOR = 0
SCALE_NOCLIP = 1
MAX_DIM = 1 << 22
_RULES = {"floor": SCALE_FLOOR, "noclip": SCALE_NOCLIP}
_INT_MAX = (1 << 31) - 1


def _bind(lib):
    """Argument types of the 4-bit entry points."""
    i, p, f, ll = ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_longlong
    size = ctypes.POINTER(ll)
    for name, types in (
            ("bytes", [i, i, size, size]),
            ("quantize", [i, i, i, p, i, i, p, p, p, p, p]),
            ("dequantize", [i, i, p, p, i, p, i, p]),
            ("gemm", [i, i, i, f, p, p, p, p, f, i, p, i, p]),
            ("train_forward", [i, i, i, i, p, i, i, p, i, i, p, i, p, p, p, p, p, ll, p]),
            ("train_backward", [i, i, i, i, p, i, i, p, p, p, p, p, i, f, p, i, p, ll, p]),
            ("train_scratch", [i, i, i, size, size]),
            ("linear", [i, i, i, i, p, i, p, p, p, i, p, ll, p]),
            ("linear_scratch", [i, i, i, i, size]),
            ("moe", [i, i, i, i, i, i, i, p, i, p, i, p, p, p, p, p, i, p, ll, p]),
            ("moe_scratch", [i, i, i, i, i, i, size])):
        fn = getattr(lib, "sgemm_f32_mx4_" + name)
        fn.argtypes, fn.restype = types, i


class _Host:
    """What every call needs of PyTorch and the library, looked up once."""

    def __init__(self):
        import torch

        from . import OK, SgemmError, library

        lib = library()
        self.torch, self.empty, self.Tensor, self.uint8 = torch, torch.empty, torch.Tensor, torch.uint8
        self.float32 = torch.float32
        self.codes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
        self.current_device = torch.cuda.current_device
        # The current stream's handle, without the Stream object around it where PyTorch gives it so.
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        self.ok, self.error = OK, SgemmError
        for name in ("quantize", "dequantize", "gemm", "train_forward", "train_backward", "train_scratch", "linear",
                     "linear_scratch", "moe", "moe_scratch"):
            setattr(self, name, getattr(lib, "sgemm_f32_mx4_" + name))


_host = None


def _h():
    global _host
    if _host is None:
        _host = _Host()
    return _host


def _shapes(rows, cols):
    slabs = (cols + 127) // 128
    return (rows, slabs * 64), (slabs, (rows + 31) // 32 * 32, 4)


def _sizes(rows, cols):
    """Bytes of codes (a multiple of 64) and scales."""
    slabs = (cols + 127) // 128
    return rows * slabs * 64, slabs * ((rows + 31) // 32 * 128)


class Mx4:
    """A rows x cols matrix in 4-bit codes with a scale byte per 32 values of a row.

    codes: uint8 (rows, kp / 2), kp = cols rounded up to 128; column k of a row
    in its byte k // 2, even k in the low four bits.  scales: uint8
    (kp / 128, rows rounded up to 32, 4); the scale of block b of row r is at
    [b // 4, r, b % 4] and stands for 2 ** (s - 127).  Both contiguous, zeros
    beyond cols (and, for scales, beyond rows).
    """

    __slots__ = ("_codes", "_scales", "_base", "_at", "shape")

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
        self._codes, self._scales, self._base, self._at, self.shape = codes, scales, None, 0, (rows, cols)

    @classmethod
    def _of(cls, base, at, rows, cols):
        """The matrix whose codes and then scales lie in base (1-D uint8) from byte `at` on."""
        q = object.__new__(cls)
        q._codes, q._scales, q._base, q._at, q.shape = None, None, base, at, (rows, cols)
        return q

    def _view(self):
        n, m = _sizes(*self.shape)
        c, s = _shapes(*self.shape)
        self._codes = self._base[self._at:self._at + n].view(c)
        self._scales = self._base[self._at + n:self._at + n + m].view(s)

    @property
    def codes(self):
        if self._codes is None:
            self._view()
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._view()
        return self._scales

    @property
    def device(self):
        return (self._codes if self._base is None else self._base).device

    def _pointers(self):
        if self._base is None:
            return self._codes.data_ptr(), self._scales.data_ptr()
        p = self._base.data_ptr() + self._at
        return p, p + _sizes(*self.shape)[0]

    def record_stream(self, stream):
        for t in (self._codes, self._scales) if self._base is None else (self._base,):
            t.record_stream(stream)

    def __repr__(self):
        return f"Mx4({self.shape[0]} x {self.shape[1]}, {self.device})"


def _floats(t, name, device=None):
    """(type, leading dimension) of a row-major float matrix on a HIP device."""
    h = _h()
    if not isinstance(t, h.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a tensor on a HIP device")
    code = h.codes.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, not {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    if rows == 0 or cols == 0:      # nothing is read or written through it
        ld = cols
    else:
        ld, unit = t.stride()
        if unit != 1 and cols > 1:
            raise ValueError(f"{name} must be row-major (unit column stride)")
        if rows == 1:
            ld = cols
    if rows > _INT_MAX or ld > _INT_MAX:
        raise ValueError(f"{name} is too large")
    return code, ld


def _dtype_code(dtype):
    code = _h().codes.get(dtype)
    if code is None:
        raise TypeError(f"type must be float32, bfloat16 or float16, not {dtype}")
    return code


def _packed(q, name, device=None):
    if not isinstance(q, Mx4):
        raise TypeError(f"{name} must be an Mx4")
    d = q.device
    if d.type != "cuda":
        raise TypeError(f"{name} must be on a HIP device")
    if device is not None and d != device:
        raise ValueError(f"{name} must be on {device}")
    return d


class _Run:
    """One call: the stream it runs on, its allocations, its launch."""

    __slots__ = ("h", "device", "handle", "other")

    def __init__(self, device, stream):
        h = self.h = _host
        self.device = device
        handle = h.raw_stream(device.index)
        self.other = None
        if stream is not None and stream.cuda_stream != handle:
            self.other = stream
            handle = stream.cuda_stream
        self.handle = handle

    def empty(self, shape, dtype):
        if self.other is not None:
            with self.h.torch.cuda.stream(self.other):
                return self.h.empty(shape, dtype=dtype, device=self.device)
        return self.h.empty(shape, dtype=dtype, device=self.device)

    def bytes(self, n):
        return self.empty(n, self.h.uint8)

    def mx4(self, rows, cols):
        if rows > MAX_DIM or cols > MAX_DIM:
            raise ValueError(f"rows and cols must be in [0, {MAX_DIM}]")
        n, m = _sizes(rows, cols)
        return Mx4._of(self.bytes(n + m), 0, rows, cols)

    def call(self, fn, tensors, *args):
        """fn(*args, stream); `tensors` are the caller's that it uses."""
        h = self.h
        if self.other is not None:
            for t in tensors:
                t.record_stream(self.other)
        if h.current_device() == self.device.index:
            st = fn(*args, self.handle)
        else:
            with h.torch.cuda.device(self.device):
                st = fn(*args, self.handle)
        if st != h.ok:
            raise h.error(st, fn.__name__)


@functools.lru_cache(maxsize=1024)
def _scratch(name, *sizes):
    """Bytes of scratch memory of a call with these sizes (a function of them alone)."""
    fn = getattr(_host, name)
    n = ctypes.c_longlong()
    st = fn(*sizes, ctypes.byref(n))
    if st != _host.ok:
        raise _host.error(st, fn.__name__)
    return n.value


@functools.lru_cache(maxsize=1024)
def _train_scratch(M, N, K):
    """The same of the forward and the backward call of a training step."""
    f, b = ctypes.c_longlong(), ctypes.c_longlong()
    st = _host.train_scratch(M, N, K, ctypes.byref(f), ctypes.byref(b))
    if st != _host.ok:
        raise _host.error(st, "sgemm_f32_mx4_train_scratch")
    return f.value, b.value


def _out(run, out, shape, dtype, name="out"):
    """out, or a new tensor; with its type and leading dimension."""
    if out is None:
        code = _dtype_code(dtype)
        return run.empty(shape, dtype), code, shape[1]
    if not isinstance(out, run.h.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if tuple(out.shape) != tuple(shape) or dtype not in (None, out.dtype):
        raise ValueError(f"{name} must be {tuple(shape)} of {dtype}")
    return (out, *_floats(out, name, run.device))


def _rule(rule):
    if rule not in _RULES:
        raise ValueError(f"rule must be one of {sorted(_RULES)}")
    return _RULES[rule]


def _column_major(X):
    return isinstance(X, _h().Tensor) and X.dim() == 2 and X.shape[1] > 1 and X.stride(1) != 1 and X.stride(0) == 1


def _quantize(X, along, down, rule, stream):
    code = _rule(rule)
    if _column_major(X):
        # Its memory read the other way, without a copy.
        qt, q = _quantize(X.t(), down, along, rule, stream)
        return q, qt
    ty, ld = _floats(X, "X")
    rows, cols = X.shape
    run = _Run(X.device, stream)
    q = run.mx4(rows, cols) if along else None
    qt = run.mx4(cols, rows) if down else None
    run.call(run.h.quantize, (X,), rows, cols, ty, X.data_ptr(), ld, code, *(q._pointers() if along else (None, None)),
             *(qt._pointers() if down else (None, None)))
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
    device = _packed(q, "q")
    h = _h()
    run = _Run(device, stream)
    out, ty, ld = _out(run, out, q.shape, h.float32 if out is None and dtype is None else dtype)
    run.call(h.dequantize, (q, out), *q.shape, *q._pointers(), ty, out.data_ptr(), ld)
    return out


def mx4_gemm(A, B, out=None, dtype=None, alpha=1.0, beta=0.0, stream=None):
    """alpha * A @ B^T + beta * out for Mx4 matrices A (M, K) and B (N, K), sums in fp32.

    out (M, N) is allocated as float32 (or `dtype`) if None (then beta must be 0).
    """
    device = _packed(A, "A")
    _packed(B, "B", device)
    (M, K), (N, K2) = A.shape, B.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if out is None and beta != 0.0:
        raise ValueError("beta != 0 needs out")
    h = _h()
    run = _Run(device, stream)
    out, ty, ld = _out(run, out, (M, N), h.float32 if out is None and dtype is None else dtype)
    run.call(h.gemm, (A, B, out), M, N, K, float(alpha), *A._pointers(), *B._pointers(), float(beta), ty, out.data_ptr(), ld)
    return out


def mx4_train_forward(X, W, rule="floor", stream=None):
    """Y = q(X) q(W)^T for X (M, K) and a layer's weights W (N, K), in X's type.

    Returns (Y, saved); `saved` holds X^T and W^T in 4 bits, quantised along M
    and N, for mx4_train_backward.
    """
    code = _rule(rule)
    if _column_major(X) or _column_major(W):
        q, qt = mx4_quantize_both(X, rule, stream)
        w, wt = mx4_quantize_both(W, rule, stream)
        return mx4_gemm(q, w, dtype=X.dtype, stream=stream), (qt, wt, rule)
    tx, ldx = _floats(X, "X")
    device = X.device
    tw, ldw = _floats(W, "W", device)
    (M, K), (N, K2) = X.shape, W.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if M > MAX_DIM or N > MAX_DIM or K > MAX_DIM:
        raise ValueError(f"sizes must be in [0, {MAX_DIM}]")
    h = _host
    run = _Run(device, stream)
    of_x, of_w = sum(_sizes(K, M)), sum(_sizes(K, N))
    at_w = (of_x + 255) // 256 * 256
    kept = run.bytes(at_w + of_w)
    xt, wt = Mx4._of(kept, 0, K, M), Mx4._of(kept, at_w, K, N)
    need = _train_scratch(M, N, K)[0]
    scratch = run.bytes(need)
    Y = run.empty((M, N), X.dtype)
    run.call(h.train_forward, (X, W), M, N, K, tx, X.data_ptr(), ldx, tw, W.data_ptr(), ldw, code, Y.data_ptr(), N,
             *xt._pointers(), *wt._pointers(), scratch.data_ptr(), need)
    return Y, (xt, wt, rule)


def mx4_train_backward(dY, saved, dW=None, stream=None):
    """(dX, dW) = (q(dY) q(W^T)^T, q(dY^T) q(X^T)^T): the gradients of
    mx4_train_forward with the rounding taken as the identity.  dX comes in
    dY's type, dW in float32; a dW given is added to."""
    xt, wt, rule = saved
    code = _rule(rule)
    if _column_major(dY):
        d, dt = mx4_quantize_both(dY, rule, stream)
        dX = mx4_gemm(d, wt, dtype=dY.dtype, stream=stream)
        return dX, mx4_gemm(dt, xt, out=dW, dtype=_h().float32, beta=0.0 if dW is None else 1.0, stream=stream)
    ty, ld = _floats(dY, "dY")
    device = dY.device
    _packed(xt, "saved", device)
    _packed(wt, "saved", device)
    (M, N), (K, M2), (K2, N2) = dY.shape, xt.shape, wt.shape
    if (M, N, K) != (M2, N2, K2):
        raise ValueError(f"dY {(M, N)} does not fit what the forward pass saved of {M2} x {K} and {N2} x {K2} matrices")
    h = _host
    run = _Run(device, stream)
    need = _train_scratch(M, N, K)[1]
    scratch = run.bytes(need)
    dX = run.empty((M, K), dY.dtype)
    beta = 0.0 if dW is None else 1.0
    dW, _, ldw = _out(run, dW, (N, K), h.float32, "dW")
    run.call(h.train_backward, (dY, xt, wt, dW), M, N, K, ty, dY.data_ptr(), ld, code, *xt._pointers(), *wt._pointers(),
             dX.data_ptr(), K, beta, dW.data_ptr(), ldw, scratch.data_ptr(), need)
    return dX, dW


def mx4_linear(X, W, out=None, stream=None):
    """X @ W^T for float rows X (M, K) and 4-bit weights W (N, K), in X's type.

    X is used as it is (no rounding to 4 bits), sums are in fp32.  Made for one
    token or a few: W is read once for up to 64 rows (32 in float32).
    """
    ty, ldx = _floats(X, "X")
    device = X.device
    _packed(W, "W", device)
    (M, K), (N, K2) = X.shape, W.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    h = _host
    run = _Run(device, stream)
    out, _, ldy = _out(run, out, (M, N), X.dtype)
    need = _scratch("linear_scratch", M, N, K, ty)
    scratch = run.bytes(need) if need else None
    run.call(h.linear, (X, W, out), M, N, K, ty, X.data_ptr(), ldx, *W._pointers(), out.data_ptr(), ldy,
             scratch.data_ptr() if need else None, need)
    return out


def mx4_moe(X, router, gate_up, down, top, norm=True, out=None, stream=None):
    """A mixture-of-experts layer for up to 64 tokens X (T, H), in X's type.

    router (E, H) in X's type; gate_up an Mx4 of (E * 2 * F, H), expert after
    expert, F gate rows and then F up rows; down an Mx4 of (E * H, F).  A token
    goes to the `top` experts of largest logit X router^T (lower index first on
    equal ones) and gets the sum of p_e D_e (silu(G_e x) * (U_e x)), with p the
    softmax over those (norm) or over all experts.
    """
    ty, ldx = _floats(X, "X")
    device = X.device
    tr, ldr = _floats(router, "router", device)
    _packed(gate_up, "gate_up", device)
    _packed(down, "down", device)
    T, H = X.shape
    E, F = router.shape[0], down.shape[1]
    if tr != ty:
        raise TypeError("router must have X's type")
    if router.shape[1] != H or gate_up.shape != (E * 2 * F, H) or down.shape[0] != E * H:
        raise ValueError(f"router {tuple(router.shape)}, gate_up {gate_up.shape} and down {down.shape} do not fit "
                         f"together with {H} columns of X")
    top = max(0, min(operator.index(top), _INT_MAX))    # the library says which are too few or too many
    h = _host
    need = _scratch("moe_scratch", T, H, F, E, top, ty)
    run = _Run(device, stream)
    out, _, ldy = _out(run, out, (T, H), X.dtype)
    scratch = run.bytes(need)
    run.call(h.moe, (X, router, gate_up, down, out), T, H, F, E, top, int(bool(norm)), ty, X.data_ptr(), ldx,
             router.data_ptr(), ldr, *gate_up._pointers(), *down._pointers(), out.data_ptr(), ldy, scratch.data_ptr(), need)
    return out
