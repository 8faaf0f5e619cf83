"""Binding of the 8-bit integer calls of libsgemm_f32.

An 8-bit matrix is an I8: the two device arrays that include/sgemm_f32.h
describes, and the size they stand for.  Streams, allocations and checks are
those of the 4-bit binding (mx4.py), whose helpers this file uses.  Nothing
here is recorded for automatic differentiation: i8_train_backward and
i8_swiglu_backward are the gradients of the calls before them.
"""
import ctypes
import functools

from . import mx4

GROUP = 128
FLOOR = 2.0 ** -126     # the least scale
MAX_DIM = 1 << 22
MAX_VALUES = 1 << 34
MAX_SUM = 1 << 17


def _bind(lib):
    """Argument types of the 8-bit entry points."""
    i, p, f, ll = ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_longlong
    size = ctypes.POINTER(ll)
    for name, types in (
            ("bytes", [i, i, i, size, size]),
            ("quantize", [i, i, i, i, i, p, i, p, p, p, ll, p]),
            ("quantize_scratch", [i, i, i, size]),
            ("dequantize", [i, i, i, p, p, i, p, i, p]),
            ("gemm", [i, i, i, f, p, p, p, p, f, i, p, i, p]),
            ("linear", [i, i, i, i, p, i, p, p, p, i, p, ll, p]),
            ("linear_scratch", [i, i, i, i, size]),
            ("train_forward", [i, i, i, i, p, i, i, p, i, p, i, p, p, p, p, p]),
            ("train_backward", [i, i, i, i, p, i, p, p, p, p, p, i, f, p, i, p, ll, p]),
            ("train_scratch", [i, i, i, size]),
            ("swiglu_forward", [i, i, i, p, i, p, i, p, p, p, p, p]),
            ("swiglu_backward", [i, i, i, p, i, p, p, p, p, p, i, p])):
        fn = getattr(lib, "sgemm_f32_i8_" + name)
        fn.argtypes, fn.restype = types, i


class _Calls:
    """The library's functions, looked up once."""

    def __init__(self):
        from . import library

        lib = library()
        for name in ("quantize", "quantize_scratch", "dequantize", "gemm", "linear", "linear_scratch", "train_forward",
                     "train_backward", "train_scratch", "swiglu_forward", "swiglu_backward"):
            setattr(self, name, getattr(lib, "sgemm_f32_i8_" + name))


_calls = None


def _c():
    global _calls
    if _calls is None:
        _calls = _Calls()
    return _calls


def _ld(cols):
    return (cols + 127) // 128 * 128


def _scales(rows, cols, group):
    return (rows, _ld(cols) // 128) if group else (rows,)


def _size(rows, cols):
    if not (0 <= rows <= MAX_DIM and 0 <= cols <= MAX_DIM):
        raise ValueError(f"rows and cols must be in [0, {MAX_DIM}]")
    if rows * _ld(cols) > MAX_VALUES:
        raise ValueError(f"a {rows} x {cols} matrix holds more than {MAX_VALUES} values")


@functools.lru_cache(maxsize=4096)
def _layout(rows, cols, group):
    """(bytes of the values, of both arrays); refuses what no matrix can be."""
    _size(rows, cols)
    ld = _ld(cols)
    return rows * ld, rows * ld + 4 * rows * (ld // 128 if group else 1)


class I8:
    """A rows x cols matrix of signed bytes with a float scale for each row, or for each 128 columns of a row.

    values: int8 (rows, kp), kp = cols rounded up to 128, zeros beyond cols,
    all in [-127, 127].  scales: float32 (rows,), or with group = 128 (rows, kp /
    128).  Both contiguous.  The matrix is values * scales.
    """

    __slots__ = ("_values", "_scales", "_base", "_at", "shape", "group")

    def __init__(self, values, scales, rows, cols, group=None):
        import torch

        _size(rows, cols)
        if group not in (None, GROUP):
            raise ValueError(f"group must be None or {GROUP}")
        for t, n, ty, shape in ((values, "values", torch.int8, (rows, _ld(cols))),
                                (scales, "scales", torch.float32, _scales(rows, cols, group))):
            if not isinstance(t, torch.Tensor) or t.dtype != ty:
                raise TypeError(f"{n} must be a {ty} tensor")
            if tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{n} of a {rows} x {cols} matrix must be contiguous {shape}, not {tuple(t.shape)}")
        if values.device != scales.device:
            raise ValueError("values and scales must be on one device")
        self._values, self._scales, self._base, self._at, self.shape, self.group = values, scales, None, 0, (rows, cols), group

    @classmethod
    def _of(cls, base, at, rows, cols, group=None):
        """The matrix whose values and then scales lie in base (1-D uint8) from byte `at` on."""
        q = object.__new__(cls)
        q._values, q._scales, q._base, q._at, q.shape, q.group = None, None, base, at, (rows, cols), group
        return q

    def _view(self):
        rows, cols = self.shape
        n, end = _layout(rows, cols, self.group)
        torch = mx4._h().torch
        self._values = self._base[self._at:self._at + n].view(torch.int8).view(rows, _ld(cols))
        self._scales = self._base[self._at + n:self._at + end].view(torch.float32).view(_scales(rows, cols, self.group))

    @property
    def values(self):
        if self._values is None:
            self._view()
        return self._values

    @property
    def scales(self):
        if self._scales is None:
            self._view()
        return self._scales

    @property
    def device(self):
        return (self._values if self._base is None else self._base).device

    def _pointers(self):
        if self._base is None:
            return self._values.data_ptr(), self._scales.data_ptr()
        p = self._base.data_ptr() + self._at
        return p, p + _layout(*self.shape, self.group)[0]

    def record_stream(self, stream):
        for t in (self._values, self._scales) if self._base is None else (self._base,):
            t.record_stream(stream)

    def __repr__(self):
        return f"I8({self.shape[0]} x {self.shape[1]}{', groups of 128' if self.group else ''}, {self.device})"


def _held(q, name, device=None, group=None):
    """The device of an I8 with the scales that a call takes."""
    if not isinstance(q, I8):
        raise TypeError(f"{name} must be an I8")
    d = q.device
    if d.type != "cuda":
        raise TypeError(f"{name} must be on a HIP device")
    if device is not None and d != device:
        raise ValueError(f"{name} must be on {device}")
    if q.group != group:
        raise ValueError(f"{name} must have a scale for each {'row' if group is None else '128 columns of a row'}")
    return d


def _new(run, rows, cols, group=None):
    q = I8._of(run.bytes(_layout(rows, cols, group)[1]), 0, rows, cols, group)
    return q if cols else _without_columns(run, q)


def _two(run, shape, other, group=None):
    """Two new matrices in one allocation, with equally many columns."""
    at = (_layout(*shape, group)[1] + 255) // 256 * 256
    base = run.bytes(at + _layout(*other, group)[1])
    q, p = I8._of(base, 0, *shape, group), I8._of(base, at, *other, group)
    return (q, p) if shape[1] else (_without_columns(run, q), _without_columns(run, p))


def _without_columns(run, q):
    """q with its scales, those of a largest magnitude of 0: the library neither reads nor writes any there."""
    if q.group is None:
        with run.h.torch.cuda.stream(run.other):     # (of None: the current one)
            q.scales.fill_(FLOOR)
    return q


@functools.lru_cache(maxsize=1024)
def _scratch(name, *sizes):
    """Bytes of scratch memory of a call with these sizes (a function of them alone)."""
    fn = getattr(_c(), name)
    n = ctypes.c_longlong()
    st = fn(*sizes, ctypes.byref(n))
    if st != mx4._h().ok:
        raise mx4._host.error(st, fn.__name__)
    return n.value


def _sum(k):
    if k > MAX_SUM:
        raise ValueError(f"a sum of {k} products is longer than {MAX_SUM}")


def i8_quantize(X, group=None, stream=None):
    """X (float32, bfloat16 or float16) as an I8, with a scale for each row (group = None) or each 128 columns of a row.

    For the largest magnitude m of a row or group the scale is m / 127 (at least
    2^-126), and values are rounded to the nearest whole multiple, ties to the
    even one.  A row or group with a NaN or an infinity becomes NaN.  X is
    row-major, or (without groups) column-major: i8_quantize(X.t()) gives the
    scales of X's columns.
    """
    if group not in (None, GROUP):
        raise ValueError(f"group must be None or {GROUP}")
    c = _c()
    trans = group is None and mx4._column_major(X)
    ty, ld = mx4._floats(X.t() if trans else X, "X")
    rows, cols = X.shape
    _layout(rows, cols, group)
    run = mx4._Run(X.device, stream)
    need = 0
    if trans:
        _layout(cols, rows, None)
        need = _scratch("quantize_scratch", 1, rows, cols)
    scratch = run.bytes(need) if need else None
    q = _new(run, rows, cols, group)
    run.call(c.quantize, (X,), int(trans), rows, cols, group or 0, ty, X.data_ptr(), ld, *q._pointers(),
             scratch.data_ptr() if need else None, need)
    return q


def i8_dequantize(q, dtype=None, out=None, stream=None):
    """The values of an I8 as float32 (or `dtype`, or `out`'s type)."""
    h, c = mx4._h(), _c()
    device = _held(q, "q", None, q.group if isinstance(q, I8) else None)
    run = mx4._Run(device, stream)
    out, ty, ld = mx4._out(run, out, q.shape, h.float32 if out is None and dtype is None else dtype)
    run.call(c.dequantize, (q, out), *q.shape, q.group or 0, *q._pointers(), ty, out.data_ptr(), ld)
    return out


def i8_gemm(A, B, out=None, dtype=None, alpha=1.0, beta=0.0, stream=None):
    """alpha * A @ B^T + beta * out for I8 matrices A (M, K) and B (N, K) with a scale for each row.

    The sums are exact (K up to 131072), the scales enter in fp32.  out (M, N) is
    allocated as float32 (or `dtype`) if None (then beta must be 0).
    """
    h, c = mx4._h(), _c()
    device = _held(A, "A")
    _held(B, "B", device)
    (M, K), (N, K2) = A.shape, B.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    _sum(K)
    if out is None and beta != 0.0:
        raise ValueError("beta != 0 needs out")
    run = mx4._Run(device, stream)
    out, ty, ld = mx4._out(run, out, (M, N), h.float32 if out is None and dtype is None else dtype)
    run.call(c.gemm, (A, B, out), M, N, K, float(alpha), *A._pointers(), *B._pointers(), float(beta), ty, out.data_ptr(), ld)
    return out


def i8_linear(X, W, out=None, stream=None):
    """q(X) @ W^T for float rows X (M, K) and 8-bit weights W (N, K), in X's type.

    X is quantised by row on the way: the values of i8_gemm(i8_quantize(X), W),
    in one call, and for few tokens in one pass over W.
    """
    c = _c()
    ty, ldx = mx4._floats(X, "X")
    device = X.device
    _held(W, "W", device)
    (M, K), (N, K2) = X.shape, W.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    _sum(K)
    _layout(M, K, None)
    need = _scratch("linear_scratch", M, N, K, ty)
    run = mx4._Run(device, stream)
    out, _, ldy = mx4._out(run, out, (M, N), X.dtype)
    scratch = run.bytes(need) if need else None
    run.call(c.linear, (X, W, out), M, N, K, ty, X.data_ptr(), ldx, *W._pointers(), out.data_ptr(), ldy,
             scratch.data_ptr() if need else None, need)
    return out


@functools.lru_cache(maxsize=1024)
def _train_sizes(M, N, K):
    for n in (M, N, K):
        _sum(n)
    for r, c in ((M, K), (N, K), (M, N), (N, M)):
        _size(r, c)


def i8_train_forward(X, W, stream=None):
    """Y = q(X) q(W)^T for X (M, K) and a layer's weights W (N, K), in X's type.

    Returns (Y, saved); `saved` holds q(X) and q(W), a byte a value, which is
    all that i8_train_backward needs of this pass.  W may be an I8 with a scale
    for each row: weights quantised once for several calls.
    """
    c = _c()
    given = isinstance(W, I8)
    if mx4._column_major(X) or given or mx4._column_major(W):
        mx4._floats(X.t() if mx4._column_major(X) else X, "X")
        if given:
            _held(W, "W", X.device)
        else:
            mx4._floats(W.t() if mx4._column_major(W) else W, "W", X.device)
        _train_fit(X.shape, W.shape)
        x, w = i8_quantize(X, stream=stream), W if given else i8_quantize(W, stream=stream)
        return i8_gemm(x, w, dtype=X.dtype, stream=stream), (x, w)
    tx, ldx = mx4._floats(X, "X")
    device = X.device
    tw, ldw = mx4._floats(W, "W", device)
    M, N, K = _train_fit(X.shape, W.shape)
    run = mx4._Run(device, stream)
    x, w = _two(run, (M, K), (N, K))
    Y = run.empty((M, N), X.dtype)
    run.call(c.train_forward, (X, W), M, N, K, tx, X.data_ptr(), ldx, tw, W.data_ptr(), ldw, Y.data_ptr(), N, *x._pointers(),
             *w._pointers())
    return Y, (x, w)


def _train_fit(x, w):
    (M, K), (N, K2) = x, w
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    _train_sizes(M, N, K)
    return M, N, K


def i8_train_backward(dY, saved, dW=None, stream=None):
    """(dX, dW): the gradients of i8_train_forward with the rounding taken as the identity, from its 8-bit checkpoint.

    With q(X) = diag(x) Xq and q(W) = diag(w) Wq in whole numbers, dX = q(dY
    diag(w)) Wq, rounded to 8 bits by token, and dW = q(diag(x) dY)^T Xq, rounded
    to 16 bits by channel; all sums are exact.  dX comes in dY's type, dW in
    float32; a dW given is added to.
    """
    h, c = mx4._h(), _c()
    x, w = saved
    if mx4._column_major(dY):
        dY = _row_major(dY, stream)
    ty, ld = mx4._floats(dY, "dY")
    device = dY.device
    _held(x, "saved", device)
    _held(w, "saved", device)
    (M, N), (M2, K), (N2, K2) = dY.shape, x.shape, w.shape
    if (M, N, K) != (M2, N2, K2):
        raise ValueError(f"dY {(M, N)} does not fit what the forward pass saved of {M2} x {K} and {N2} x {K2} matrices")
    _train_sizes(M, N, K)
    need = _scratch("train_scratch", M, N, K)
    run = mx4._Run(device, stream)
    scratch = run.bytes(need) if need else None
    dX = run.empty((M, K), dY.dtype)
    beta = 0.0 if dW is None else 1.0
    dW, _, ldw = mx4._out(run, dW, (N, K), h.float32, "dW")
    run.call(c.train_backward, (dY, x, w, dW), M, N, K, ty, dY.data_ptr(), ld, *x._pointers(), *w._pointers(), dX.data_ptr(), K,
             beta, dW.data_ptr(), ldw, scratch.data_ptr() if need else None, need)
    return dX, dW


def _row_major(t, stream):
    """A row-major copy, made on the stream that uses it."""
    if stream is None:
        return t.contiguous()
    with mx4._h().torch.cuda.stream(stream):
        t.record_stream(stream)
        return t.contiguous()


def i8_swiglu_forward(GU, out=None, stream=None):
    """H = silu(G) * U for GU = [G, U] (M, 2 F), in GU's type.

    Returns (H, saved); `saved` holds G and U in 8 bits (group = 128), for
    i8_swiglu_backward.
    """
    c = _c()
    ty, ld = mx4._floats(GU, "GU")
    M, F = GU.shape[0], GU.shape[1] // 2
    if GU.shape[1] != 2 * F or GU.shape[1] > MAX_DIM:
        raise ValueError(f"GU must have an even number of columns, at most {MAX_DIM}, not {GU.shape[1]}")
    run = mx4._Run(GU.device, stream)
    g, u = _two(run, (M, F), (M, F), GROUP)
    out, _, ldh = mx4._out(run, out, (M, F), GU.dtype)
    run.call(c.swiglu_forward, (GU, out), M, F, ty, GU.data_ptr(), ld, out.data_ptr(), ldh, *g._pointers(), *u._pointers())
    return out, (g, u)


def i8_swiglu_backward(dH, saved, out=None, stream=None):
    """The gradient of GU (M, 2 F) from dH (M, F) and what i8_swiglu_forward saved, in dH's type."""
    c = _c()
    g, u = saved
    ty, ld = mx4._floats(dH, "dH")
    device = dH.device
    _held(g, "saved", device, GROUP)
    _held(u, "saved", device, GROUP)
    M, F = dH.shape
    if g.shape != (M, F) or u.shape != (M, F):
        raise ValueError(f"dH {(M, F)} does not fit what the forward pass saved of {g.shape} and {u.shape} matrices")
    if 2 * F > MAX_DIM:
        raise ValueError(f"2 F must be at most {MAX_DIM}")
    run = mx4._Run(device, stream)
    out, _, ldy = mx4._out(run, out, (M, 2 * F), dH.dtype)
    run.call(c.swiglu_backward, (dH, g, u, out), M, F, ty, dH.data_ptr(), ld, *g._pointers(), *u._pointers(), out.data_ptr(), ldy)
    return out
